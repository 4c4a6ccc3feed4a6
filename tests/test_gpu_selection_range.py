"""Totals of rows far from 0, rising and falling over thousands, at the types' lowest
values, and under temperatures at the ends of their range."""
import math

import numpy as np
import pytest
import torch

import rans_entropy_coding_b200 as rb
from test_gpu_selection_sums import SUM, U, V, log_sum, select
from test_gpu_tokens import numpy_rows

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def rows_of(kind, dtype):
    g = torch.Generator().manual_seed(len(kind))
    body = torch.randn(2, V, generator=g)
    if kind == "rising":
        x = torch.linspace(-6000, 6000, V) + body
    elif kind == "falling":
        x = torch.linspace(6000, -6000, V) + body
    elif kind == "far":
        x = body + torch.tensor([[30000.0], [-30000.0]])
    elif kind == "steps":  # a little more with every tile
        x = body + torch.floor(torch.arange(V) / 4096.0) * 33.0
    elif kind == "across":
        x = body + torch.where(torch.arange(V) < V // 2, -5000.0, 4090.0)
    elif kind == "few":  # nothing but a few, behind tiles of nothing
        x = torch.full((2, V), -math.inf)
        x[:, 100000:100004] = torch.tensor([[8192.0], [-8192.0]]) + body[:, :4]
    elif kind == "lowest":
        x = torch.full((2, V), torch.finfo(dtype).min)
    else:  # "lowest and a few"
        x = torch.full((2, V), torch.finfo(dtype).min)
        x[1, 90000] = -3.0
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("kind", ["rising", "falling", "far", "steps", "across", "few", "lowest",
                                  "lowest and a few"])
@pytest.mark.parametrize("many", [False, True])
def test_totals_of_far_rows(kind, dtype, many):
    x = rows_of(kind, dtype)
    z = numpy_rows(x).astype(np.float64)
    top = z.max(1)
    with np.errstate(over="ignore"):
        log_share = -np.log(np.exp(z - top[:, None]).sum(1))  # of the best token
    s = torch.from_numpy(-log_share).float().cuda()
    best, tokens, _ = (select if many else rb.beam_select)(x, s, 1, 1)
    assert tokens[:, 0].tolist() == [int(t) for t in z.argmax(1)]
    want = s.cpu().numpy().astype(np.float64) + log_share
    assert np.abs(best[:, 0].cpu().numpy() - want).max() <= SUM + U * np.abs(want).max()
    # a beam among others
    total = (want[:, None] + (z - top[:, None])).reshape(-1)
    got = (select if many else rb.beam_select)(x, s, 2, 4)
    order = np.argsort(-total, kind="stable")[:4]
    assert (np.abs(total[got[2][0].cpu().numpy() * V + got[1][0].cpu().numpy()] - total[order])
            <= 2 * SUM).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("temperature", [1e-30, 1e-3, 1e3, 1e30])
def test_temperatures_at_the_ends(dtype, temperature):
    g = torch.Generator().manual_seed(3)
    size = 1.0 if temperature > 1.0 else temperature
    if dtype is F16:
        size = max(size, 2.0 ** -14)
    x = (torch.randn(3, V, generator=g) * size * 4).to(dtype).cuda()
    inv = np.float32(1) / np.float32(temperature)
    if dtype is F16 and temperature == 1e-30:
        x.mul_(0.0)
    z = (numpy_rows(x) * inv).astype(np.float64)
    exact = z.max(1) - log_sum(z)
    s = torch.from_numpy(-exact).float().cuda()
    rules = rb.LogitAdjust(temperature=temperature)
    for call in (rb.beam_select, select):
        best, tokens, _ = call(x, s, 1, 1, rules)
        assert tokens[:, 0].tolist() == [int(t) for t in z.argmax(1)]
        want = s.cpu().numpy().astype(np.float64) + exact
        assert np.abs(best[:, 0].cpu().numpy() - want).max() <= SUM + U * np.abs(want).max()


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
def test_a_row_of_lowest_values_is_even(dtype):
    """Such a beam's score and the logits do not cancel one another: its continuations
    have a V-th of it, and better beams come first."""
    v = 5000
    x = torch.full((3, v), torch.finfo(dtype).min, device="cuda", dtype=dtype)
    x[1] = 0.0
    x[1, 7] = 20.0
    s = torch.tensor([-1.0, -2.0, -9.0], device="cuda")
    best, tokens, parents = rb.beam_select(x, s, 3, 4)
    share = 20.0 - math.log(math.exp(20.0) + v - 1)
    want = [-2.0 + share] + [-1.0 - math.log(v)] * 3
    assert parents[0].tolist() == [1, 0, 0, 0] and tokens[0].tolist() == [7, 0, 1, 2]
    assert best[0].tolist() == pytest.approx(want, rel=1e-6)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("temperature", [1.0, 1000.0])
def test_what_is_masked_or_off_the_end_counts_for_nothing(dtype, temperature):
    """In rows at the lowest value too, where nothing lies below."""
    n, v = 2, 9001
    x = torch.full((n, v + 7), 0.0, device="cuda", dtype=dtype)[:, :v]
    x.fill_(torch.finfo(dtype).min)
    x[1] = -60000.0
    allowed = torch.ones(n, v, dtype=torch.bool, device="cuda")
    allowed[:, 100:] = torch.rand(v - 100, device="cuda") < 0.5
    left = int(allowed[0].sum())
    s = torch.full((n,), -1.0, device="cuda")
    for mask, size in ((rb.pack_mask(allowed), left), (None, v)):
        rules = rb.LogitAdjust(temperature=temperature, mask=mask)
        best, tokens, _ = rb.beam_select(x, s, 1, 3, rules)
        assert tokens.tolist() == [[0, 1, 2]] * n
        assert best.flatten().tolist() == pytest.approx([-1.0 - math.log(size)] * 6, rel=1e-6)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("below", [1.0, 2.0, 3.0])
def test_steps_near_zero_under_small_temperatures(dtype, below):
    """A type's smallest step is thousands after the temperature: all but the zeros
    count for nothing."""
    v, step = 9001, {F32: 2.0 ** -100, F16: 2.0 ** -24, BF16: 2.0 ** -100}[dtype]
    for over in (20.0, 70.0, 100.0, 130.0, 260.0, 1e4):  # what a step comes to
        x = torch.full((1, v), -below * step, device="cuda", dtype=dtype)
        x[0, 5:105] = 0.0
        s = torch.tensor([-1.0], device="cuda")
        best, tokens, _ = rb.beam_select(x, s, 1, 2, rb.LogitAdjust(temperature=step / over))
        share = math.log(100 + (v - 100) * math.exp(-below * over))
        assert tokens.tolist() == [[5, 6]]
        assert best[0].tolist() == pytest.approx([-1.0 - share] * 2, rel=1e-6)
