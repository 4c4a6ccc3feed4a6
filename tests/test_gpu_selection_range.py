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
