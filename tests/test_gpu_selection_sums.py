"""How far a selection's totals are from those of 64 bits where errors do not average
out: rows whose body is one logit or a few, far below the top, over a large vocabulary."""
import numpy as np
import pytest
import torch

import rans_entropy_coding_b200 as rb
from test_gpu_tokens import numpy_rows

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = 2.0 ** -24
# A term is 2^k 2^f, f = x log2 e - k, |f| <= 0.5, and in units of itself off by
#   f's two last roundings, each half a step of a number below 0.5, times ln 2:  0.35 U
#   the special function unit, over every float32 from -0.5 to 0.5:              2.45 U
# together 2.8 U, and a vector's terms add up in three additions of 1 U each; threads and
# blocks add in 64 bits.
SUM = 5.8 * U
V = 131072
ROWS = 4736  # so many that a block takes a whole row, top and body


def body_rows(kind, dtype, n, inv=1.0):
    """(rows, each with one token at the top, exact logits in 64 bits)."""
    g = torch.Generator().manual_seed(n + len(kind))
    top = 10.0 * torch.rand(n, 1, generator=g) - 3.0
    if kind == "flat":
        body = (top - 8.0 - 5.0 * torch.rand(n, 1, generator=g)).expand(n, V).clone()
    elif kind == "levels":  # a few, in random places
        levels = top - 8.0 - 5.0 * torch.rand(n, 4, generator=g)
        body = levels.gather(1, torch.randint(0, 4, (n, V), generator=g))
    else:  # near zero, in every vector the same
        top = 11.0 + 2.0 * torch.rand(n, 1, generator=g)
        body = (1e-3 * torch.rand(n, 4, generator=g)).repeat(1, V // 4)
    body = body / inv
    body[:, 77] = top[:, 0] / inv
    x = body.to(dtype).cuda()
    z = numpy_rows(x)
    return x, (z * np.float32(inv)).astype(np.float64) if inv != 1.0 else z.astype(np.float64)


def select(x, s, beams, count, adjust=None):
    """A selection among many dead beams, whose rows are not read."""
    n = x.shape[0]
    wide = torch.empty(ROWS, V, device="cuda", dtype=x.dtype)
    wide[:n] = x
    scores = torch.full((ROWS,), -float("inf"), device="cuda")
    scores[:n] = s
    return [g[:n // beams] for g in rb.beam_select(wide, scores, beams, count, adjust)]


def log_sum(z):
    m = z.max(1, keepdims=True)
    return m[:, 0] + np.log(np.exp(z - m).sum(1))


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("kind", ["flat", "levels", "near zero"])
@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_totals_of_bodies_of_few_logits(kind, dtype, temperature):
    n = 24
    inv = 1.0 if temperature == 1.0 else float(np.float32(1) / np.float32(temperature))
    x, z = body_rows(kind, dtype, n, inv)
    exact = z.max(1) - log_sum(z)
    # scores that leave totals near 0, whose rounding to float32 then hides nothing
    s = torch.from_numpy(-exact).float().cuda()
    rules = None if temperature == 1.0 else rb.LogitAdjust(temperature=temperature)
    best, tokens, _ = select(x, s, 1, 1, rules)
    assert (tokens == 77).all()
    want = s.cpu().numpy().astype(np.float64) + exact
    assert np.abs(best[:, 0].cpu().numpy() - want).max() <= SUM + U * np.abs(want).max()


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
def test_totals_of_touched_bodies(dtype):
    """Half of a row's logits equal and touched by penalties."""
    n = 6
    x, z = body_rows("flat", dtype, n)
    history = torch.arange(0, V, 2, device="cuda", dtype=torch.int32)
    at = torch.zeros(ROWS, dtype=torch.int64, device="cuda")
    rules = rb.LogitAdjust(presence=0.3, history=(history, at, at + history.numel()))
    z[:, ::2] = (z[:, ::2].astype(np.float32) - np.float32(0.3)).astype(np.float64)
    exact = z.max(1) - log_sum(z)
    s = torch.from_numpy(-exact).float().cuda()
    best, tokens, _ = select(x, s, 1, 1, rules)
    assert (tokens == 77).all()
    want = s.cpu().numpy().astype(np.float64) + exact
    assert np.abs(best[:, 0].cpu().numpy() - want).max() <= SUM + U * np.abs(want).max()


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
def test_beams_a_few_errors_apart_are_in_order(dtype):
    """Two beams of different bodies whose totals differ by little more than errors."""
    texts = 40
    x, z = body_rows("flat", dtype, 2 * texts)
    exact = z.max(1) - log_sum(z)
    gap = np.linspace(12.0, 24.0, texts) * U * np.where(np.arange(texts) % 2, 1, -1)
    s = -exact
    s[1::2] += gap
    s = s.astype(np.float32)
    total = (s.astype(np.float64) + exact).reshape(texts, 2)
    apart = np.abs(total[:, 0] - total[:, 1]) > 2 * SUM
    assert apart.sum() > texts // 2
    _, tokens, parents = select(x, torch.from_numpy(s).cuda(), 2, 2)
    assert (tokens == 77).all()
    assert (parents[:, 0].cpu().numpy() == total.argmax(1))[apart].all()
