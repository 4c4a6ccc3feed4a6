"""What a selection keeps at the ends of the order: the types' lowest values, equal
totals of different logits."""
import math

import numpy as np
import pytest
import torch

import rans_entropy_coding_b200 as rb

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("by", ["logits", "mask", "bias"])
def test_lowest_values_behind_tiles_of_nothing(by, dtype):
    """Rows of several tiles a block: three good tokens, then nothing, then tokens at
    the type's lowest value, which are continuations where there are no better ones."""
    n, v, count = 1300, 40000, 8  # (so many rows that a block walks several tiles of one)
    low = torch.finfo(dtype).min
    x = torch.full((n, v), -math.inf, device="cuda", dtype=dtype)
    good, tail = [3, 700, 1999], 39000
    x[:, good] = torch.tensor([1.0, 3.0, 2.0], device="cuda", dtype=dtype)
    x[:, tail:] = low
    adjust = None
    if by == "mask":
        allowed = x[0] > -math.inf
        x[x == -math.inf] = 0.0
        adjust = rb.LogitAdjust(mask=rb.pack_mask(allowed))
    elif by == "bias":  # (one more token touched, without a change)
        at = torch.zeros(n, dtype=torch.int64, device="cuda")
        adjust = rb.LogitAdjust(bias=(torch.tensor([700], dtype=torch.int32, device="cuda"),
                                      torch.zeros(1, device="cuda"), at, at + 1))
    s = torch.full((n,), -1.0, device="cuda")
    best, tokens, parents = rb.beam_select(x, s, 1, count, adjust)
    want = [700, 1999, 3] + list(range(tail, tail + count - 3))
    assert (tokens.cpu() == torch.tensor(want, dtype=torch.int32)).all()
    assert (parents == 0).all()
    lse = math.log(sum(math.exp(t) for t in (1.0, 2.0, 3.0)))
    exact = np.array([-1.0 + t - lse for t in (3.0, 2.0, 1.0, low, low, low, low, low)])
    got = best.cpu().numpy().astype(np.float64)
    assert (np.abs(got - exact) <= 2.0 ** -20 + 2.0 ** -24 * np.abs(exact)).all()


@pytest.mark.parametrize("v", [40, 5000, 70000])
@pytest.mark.parametrize("count", [1, 3, 6, 64])
def test_equal_totals_of_different_logits(v, count):
    """Logits too close for their totals to differ: the lower beam first, within a
    beam the larger logit, and of equal ones the lower token, whatever is thinned out
    on the way."""
    x = torch.zeros(2, v, device="cuda")
    x[0, [v - 1, 30, 7]] = torch.tensor([1e-20, 2e-20, -1e-20], device="cuda")
    x[1, [0, v - 3]] = torch.tensor([-3e-20, 3e-20], device="cuda")
    s = torch.full((2,), -2.0, device="cuda")
    rest = [t for t in range(v) if t not in (v - 1, 30, 7)]
    first = [30, v - 1] + rest + [7]
    rest = [t for t in range(v) if t not in (0, v - 3)]
    second = [v - 3] + rest + [0]
    want = ([(0, t) for t in first] + [(1, t) for t in second])[:count]
    best, tokens, parents = rb.beam_select(x, s, 2, count)
    n = len(want)
    assert list(zip(parents[0, :n].tolist(), tokens[0, :n].tolist())) == want
    for b in (0, 1):
        one = rb.beam_select(x[b:b + 1], s[:1], 1, count)[1][0].tolist()
        want = (first, second)[b][:count]
        assert one[:len(want)] == want


def test_equal_totals_of_far_scores():
    """Scores so large that a row's logits do not show in its totals."""
    v = 20000
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(3, v, device="cuda", generator=g)
    s = torch.full((3,), -1e30, device="cuda")
    _, tokens, parents = rb.beam_select(x, s, 3, 5)
    order = torch.sort(x[0], descending=True, stable=True).indices[:5]
    assert tokens[0].tolist() == order.tolist() and parents[0].tolist() == [0] * 5
