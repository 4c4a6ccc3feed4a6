"""Refusals of selections and state moves that must come before anything has run, at the C
entry points without a GPU: what is not refused there would fail with RANS_ERR_CUDA."""
import ctypes

import pytest

import rans_entropy_coding_b200 as rb
from rans_entropy_coding_b200 import build as rbuild
from test_beams import A, adjust, select


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rb.lib()


def states(n, large):
    """n small states; the one at `large` with more blocks than a launch takes."""
    s = (rb.rans_state * n)()
    for i in range(n):
        s[i].data, s[i].row_stride, s[i].segment_stride = A(4 + i), 64, 64
        s[i].positions, s[i].segments, s[i].position_bytes = 4, 1, 16
    s[large].data = 1 << 60
    s[large].row_stride, s[large].positions, s[large].position_bytes = 1 << 42, 1 << 38, 16
    return s


@pytest.mark.parametrize("n,large", [(1, 0), (56, 55), (57, 56), (200, 57), (200, 199)])
def test_states_too_large_for_a_later_launch_are_refused_before_the_first(lib, n, large):
    s = states(n, large)
    assert lib.rans_reorder_states(s, n, 8, 2, A(1), A(2), None, None) == rb.ERR_ARG
    assert lib.rans_reorder_states_check(s, n, 8, 2, A(1), A(2), None) == rb.ERR_ARG


def test_the_check_of_states_alone(lib):
    s = states(3, 2)
    for args, want in (((s, 2, 8, 2, A(1), A(2), None), rb.OK),
                       ((s, 2, 8, 2, None, None, None), rb.ERR_ARG),
                       ((s, 2, 8, 65, A(1), None, None), rb.ERR_ARG),
                       ((s, 2, 8, 2, A(4), None, None), rb.ERR_ARG),
                       ((None, 0, 8, 2, None, None, None), rb.OK),
                       ((s, 2, 0, 2, None, None, None), rb.OK),
                       ((s, 2, 8, 2, A(1), A(2), A(3) + 8), rb.ERR_ARG)):
        assert lib.rans_reorder_states_check(*args) == want


@pytest.mark.parametrize("at", [A(2), A(3), A(4), A(5), A(6)], ids=["scores", "tokens", "parents",
                                                                  "workspace", "status"])
@pytest.mark.parametrize("what", [
    dict(mask=-4, mask_stride=4), dict(mask=-124, mask_stride=4), dict(mask=-12),
    dict(params=-8), dict(params=-124),
    dict(history=-40, history_begin=-8, history_end=1 << 40),
    dict(history=-40, history_begin=1 << 40, history_end=-56),
    dict(bias_ids=-40, bias_values=-40, bias_begin=-8, bias_end=1 << 40),
    dict(bias_ids=-40, bias_values=-40, bias_begin=1 << 40, bias_end=-56)], ids=str)
def test_selections_that_would_write_to_rules_are_refused(lib, what, at):
    """8 rows of 100 tokens; offsets from a result's place (strides and lengths as they are)."""
    rules = adjust(**{k: x if k == "mask_stride" else at + x for k, x in what.items()})
    assert select(lib, adj=rules, status=A(6)) == rb.ERR_ARG
