"""Beam search without a GPU: refusals at the C entry points and in the Python
layer."""
import ctypes

import pytest
import torch

import rans_entropy_coding_b200 as rb
from rans_entropy_coding_b200 import build as rbuild

P = 1 << 20  # an address that nothing reads: every call here is refused on the host


def A(k):
    """Addresses far from P and from one another."""
    return P + (k << 24)


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rb.lib()


def logits(data=P, dtype=0, vocab=100, rows=8, stride=100):
    c = rb.rans_logits()
    c.data, c.dtype, c.vocab, c.rows, c.row_stride = data, dtype, vocab, rows, stride
    return ctypes.byref(c)


def adjust(**kw):
    c = rb.rans_adjust()
    c.repetition = c.inv_temperature = 1.0
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def select(lib, lg=None, adj=None, scores=A(1), beams=4, count=8, out=A(2), tokens=A(3),
           parents=A(4), ws=A(5), size=1 << 22, status=None):
    return lib.rans_beam_select(lg or logits(), adj, scores, beams, count, out, tokens, parents, ws,
                                size, status, None)


@pytest.mark.parametrize("bad", [
    dict(lg=logits(None)), dict(lg=logits(vocab=0)), dict(lg=logits(stride=99)),
    dict(lg=logits(rows=7)), dict(lg=logits(dtype=3)), dict(adj=adjust(repetition=0.0)),
    dict(adj=adjust(mask=P, mask_stride=3)), dict(scores=None), dict(scores=A(1) + 2),
    dict(beams=0), dict(beams=65), dict(beams=3), dict(count=0), dict(count=129), dict(out=None),
    dict(tokens=None), dict(parents=None), dict(tokens=A(3) + 1), dict(ws=None),
    dict(ws=A(5) + 128), dict(status=A(6) + 8), dict(out=A(1) + 16), dict(out=P + 64),
    dict(tokens=A(2) + 60), dict(parents=A(3)), dict(status=A(2)),
    dict(adj=adjust(history=A(3), history_begin=A(7), history_end=A(8), history_len=5))], ids=str)
def test_bad_selections_are_refused(lib, bad):
    assert select(lib, **bad) == rb.ERR_ARG


def test_no_rows_do_nothing(lib):
    assert select(lib, logits(None, rows=0), scores=None, out=None, tokens=None, parents=None,
                  ws=None, size=0) == rb.OK
    assert lib.rans_reorder_states(None, 0, 5, 4, None, None, None, None) == rb.OK
    assert lib.rans_reorder_states(state(), 1, 0, 4, None, None, None, None) == rb.OK
    assert advance(lib, texts=0, **{k: None for k in ARRAYS}) == rb.OK
    for bad in ((3, 1, 1, 1), (0, -1, 1, 1), (0, 1, 0, 1), (0, 1, 1, 0), (0, 1, 1, 129),
                (0, 1, rb.MAX_VOCAB + 1, 1)):
        assert lib.rans_beam_workspace_bytes(*bad) == 0


ARRAYS = ["scores", "tokens", "parents", "history", "window_end", "lengths", "over", "done_scores",
          "done_lengths", "done_tokens", "done_counts"]


def advance(lib, count=8, cands=(A(1), A(2), A(3)), **kw):
    c = rb.rans_beams()
    c.texts, c.beams, c.capacity, c.n_ends, c.ends = 2, 4, 10, 1, A(4)
    for i, k in enumerate(ARRAYS):
        setattr(c, k, A(5 + i))
    for k, v in kw.items():
        setattr(c, k, v)
    return lib.rans_beam_advance(*cands, count, ctypes.byref(c), None)


@pytest.mark.parametrize("bad", [
    dict(count=0), dict(count=129), dict(texts=-1), dict(beams=0), dict(beams=65),
    dict(capacity=0), dict(n_ends=-1), dict(n_ends=65), dict(ends=None),
    dict(length_penalty=float("nan")), dict(length_penalty=float("inf")),
    dict(cands=(None, A(2), A(3))), dict(cands=(A(1), A(2) + 2, A(3))),
    dict(cands=(A(1), A(2), A(5))), dict(window_end=A(9) + 4), dict(history=A(5)),
    dict(history=A(4)), dict(over=A(10) + 4)] + [{k: None} for k in ARRAYS], ids=str)
def test_bad_advances_are_refused(lib, bad):
    assert advance(lib, **bad) == rb.ERR_ARG


def state(**kw):
    c = rb.rans_state()
    c.data, c.row_stride, c.segment_stride, c.positions = A(1), 400, 100, 10
    c.segments, c.position_bytes = 4, 10
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def reorder(lib, s=None, n=1, texts=2, beams=4, parents=A(2), lengths=A(3), status=None):
    return lib.rans_reorder_states(s or state(), n, texts, beams, parents, lengths, status, None)


@pytest.mark.parametrize("bad", [
    dict(s=state(data=None)), dict(s=state(row_stride=399)), dict(s=state(segment_stride=99)),
    dict(s=state(positions=-1)), dict(s=state(segments=-1)), dict(s=state(position_bytes=-1)),
    dict(s=state(row_stride=-400)), dict(s=state(positions=1 << 60)),
    dict(s=state(row_stride=1 << 62)), dict(n=-1), dict(n=rb.MAX_STATES + 1), dict(texts=-1),
    dict(texts=1 << 31), dict(beams=0), dict(beams=65), dict(parents=None),
    dict(parents=A(2) + 2), dict(lengths=A(3) + 2), dict(status=A(4) + 4),
    dict(parents=A(1) + 3196), dict(lengths=A(1)), dict(status=A(1) + 256)], ids=str)
def test_bad_states_are_refused(lib, bad):
    assert reorder(lib, **bad) == rb.ERR_ARG


def test_states_that_overlap_are_refused(lib):
    def two(**kw):
        both = (rb.rans_state * 3)()
        for i, x in enumerate((state(), state(data=A(4)), state(**kw))):
            both[i] = x._obj
        return lib.rans_reorder_states(both, 3, 2, 4, A(2), A(3), None, None)

    assert two() == rb.ERR_ARG                            # the same state twice
    assert two(data=A(1) + 3199) == rb.ERR_ARG
    assert two(data=A(4) + 4) == rb.ERR_ARG
    assert two(data=A(1) + 100, row_stride=800) == rb.ERR_ARG
    assert two(data=A(1) - 7 * 800 - 399, row_stride=800) == rb.ERR_ARG


def test_host_tensors_and_bad_parts_are_refused(lib):
    x, s = torch.zeros(4, 10), torch.zeros(4)
    for call in (lambda: rb.beam_select(x, s, 2), lambda: rb.beam_select(None, s, 2),
                 lambda: rb.reorder_states(x, torch.zeros(2, 2, dtype=torch.int32)),
                 lambda: rb.reorder_states(x, None),
                 lambda: rb.BeamSearch(1, 0, 5), lambda: rb.BeamSearch(1, 65, 5),
                 lambda: rb.BeamSearch(1, 2, 0), lambda: rb.BeamSearch(-1, 2, 5),
                 lambda: rb.BeamSearch(1, 2, 5, ends=range(65)),
                 lambda: rb.BeamSearch(1, 2, 5, ends=[-1]),
                 lambda: rb.BeamSearch(1, 2, 5, length_penalty=float("nan"), device="cpu"),
                 lambda: rb.BeamSearch(1, 2, 5, pad=1 << 31),
                 lambda: rb.BeamSearch(1, 2, 5, device="cpu")):
        with pytest.raises(ValueError):
            call()
