"""Tokens under a model's logits, without a GPU: refusals at the C entry
points and in the Python layer, the mask packing, and the oracle's own coder."""
import contextlib
import ctypes
import weakref
from fractions import Fraction

import numpy as np
import pytest
import torch

import rans_entropy_coding_b200 as rb
import token_oracle as TO
from rans_entropy_coding_b200 import build as rbuild

P = 1 << 20  # an address that nothing reads: every call here is refused on the host


def A(k):
    """Addresses far from P and from one another."""
    return P + (k << 24)


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rb.lib()


def logits(data=P, dtype=0, vocab=100, rows=4, stride=100):
    c = rb.rans_logits()
    c.data, c.dtype, c.vocab, c.rows, c.row_stride = data, dtype, vocab, rows, stride
    return c


def adjust(**kw):
    c = rb.rans_adjust()
    c.repetition = c.inv_temperature = 1.0
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_LOGITS = [dict(data=None), dict(dtype=3), dict(dtype=-1), dict(vocab=0),
              dict(vocab=rb.MAX_VOCAB + 1, stride=rb.MAX_VOCAB + 1), dict(rows=-1),
              dict(stride=99), dict(data=P + 2)]
BAD_ADJUST = [dict(repetition=0.0), dict(repetition=float("inf")), dict(repetition=float("nan")),
              dict(inv_temperature=0.0), dict(inv_temperature=-1.0),
              dict(inv_temperature=float("inf")), dict(frequency=float("nan")),
              dict(presence=float("inf")), dict(history=P), dict(history=P, history_begin=P),
              dict(history=P, history_begin=P, history_end=P, history_len=-1), dict(bias_ids=P),
              dict(bias_ids=P, bias_values=P, bias_begin=P),
              dict(bias_ids=P, bias_values=P, bias_begin=P, bias_end=P, bias_len=-1),
              dict(mask=P, mask_stride=3), dict(mask=P, mask_stride=-4)]


def calls(lib, lg, ad=None):
    """Every entry point that takes logits, with good other arguments."""
    a = None if ad is None else ctypes.byref(ad)
    x = ctypes.byref(lg)
    yield lib.rans_adjust_logits(x, a, A(1), 0, 100, None)
    yield lib.rans_token_intervals(x, a, A(1), A(2), A(3), A(4), None)
    yield lib.rans_decode_tokens(x, a, A(1), 64, A(2), 8, None, A(3), A(4), A(5), A(6), None)
    if ad is None:
        yield lib.rans_distill_forward(x, A(1), A(2), 5, 1.0, 1, A(3), A(4), A(5), None)
        yield lib.rans_distill_backward(x, A(1), A(2), 5, 1.0, A(3), A(4), A(5), 100, None)
        yield lib.rans_distill(x, A(1), A(2), 5, 1.0, 1, A(3), A(4), A(5), 100, A(6), None)


@pytest.mark.parametrize("bad", BAD_LOGITS, ids=str)
def test_bad_logits_are_refused(lib, bad):
    assert list(calls(lib, logits(**bad))) == [rb.ERR_ARG] * 6


@pytest.mark.parametrize("bad", BAD_ADJUST, ids=str)
def test_bad_adjustments_are_refused(lib, bad):
    assert list(calls(lib, logits(), adjust(**bad))) == [rb.ERR_ARG] * 3


def test_no_rows_do_nothing(lib):
    assert list(calls(lib, logits(rows=0, data=None))) == [rb.OK] * 6
    x = ctypes.byref(logits(rows=0, data=None))
    assert lib.rans_adjust_logits(x, None, None, 0, 0, None) == rb.OK
    assert lib.rans_token_states(None, 0, P, 0, None, P, None) == rb.OK
    assert lib.rans_token_states_finish(None, 0, None, P, None) == rb.OK


def test_results_that_overlap_are_refused(lib):
    x = logits(rows=3, vocab=100, stride=256)

    def result(out, dtype=0, stride=256, lg=x):
        return lib.rans_adjust_logits(ctypes.byref(lg), None, out, dtype, stride, None)

    assert result(P, dtype=1) == rb.ERR_ARG              # in place with another type
    assert result(P, stride=300) == rb.ERR_ARG           # or another stride
    assert result(P + 4) == rb.ERR_ARG                   # shifted by one element
    assert result(P + 4 * 99) == rb.ERR_ARG
    assert result(P - 4 * 99) == rb.ERR_ARG
    assert result(P + 4 * 157) == rb.ERR_ARG             # its row 0 reaches row 1
    assert result(P + 4 * 355) == rb.ERR_ARG             # the last element of row 1
    assert result(P + 4, lg=logits(rows=1)) == rb.ERR_ARG
    assert result(0) == rb.ERR_ARG
    assert result(P + (1 << 20), dtype=7) == rb.ERR_ARG
    assert result(P + (1 << 20), stride=99) == rb.ERR_ARG
    assert result(P + (1 << 20) + 2) == rb.ERR_ARG       # not aligned to the type
    assert lib.rans_distill(ctypes.byref(x), P, P, 5, 1.0, 1, P, P, P + 4, 256, P,
                            None) == rb.ERR_ARG
    assert lib.rans_distill_backward(ctypes.byref(x), P, P, 5, 1.0, P, P, P + 4, 256,
                                     None) == rb.ERR_ARG


def test_bad_pointers_and_counts_are_refused(lib):
    x = ctypes.byref(logits())
    S = rb.ERR_ARG
    good = [x, None, A(1), A(2), A(3), A(4), None]
    for k, v in ((2, None), (3, None), (4, None), (5, None), (5, A(4) + 8),
                 (3, A(1)), (4, A(1) + 12), (4, A(2) - 12), (5, A(1) & ~255)):
        args = list(good)
        args[k] = v
        assert lib.rans_token_intervals(*args) == S, (k, v)
    good = [x, None, A(1), 64, A(2), 8, A(3), A(4), A(5), A(6), A(7), None]
    for k, v in ((2, None), (2, A(1) + 2), (4, None), (5, -1), (7, None), (8, None), (9, None),
                 (10, None), (10, A(7) + 4),
                 (8, A(4) + 16),            # states that overlap but are not the same
                 (9, A(3) + 4),             # tokens over stream ids
                 (9, A(4)), (9, A(5) + 124), (6, A(5)), (10, A(3)), (10, A(4))):
        args = list(good)
        args[k] = v
        assert lib.rans_decode_tokens(*args) == S, (k, v)
    args = list(good)
    args[5], args[6] = 3, None              # fewer streams than rows
    assert lib.rans_decode_tokens(*args) == S
    assert lib.rans_token_states(P, 64, None, 2, P, P, None) == S
    assert lib.rans_token_states(P, 64, P, 2, None, P, None) == S
    assert lib.rans_token_states(P + 1, 64, P, 2, P, P, None) == S
    assert lib.rans_token_states_finish(P, 2, None, P, None) == S
    assert lib.rans_token_states_finish(P, -1, P, P, None) == S
    for K in (0, -1, rb.MAX_TOP + 1):
        assert lib.rans_distill_forward(x, P, P, K, 1.0, 1, P, P, P, None) == S
    for t in (0.0, -1.0, float("inf"), float("nan")):
        assert lib.rans_distill_forward(x, P, P, 4, t, 1, P, P, P, None) == S
    assert lib.rans_distill_forward(x, P, P, 4, 1.0, 1, P, P + 8, P, None) == S  # stats alignment
    assert lib.rans_distill_forward(x, None, P, 4, 1.0, 1, P, P, P, None) == S
    assert lib.rans_distill(x, P, P, 4, 1.0, 1, None, P, P + (1 << 20), 100, P, None) == S


def test_encode_intervals_refusals(lib):
    def call(ch, starts=P, freqs=P, n=10, out=P, cap=4096, offs=P, ws=P, ws_bytes=1 << 20):
        return lib.rans_encode_intervals(starts, freqs, n, ctypes.byref(ch.c), out, cap, offs, ws,
                                         ws_bytes, None)

    one = rb.Chunking.contig(2)
    assert call(rb.Chunking.contig(2, interleave=32)) == rb.ERR_ARG
    assert call(rb.Chunking.contig(2, index_block=2)) == rb.ERR_ARG
    assert call(rb.Chunking.contig(2, fmt="rans32_16")) == rb.ERR_ARG
    assert call(rb.Chunking.contig(2, alias=True)) == rb.ERR_ARG
    assert call(rb.Chunking.tiled((1, 1, 2, 5), 1, 2, 5, interleave=1)) == rb.ERR_ARG
    assert call(one, starts=None) == rb.ERR_ARG
    assert call(one, out=P + 2) == rb.ERR_ARG
    assert call(one, ws=P + 16) == rb.ERR_ARG
    assert call(one, offs=None) == rb.ERR_ARG
    assert call(one, n=-1) == rb.ERR_ARG
    assert call(one, ws_bytes=256) == rb.ERR_CAPACITY


def test_python_layer_refuses_host_tensors_and_bad_shapes():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        rb.adjust_logits(x, rb.LogitAdjust())
    with pytest.raises(ValueError):
        rb.distill_loss(x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1))
    for kw in (dict(temperature=0.0), dict(temperature=float("nan")), dict(repetition=-1.0),
               dict(frequency=float("inf")), dict(temperature=float("inf"))):
        with pytest.raises(ValueError):
            rb.LogitAdjust(**kw)
    with pytest.raises(ValueError):   # host tensors
        rb.LogitAdjust(mask=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):   # wrong type
        rb.LogitAdjust(mask=torch.zeros(4, dtype=torch.int64))


@pytest.mark.parametrize("vocab", [1, 31, 32, 33, 100])
def test_pack_mask(vocab):
    g = torch.Generator().manual_seed(vocab)
    ok = torch.rand(3, vocab, generator=g) < 0.5
    words = rb.pack_mask(ok)
    assert words.dtype == torch.int32 and words.shape == (3, (vocab + 31) // 32)
    for r in range(3):
        assert np.array_equal(TO.allowed(dict(mask=words.numpy()), r, vocab), ok[r].numpy())
    assert torch.equal(rb.pack_mask(ok[1]), words[1])


def test_oracle_intervals_tile_the_range_and_follow_the_softmax():
    rng = np.random.default_rng(3)
    row = rng.normal(0, 3, 500).astype(np.float32)
    row[7] = -np.inf
    adj = dict(temperature=0.7)
    b = TO.bounds(row, adj, 0)
    f = np.diff(np.array(b))
    assert b[0] == 0 and b[-1] == 1 << 24 and f[7] == 0 and (np.delete(f, 7) >= 1).all()
    z = row.astype(np.float64) / 0.7
    p = np.exp(z - z.max())
    p /= p.sum()
    # 2^f to 1.02e-4 (also in the sum), a weight's rounding half a unit of 2^21
    # times the largest weight's share, the room given up for N ones, flooring
    bound = 2.1e-4 * p + 0.5 * 2.0 ** -21 * (1 + 500 * p) + 500 * 2.0 ** -24 * p + 2.0 ** -24 * 2
    assert (np.abs(f * 2.0 ** -24 - p) <= bound).all()


def test_oracle_coder_round_trip():
    rng = np.random.default_rng(4)
    row = rng.normal(0, 4, 300).astype(np.float32)
    b = TO.bounds(row, {}, 0)
    tokens = rng.integers(0, 300, 200)
    data = TO.encode([b[t] for t in tokens], [b[t + 1] - b[t] for t in tokens])
    d = TO.Decoder(data)
    assert [d.step(b) for _ in tokens] == list(tokens)
    assert d.x == TO.LOW and d.at == len(d.words)


# ------------------------------------------------------ the Python layer --
class Untouchable:
    """A library whose every call is a failure of the checks before it."""

    def __getattr__(self, name):
        raise AssertionError("%s was called" % name)


def test_host_tensors_never_reach_the_library(monkeypatch):
    """Every tensor on the host: no entry point may take its addresses for
    device ones (and the calls that need no logits have only these checks)."""
    i32 = torch.zeros(8, dtype=torch.int32)
    data = torch.zeros(64, dtype=torch.uint8)
    offs = torch.tensor([0, 32, 64])
    states = torch.zeros(2, 2, dtype=torch.int64)
    status = torch.zeros(32, dtype=torch.int64)
    x = torch.zeros(2, 8)
    two, chunks = i32[:2].clone(), rb.Chunking.contig(2)
    buf = torch.zeros(4096, dtype=torch.uint8)
    ids, lp = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1)
    w, stats = torch.zeros(2), torch.zeros(2, 8)
    monkeypatch.setattr(rb.tokens.L, "lib", lambda: Untouchable())
    monkeypatch.setattr(rb.tokens.L, "rans_num_streams", lambda chunking, n: 2)
    for call in (
            lambda: rb.encode_intervals(i32, i32, chunks),
            lambda: rb.rans_encode_intervals(i32, i32, 8, chunks, buf, offs, buf),
            lambda: rb.token_states(data, offs),
            lambda: rb.token_states(data, offs, status),
            lambda: rb.rans_token_states(data, offs, states, status),
            lambda: rb.rans_token_states_finish(offs, states, status),
            lambda: rb.decode_tokens(x, data, offs, states),
            lambda: rb.rans_decode_tokens(x, None, data, offs, None, states, states, two, status),
            lambda: rb.token_intervals(x, two),
            lambda: rb.rans_token_intervals(x, None, two, two, two, status),
            lambda: rb.rans_adjust_logits(x, None, x),
            lambda: rb.rans_distill(x, ids, lp, 1.0, True, w, w, x, status),
            lambda: rb.rans_distill_forward(x, ids, lp, 1.0, True, w, stats, status),
            lambda: rb.rans_distill_backward(x, ids, lp, 1.0, stats, w, x),
            lambda: rb.encode_intervals([1, 2], [1, 2], chunks)):
        with pytest.raises(ValueError):
            call()


class Watching:
    """A library that asks, in every call, whether the tensors whose addresses
    it was given are still there."""

    def __init__(self):
        self.refs, self.calls = [], []

    def __getattr__(self, name):
        def call(*args):
            mine = [r for a, r in self.refs if a in args]
            self.calls.append((name, len(mine), [r() is not None for r in mine]))
            self.refs.clear()
            return rb.OK
        return call


@pytest.fixture
def watched(monkeypatch):
    """The Python layer on host tensors, with a Watching in the library's place."""
    T, lib = rb.tokens, Watching()

    def note(x):
        lib.refs.append((x.data_ptr(), weakref.ref(x)))
        return x

    def rows_of(x, what="logits"):
        return 0, x.shape[0], x.shape[1], 0, x.shape[1]

    monkeypatch.setattr(T, "_rows", rows_of)
    monkeypatch.setattr(T, "_tensor", lambda x, *args: note(x).data_ptr())
    monkeypatch.setattr(T, "_device", lambda x, what: 0)
    monkeypatch.setattr(T, "_place", lambda dev, stream: contextlib.nullcontext())
    monkeypatch.setattr(T, "_raw_stream", lambda dev: 0)
    # (an allocation that nothing else holds; its address is its own)
    monkeypatch.setattr(T, "new_status",
                        lambda dev="cuda": note(torch.zeros(1 << 16, dtype=torch.int64)))
    monkeypatch.setattr(T, "_status", lambda status, dev: T.new_status() if status is None
                        else note(status))
    monkeypatch.setattr(T.L, "lib", lambda: lib)
    return lib


def test_what_a_call_reads_outlives_it(watched):
    x, ids, lp = torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    i32 = torch.zeros(3, dtype=torch.int32)
    data, offs = torch.zeros(64, dtype=torch.uint8), torch.tensor([0, 16, 32, 48])
    states, w = torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3)
    stats = torch.zeros(3, 8)
    rb.token_intervals(x, i32)
    rb.rans_token_intervals(x, None, i32, i32, i32, None)
    rb.token_states(data, offs)
    rb.rans_token_states(data, offs, states, None)
    rb.decode_tokens(x, data, offs, states)
    rb.rans_decode_tokens(x, None, data, offs, None, states, states, i32, None)
    rb.rans_token_states_finish(offs, states, None)
    rb.rans_distill_forward(x, ids, lp, 1.0, True, w, stats, None)
    rb.rans_distill(x, ids, lp, 1.0, True, w, w, x, None)
    rb.distill_loss_and_grad(x, ids, lp, w)
    assert len(watched.calls) == 10
    y = x.clone().requires_grad_()
    # (distill_loss itself asks for CUDA logits)
    for reduce in (torch.sum, torch.mean, lambda t: (t * w).sum()):
        reduce(rb.tokens._Distill.apply(y, ids, lp, 1.0, True, None)).backward()
    names = [c[0] for c in watched.calls]
    assert names[10:] == ["rans_distill_forward", "rans_distill_backward"] * 3
    for name, seen, alive in watched.calls:
        assert seen >= 2 and all(alive), (name, alive)


def test_a_number_and_a_row_that_holds_it_have_the_same_reciprocal():
    """The float32 nearest to 1 / float32(T), here from exact fractions."""
    for i in range(1, 800):
        t = i / 200
        f = np.float32(t)
        exact = 1 / Fraction(float(f))
        near = np.float32(float(exact))
        best = min((np.nextafter(near, np.float32(0)), near, np.nextafter(near, np.float32(9))),
                   key=lambda c: abs(Fraction(float(c)) - exact))
        assert np.float32(rb.tokens._inverse(t)) == best, t
        assert torch.tensor([f]).double().reciprocal().float().item() == best, t
        assert rb.LogitAdjust(temperature=t)._c[12:16] == best.tobytes(), t
    for kw in (dict(repetition=1e-50), dict(repetition=1e39), dict(frequency=1e39),
               dict(presence=-1e39), dict(temperature=1e-50), dict(temperature=1e-39),
               dict(temperature=1e39)):
        with pytest.raises(ValueError):
            rb.LogitAdjust(**kw)


def test_numbers_beside_per_row_tensors_are_checked_too(monkeypatch):
    """... and are float32 whatever the default type is."""
    monkeypatch.setattr(rb.LogitAdjust, "_on", lambda self, x, n: -1)
    monkeypatch.setattr(rb.tokens, "_place", lambda dev, stream: contextlib.nullcontext())
    monkeypatch.setattr(rb.tokens, "_MadeOn", lambda x, dev: None)
    rows = torch.full((3,), 0.7)
    for kw in (dict(repetition=-1.0), dict(repetition=0.0), dict(repetition=1e39),
               dict(frequency=float("nan")), dict(presence=float("inf"))):
        with pytest.raises(ValueError):
            rb.LogitAdjust(temperature=rows, **kw)
    for t in (0.0, -1.0, float("inf"), float("nan"), 1e39, 1e-39):
        with pytest.raises(ValueError):
            rb.LogitAdjust(repetition=rows, temperature=t)
    torch.set_default_dtype(torch.float64)
    try:
        a = rb.LogitAdjust(temperature=rows, repetition=1.1, frequency=0.25)
    finally:
        torch.set_default_dtype(torch.float32)
    params = a._keep[-1]
    assert params.dtype == torch.float32 and params.shape == (3, 4)
    want = np.array([1.1, 0.25, 0.0, 1 / np.float32(0.7)], np.float32)
    assert np.array_equal(params.numpy(), np.tile(want, (3, 1)))


def test_autograd_learns_of_what_a_call_writes(watched, monkeypatch):
    monkeypatch.setattr(rb.tokens.L, "rans_num_streams", lambda chunking, n: 2)
    x, ids, lp = torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    i32, w, stats = torch.zeros(3, dtype=torch.int32), torch.zeros(3), torch.zeros(3, 8)
    data, offs = torch.zeros(64, dtype=torch.uint8), torch.tensor([0, 16, 32, 48])
    states, chunks = torch.zeros(3, 2, dtype=torch.int64), rb.Chunking.contig(2)

    def new(like):
        return torch.zeros_like(like)

    # (a call given its outputs, the outputs)
    for call, outs in (
            (lambda o: rb.adjust_logits(x, None, out=o), (x,)),
            (lambda o: rb.rans_adjust_logits(x, None, o), (x,)),
            (lambda a, b: rb.token_intervals(x, i32, starts=a, freqs=b), (i32, i32)),
            (lambda a: rb.token_intervals(x, i32, freqs=a), (i32,)),
            (lambda a, b: rb.rans_token_intervals(x, None, i32, a, b, None), (i32, i32)),
            (lambda a, b: rb.encode_intervals(i32, i32, chunks, out=a, ws=b), (data, data)),
            (lambda a, b, c: rb.rans_encode_intervals(i32, i32, 3, chunks, a, b, c),
             (data, offs, data)),
            (lambda a: rb.rans_token_states(data, offs, a, None), (states,)),
            (lambda a, b: rb.decode_tokens(x, data, offs, states, out_states=a, tokens=b),
             (states, i32)),
            (lambda a, b: rb.rans_decode_tokens(x, None, data, offs, None, states, a, b, None),
             (states, i32)),
            (lambda a, b: rb.rans_distill_forward(x, ids, lp, 1.0, True, a, b, None), (w, stats)),
            (lambda a: rb.rans_distill_backward(x, ids, lp, 1.0, stats, w, a), (x,)),
            (lambda a, b: rb.rans_distill(x, ids, lp, 1.0, True, w, a, b, None), (w, x)),
            (lambda a: rb.distill_loss_and_grad(x, ids, lp, w, grad=a), (x,))):
        mine = [new(o) for o in outs]
        call(*mine)
        assert [o._version for o in mine] == [1] * len(mine)
    for read in (x, ids, lp, i32, w, data, offs, states, stats):
        assert read._version == 0
    # a backward pass whose logits were written over says so
    y = torch.zeros(3, 8, requires_grad=True)
    z = y * 1.0
    loss = rb.tokens._Distill.apply(z, ids, lp, 1.0, True, None).sum()
    rb.adjust_logits(z, None, out=z)
    with pytest.raises(RuntimeError, match="inplace operation"):
        loss.backward()


def test_wide_token_ids_do_not_wrap_into_the_vocabulary():
    from rans_entropy_coding_b200.interface import _token_ids
    wide = torch.tensor([[5, -1, -2], [2**32 + 5, 2**31, -2**32 - 1], [-2**33, 2**31 - 1, 0]])
    ids = _token_ids(wide, "cpu")
    assert ids.dtype == torch.int32
    assert ids.tolist() == [5, -1, -2, 2**31 - 1, 2**31 - 1, -2, -2, 2**31 - 1, 0]
    assert all(v in (-1, -2, 2**31 - 1) or 0 <= v < 6 for v in ids.tolist())
    for same in ([3, 1], np.array([3, 1]), torch.tensor([3, 1], dtype=torch.int16),
                 torch.tensor([[3], [1]], dtype=torch.int32)):
        assert _token_ids(same, "cpu").tolist() == [3, 1]
    assert _token_ids([], "cpu").tolist() == []


def test_a_status_is_read_on_its_own_device(monkeypatch):
    """With another device current, its stream is not ordered behind the calls
    that wrote the word (and a default stream's address names the current one)."""
    now, got = ["cuda:0"], []

    class Word:
        device = torch.device("cuda:1")

        def data_ptr(self):
            return 99

    class Lib:
        def rans_get_status(self, word, stream):
            got.append((word.value, stream.value, now[0]))
            return rb.OK

    @contextlib.contextmanager
    def device(d):
        was, now[0] = now[0], str(d)
        yield
        now[0] = was

    stream = type("Stream", (), dict(cuda_stream=7))
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: stream)
    monkeypatch.setattr(rb._lib, "lib", lambda: Lib())
    assert rb.rans_get_status(Word()) == rb.OK and now == ["cuda:0"]
    assert got == [(99, 7, "cuda:1")]


def test_pointers_off_their_types_boundaries_are_refused(lib):
    """Half an element (or, for arrays of rows, a byte) beside where one lies."""
    lg, one = logits(), rb.Chunking.contig(2)
    x = ctypes.byref(lg)

    def off(call, good, at, by):
        for k in at:
            args = list(good)
            args[k] += by
            assert call(*args) == rb.ERR_ARG, (call.__name__, k)

    off(lib.rans_token_intervals, [x, None, A(1), A(2), A(3), A(4), None], (2, 3, 4), 2)
    good = [x, None, A(1), 64, A(2), 8, A(3), A(4), A(5), A(6), A(7), None]
    off(lib.rans_decode_tokens, good, (4, 7, 8), 4)
    off(lib.rans_decode_tokens, good, (6, 9), 2)
    off(lib.rans_token_states, [A(1), 64, A(2), 2, A(3), A(4), None], (2, 4), 4)
    off(lib.rans_token_states_finish, [A(1), 2, A(2), A(3), None], (0, 2), 4)
    off(lib.rans_distill_forward, [x, A(1), A(2), 5, 1.0, 1, A(3), A(4), A(5), None], (1, 2, 6), 2)
    off(lib.rans_distill_backward, [x, A(1), A(2), 5, 1.0, A(3), A(4), A(5), 100, None],
        (1, 2, 6, 7), 2)
    off(lib.rans_distill, [x, A(1), A(2), 5, 1.0, 1, A(3), A(4), A(5), 100, A(6), None],
        (1, 2, 6, 7, 8), 2)
    off(lib.rans_encode_intervals, [A(1), A(2), 10, ctypes.byref(one.c), A(3), 4096, A(4), A(5),
                                    1 << 20, None], (0, 1, 6), 2)
    c = rb.rans_chunking()
    c.kind, c.interleave, c.n_streams, c.index_block = rb._lib.CHUNK_EXPLICIT, 1, 2, 1
    c.stream_starts = A(6) + 4
    assert lib.rans_encode_intervals(A(1), A(2), 10, ctypes.byref(c), A(3), 4096, A(4), A(5),
                                     1 << 20, None) == rb.ERR_ARG
    whole = dict(history=A(8), history_begin=A(9), history_end=A(10), history_len=5,
                 bias_ids=A(11), bias_values=A(12), bias_begin=A(13), bias_end=A(14), bias_len=5,
                 mask=A(15), mask_stride=4, params=A(16))
    for k, v in whole.items():
        if k not in ("history_len", "bias_len", "mask_stride"):
            by = 4 if k.endswith(("begin", "end")) else 2
            assert list(calls(lib, lg, adjust(**{**whole, k: v + by}))) == [rb.ERR_ARG] * 3, k


def test_distillations_whose_results_overlap_are_refused(lib):
    lg = logits(rows=4, vocab=100, stride=160)   # 640 bytes a row, 400 of them logits
    x, S = ctypes.byref(lg), rb.ERR_ARG

    def refused(call, good, changes):
        for k, v in changes:
            args = list(good)
            args[k] = v
            assert call(*args) == S, (call.__name__, k, v)

    # ids, logprobs (4 x 5 each), weights, losses, grad (stride 160)
    good = [x, A(1), A(2), 5, 1.0, 1, A(3), A(4), A(5), 160, A(6), None]
    refused(lib.rans_distill, good, [
        (7, A(1)), (7, A(1) + 76), (7, A(2) - 12), (7, A(3) + 4), (7, P), (7, P + 3 * 640 + 396),
        (7, A(5)), (7, A(5) + 640 + 396), (7, A(5) + 632), (8, A(1)), (8, A(2) + 76),
        (8, A(3) - 396), (8, A(4) + 12), (1, A(5) + 640), (2, A(5) + 3 * 640 + 100),
        (6, A(5) + 396)])
    # ids, logprobs, losses, stats (4 x 8)
    good = [x, A(1), A(2), 5, 1.0, 1, A(3), A(4), A(5), None]
    refused(lib.rans_distill_forward, good, [
        (6, A(1) + 76), (6, A(2)), (6, A(4) + 124), (6, P + 640), (7, A(1) + 64), (7, A(2) - 112),
        (7, A(3)), (7, P + 2 * 640)])
    # ids, logprobs, stats, weights, grad
    good = [x, A(1), A(2), 5, 1.0, A(3), A(4), A(5), 160, None]
    refused(lib.rans_distill_backward, good, [
        (7, A(1)), (7, A(2) + 76), (7, A(3) + 124), (7, A(4) + 12), (1, A(5) + 396),
        (5, A(5) + 384)])
