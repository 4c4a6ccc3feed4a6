"""Beam search under a language model's logits (include/rans_b200.h, "beam
search"): the best continuations of every text, a search's bookkeeping, and
states that follow their beams.

Argument checks and marshalling only, as in ``tokens``: every step of a search
runs in the library's kernels (making a BeamSearch and reading its results are
torch operations).  Calls run on the tensors' device, on ``stream`` or that
device's current stream; nothing here takes part in autograd.
"""
import ctypes
import functools
import math
import struct

import torch

from . import _lib as L
from . import tokens as T
from .mxfp4 import _word

MAX_BEAMS = 64
MAX_CONTINUATIONS = 128
MAX_STATES = 4096
_pack_address = struct.Struct("@P").pack
_pack_layout = struct.Struct("@qqqii").pack
_pack_beams = struct.Struct("@qiiPiifiPPPPPPPPPPP").pack
assert struct.calcsize("@Pqqqii") == ctypes.sizeof(L.rans_state)
assert struct.calcsize("@P") + struct.calcsize("@qqqii") == struct.calcsize("@Pqqqii")
assert struct.calcsize("@qiiPiifiPPPPPPPPPPP") == ctypes.sizeof(L.rans_beams)


# ---------------------------------------------------------- C entry points --
def rans_beam_workspace_bytes(dtype, rows, vocab, count):
    """For logits of a torch dtype, on the current device."""
    return L.lib().rans_beam_workspace_bytes(T._LOGITS_CODE[dtype], rows, vocab, count)


def rans_beam_select(logits, adjust, scores, beams, count, scores_out, tokens, parents, workspace,
                     status, stream=None):
    rows = T._rows(logits)
    with T._place(rows[0], stream):
        result = _select(rows, logits, adjust, scores, beams, count, scores_out, tokens, parents,
                         workspace, status)
    T._written(scores_out, tokens, parents, workspace)
    return result


def _shape(rows, beams, count):
    """Texts of so many rows."""
    if not 1 <= beams <= MAX_BEAMS or rows[1] % beams != 0:
        raise ValueError("beams: 1 to %d, dividing the %d rows" % (MAX_BEAMS, rows[1]))
    if not 1 <= count <= MAX_CONTINUATIONS:
        raise ValueError("count: 1 to %d" % MAX_CONTINUATIONS)
    return rows[1] // beams


def _select(rows, logits, adjust, scores, beams, count, scores_out, tokens, parents, workspace,
            status):
    dev, n = rows[:2]
    t = _shape(rows, beams, count)
    if not isinstance(scores, torch.Tensor) or scores.numel() != n:
        raise ValueError("scores: a float32 tensor of %d elements" % n)
    c = T._tensor(scores, torch.float32, None, dev, "scores")
    s = T._tensor(scores_out, torch.float32, (t, count), dev, "scores_out")
    k = T._tensor(tokens, torch.int32, (t, count), dev, "tokens")
    p = T._tensor(parents, torch.int32, (t, count), dev, "parents")
    w = T._tensor(workspace, torch.uint8, None, dev, "workspace")
    return L.lib().rans_beam_select(T._packed(logits, rows), T._ref(adjust, rows), c, beams, count,
                                    s, k, p, w, workspace.numel(), _word(status, dev),
                                    T._raw_stream(dev))


def rans_beam_advance(scores, tokens, parents, search, stream=None):
    """search: a BeamSearch."""
    with T._place(search.dev, stream):
        result = _advance(scores, tokens, parents, search)
    T._written(*search._parts)
    return result


def _advance(scores, tokens, parents, search):
    shape = (search.texts, scores.shape[-1])
    s = T._tensor(scores, torch.float32, shape, search.dev, "scores")
    k = T._tensor(tokens, torch.int32, shape, search.dev, "tokens")
    p = T._tensor(parents, torch.int32, shape, search.dev, "parents")
    return L.lib().rans_beam_advance(s, k, p, shape[1], search._c, T._raw_stream(search.dev))


def rans_reorder_states(states, parents, lengths, axis, status, stream=None):
    dev = T._device(parents, "parents")
    with T._place(dev, stream):
        result = _reorder(dev, states, parents, lengths, axis, status)
    T._written(*states)
    return result


def _state(x, rows, axis, dev, known):
    """A rans_state's bytes.  known: of this call's shapes so far, all but the address."""
    if not isinstance(x, torch.Tensor) or x.get_device() != dev:
        raise ValueError("states: CUDA tensors on cuda:%d" % dev)
    key = (x.shape, x.stride(), x.element_size(), axis)
    rest = known.get(key)
    if rest is None:
        rest = known[key] = _layout(x, rows, axis)
    return _pack_address(x.data_ptr()) + rest


def _layout(x, rows, axis):
    shape, e = x.shape, x.element_size()
    if x.dim() < 1 or shape[0] != rows:
        raise ValueError("states: tensors of %d rows" % rows)
    if not x.is_contiguous() and rows > 0 and not x[0].is_contiguous():
        raise ValueError("states: each row must be contiguous")
    step, row = x.stride(0), math.prod(shape[1:])
    if rows > 1 and step < row:
        raise ValueError("states: rows must not overlap")
    if axis is None:  # one piece, in positions of a size that the library counts
        return _pack_layout(step * e, row * e, 1, 1, row * e) if row * e < 1 << 31 else \
            _pack_layout(step * e, row * e, row, 1, e)
    if not 1 <= axis < len(shape):
        raise ValueError("axis: 1 to %d for a state of shape %s" % (len(shape) - 1, tuple(shape)))
    outer, inner = math.prod(shape[1:axis]), math.prod(shape[axis + 1:])
    if outer >= 1 << 31 or inner * e >= 1 << 31:
        raise ValueError("states: a shape of %s is too large around axis %d" % (
            tuple(shape), axis))
    return _pack_layout(step * e, shape[axis] * inner * e, shape[axis], outer, inner * e)


def _reorder(dev, states, parents, lengths, axis, status):
    return L.lib().rans_reorder_states(*_moves(dev, states, parents, lengths, axis, status),
                                       T._raw_stream(dev))


def _moves(dev, states, parents, lengths, axis, status):
    """The arguments of a move of states, up to the stream."""
    if parents.dim() != 2 or not 1 <= parents.shape[1] <= MAX_BEAMS:
        raise ValueError("parents: int32 [texts, beams], 1 to %d beams" % MAX_BEAMS)
    t, k = parents.shape
    p = T._tensor(parents, torch.int32, None, dev, "parents")
    n = None if lengths is None else T._tensor(lengths, torch.int32, (t,), dev, "lengths")
    if len(states) > MAX_STATES:
        raise ValueError("states: %d at most" % MAX_STATES)
    if axis is None and lengths is not None:
        raise ValueError("lengths: say which axis of the states they count")
    one = axis is None or isinstance(axis, int)
    if not one and len(axis) != len(states):
        raise ValueError("axis: %d for %d states" % (len(axis), len(states)))
    known = {}
    packed = b"".join([_state(x, t * k, axis if one else axis[i], dev, known)
                       for i, x in enumerate(states)])
    return packed, len(states), t, k, p, n, _word(status, dev)


# ----------------------------------------------------------------- helpers --
def beam_select(logits, scores, beams, count=None, adjust=None, status=None, stream=None):
    """The `count` best continuations (default 2 * beams) of every text: (scores
    float32, tokens int32, parents int32), each [texts, count], best first.

    logits: a row per beam, `beams` rows a text; scores: float32, each beam's log
    probability so far (-inf: a dead beam).  A continuation's total is its beam's
    score and the log probability of its token under the adjusted logits.
    Totals are compared in 64 bits, ties go to the lower beam, within a beam to the
    larger logit, then to the lower token; where there are too few, the rest is -inf,
    -1, -1.
    """
    rows = T._rows(logits)
    if count is None:
        count = 2 * beams
    t = _shape(rows, beams, count)
    dev, n = rows[:2]
    if not isinstance(scores, torch.Tensor) or scores.numel() != n:
        raise ValueError("scores: a float32 tensor of %d elements" % n)
    c = T._tensor(scores, torch.float32, None, dev, "scores")
    with T._place(dev, stream):
        best = scores.new_empty((t, count))
        tokens = scores.new_empty((t, count), dtype=torch.int32)
        parents = scores.new_empty((t, count), dtype=torch.int32)
        size = _workspace(rows[3], n, rows[2], count, dev)
        ws = scores.new_empty(size, dtype=torch.uint8)
        word = None if status is None else T._status(status, dev).data_ptr()
        L.check(L.lib().rans_beam_select(
            T._packed(logits, rows), T._ref(adjust, rows), c, beams, count, best.data_ptr(),
            tokens.data_ptr(), parents.data_ptr(), ws.data_ptr(), size, word,
            T._raw_stream(dev)), "beam_select")
    return best, tokens, parents


@functools.lru_cache(maxsize=256)
def _workspace(code, rows, vocab, count, dev):
    """Bytes for sizes on a device (the current one)."""
    return L.lib().rans_beam_workspace_bytes(code, rows, vocab, count)


def rans_reorder_states_check(states, parents, lengths, axis, status):
    return L.lib().rans_reorder_states_check(
        *_moves(T._device(parents, "parents"), states, parents, lengths, axis, status))


def reorder_states(states, parents, lengths=None, axis=None, status=None, stream=None):
    """A model's states following their beams, in place: row b of text t becomes
    what row parents[t, b] was.  Returns the states.

    states: a tensor or a list, [texts * beams, ...] with contiguous rows.
    parents: int32 [texts, beams]; -1 leaves a row as it is.
    lengths: int32 [texts], how many positions of `axis` (a number, or one for
        each state) are moved; what lies behind is left as it was.
    """
    dev = T._device(parents, "parents")
    every = [states] if isinstance(states, torch.Tensor) else states
    with T._place(dev, stream):
        L.check(_reorder(dev, every, parents, lengths, axis, status), "reorder_states")
    T._written(*every)
    return states


class BeamSearch:
    """A search over texts of `beams` beams each, without reading anything back.

    Every step takes a row of logits per beam (text after text) and yields the
    beams' tokens.  A text's results are the continuations that ended; their
    scores are log probabilities divided by length^length_penalty.  The beams of a
    text keep their slots where they can: `parents` says which slot each comes
    from, and moved slots copy from ones that stay.

    capacity: most tokens of a text.  ends: ids that end a text (up to 64).  early: a
    text is over as soon as it has `beams` results; otherwise when none can be
    improved.  pad: the token of dead beams.

    scores (float32 [texts * beams]), tokens (int32, the same), parents (int32
    [texts, beams]), lengths and over (int32 [texts]) are the search's state
    on the device, updated in place; `window` is the beams' tokens as
    LogitAdjust takes a history.  Steps may be captured into a graph.  They may run on
    another stream than the one on which the search was made (they wait for that; captured
    steps do not); steps on several streams, and results, are for the program to order.
    """

    def __init__(self, texts, beams, capacity, ends=(), length_penalty=0.0, early=False, pad=0,
                 device="cuda"):
        if not 1 <= beams <= MAX_BEAMS:
            raise ValueError("beams: 1 to %d" % MAX_BEAMS)
        if texts < 0 or not 1 <= capacity < 1 << 31:
            raise ValueError("texts: not negative, capacity: at least 1")
        ends = [int(e) for e in ends]
        if len(ends) > 64 or any(not 0 <= e < 1 << 31 for e in ends):
            raise ValueError("ends: up to 64 token ids")
        if not -(1 << 31) <= pad < 1 << 31:
            raise ValueError("pad: an int32")
        self.texts, self.beams, self.capacity = texts, beams, capacity
        self.length_penalty = T._in_float32(length_penalty, T._finite, "length_penalty")
        n = texts * beams
        dev = torch.device(device)

        def zeros(*shape, dtype=torch.int32):
            return torch.zeros(shape, dtype=dtype, device=dev)

        self.scores = torch.full((texts, beams), -math.inf, dtype=torch.float32, device=dev)
        self.scores[:, 0] = 0.0
        self.scores = self.scores.view(-1)
        self.dev = T._device(self.scores, "device")
        self.tokens = torch.full((n,), pad, dtype=torch.int32, device=dev)
        self.parents = torch.arange(beams, dtype=torch.int32, device=dev).repeat(texts, 1)
        self.lengths, self.over = zeros(texts), zeros(texts)
        self._history = zeros(texts, beams, capacity)
        self._begin = torch.arange(n, dtype=torch.int64, device=dev) * capacity
        self._end = self._begin.clone()
        self._ends = torch.tensor(ends, dtype=torch.int32, device=dev)
        self._done_scores = torch.full((texts, beams), -math.inf, device=dev)
        self._done_lengths, self._done_counts = zeros(texts, beams), zeros(texts)
        self._done_tokens = zeros(texts, beams, capacity)
        self._parts = (self.scores, self.tokens, self.parents, self._history, self._end,
                       self.lengths, self.over, self._done_scores, self._done_lengths,
                       self._done_tokens, self._done_counts)
        self._made = T._MadeOn(self._begin, self.dev, self._ends, *self._parts)
        self._c = _pack_beams(texts, beams, capacity, self._ends.data_ptr(), len(ends), pad,
                              self.length_penalty, int(bool(early)),
                              *[x.data_ptr() for x in self._parts])

    @property
    def window(self):
        """(tokens, begin, end): every beam's tokens so far, for LogitAdjust."""
        return self._history.view(-1), self._begin, self._end

    def step(self, logits, adjust=None, states=(), lengths=None, axis=None, status=None,
             stream=None):
        """The next tokens (int32 [texts * beams], the search's own tensor).
        states, lengths, axis: a model's states to reorder along (see
        reorder_states).  Steps past the capacity change nothing."""
        rows = T._rows(logits)
        if rows[0] != self.dev or rows[1] != self.texts * self.beams:
            raise ValueError("logits: %d rows on cuda:%d" % (self.texts * self.beams, self.dev))
        # enough that `beams` go on even if every beam ends in every way (as far as
        # a selection goes: beyond it beams may die out)
        count = min(self.beams * max(2, 1 + self._ends.numel()), MAX_CONTINUATIONS)
        moves = None
        if len(states) > 0:
            # (before anything has run: a search is not to be a step ahead of its states)
            every = [states] if isinstance(states, torch.Tensor) else states
            moves = _moves(self.dev, every, self.parents, lengths, axis, status)
            L.check(L.lib().rans_reorder_states_check(*moves), "reorder_states")
        with T._place(self.dev, stream):
            self._made.use()
            best = beam_select(logits, self.scores, self.beams, count, adjust, status)
            L.check(_advance(*best, self), "beam_advance")
            T._written(*self._parts)
            if moves is not None:
                L.check(L.lib().rans_reorder_states(*moves, T._raw_stream(self.dev)),
                        "reorder_states")
                T._written(*every)
        return self.tokens

    def results(self, n=1):
        """(tokens int32 [texts, n, capacity], lengths int32 [texts, n], scores
        float32 [texts, n]): the best of what has ended and of the beams still under
        way, best first.  Missing ones have length 0 and score -inf."""
        if not 1 <= n <= self.beams:
            raise ValueError("n: 1 to %d" % self.beams)
        length = self.lengths[:, None].expand(-1, self.beams)
        going = self.scores.view(self.texts, self.beams)
        if self.length_penalty != 0.0:
            going = going / length.clamp(min=1).float() ** self.length_penalty
        scores = torch.cat([self._done_scores, going], 1)
        lengths = torch.cat([self._done_lengths, length], 1)
        tokens = torch.cat([self._done_tokens, self._history], 1)
        order = scores.sort(dim=1, descending=True, stable=True).indices[:, :n]
        scores = scores.gather(1, order)
        lengths = lengths.gather(1, order).masked_fill(scores == -math.inf, 0)
        return tokens.gather(1, order[:, :, None].expand(-1, -1, self.capacity)), lengths, scores
