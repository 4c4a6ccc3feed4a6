"""Tokens under a language model's logits (include/rans_b200.h, "tokens under
a model's logits"): logit adjustment, intervals of tokens, streams of
intervals, decoding steps and the distillation loss.

Argument checks and marshalling only, as in ``_lib``; every step of a call runs
in the library's kernels (LogitAdjust's copy of per-row numbers and pack_mask,
which prepare a call's arguments, are torch operations).  Logits are CUDA tensors [rows, vocab] of float32, float16
or bfloat16 whose rows are contiguous (a column slice of a wider buffer is
fine).  Calls run on the tensors' device, on ``stream`` or that device's
current stream.  ``status`` is a CUDA tensor from ``new_status()``; pass one to
learn of device errors (``check(rans_get_status(status))``).
"""
import contextlib
import ctypes
import struct

import torch

from . import _lib as L

_LOGITS_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
MAX_VOCAB = (1 << 19) - 8
MAX_TOP = 4096
TOKEN_PRECISION = 24

# These calls are made once per decoded token, where the host's time counts: a
# tensor's facts are asked once each, devices are compared by index, and
# the structs are packed rather than built field by field.
_pack_logits = struct.Struct("@Piiqq").pack
_pack_adjust = struct.Struct("@ffffPPPPqPPPPqPq").pack
_float4 = struct.Struct("@ffff")
_INF = float("inf")
assert struct.calcsize("@Piiqq") == ctypes.sizeof(L.rans_logits)
assert struct.calcsize("@ffffPPPPqPPPPqPq") == ctypes.sizeof(L.rans_adjust)
_no_context = contextlib.nullcontext()


def _place(dev, stream):
    """Context in which to allocate and launch: the tensors' device and the
    caller's stream, where either is not the current one."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("stream on %s, tensors on cuda:%d" % (stream.device, dev))
        return torch.cuda.stream(stream)
    if dev != torch._C._cuda_getDevice():
        return torch.cuda.device(dev)
    return _no_context


def _raw_stream(dev):
    """The device's current stream, as an address."""
    return torch._C._cuda_getCurrentRawStream(dev)


class _MadeOn:
    """A tensor (or more) of the library's own that was computed on the stream
    current at the time, for calls on other streams: they wait for it, and its memory
    for them.  Not where either is captured: a capture may not wait for work
    outside of it, nor the reverse.  There the program orders its streams, and
    its replays, as it does for its own tensors."""

    def __init__(self, x, dev, *more):
        self.tensors, self.dev = (x, *more), dev
        self.stream = torch.cuda.current_stream(dev)
        self.captured = torch.cuda.is_current_stream_capturing()
        if not self.captured:
            self.done = torch.cuda.Event()
            self.done.record(self.stream)

    def use(self):
        if _raw_stream(self.dev) == self.stream.cuda_stream:
            return
        if self.captured or torch.cuda.is_current_stream_capturing():
            return
        here = torch.cuda.current_stream(self.dev)
        here.wait_event(self.done)
        for x in self.tensors:
            x.record_stream(here)


def _rows(x, what="logits"):
    """(device index, rows, vocab, dtype code, row stride) of rows of logits."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 2:
        raise ValueError("%s: a CUDA tensor [rows, vocab]" % what)
    code = _LOGITS_CODE.get(x.dtype)
    if code is None:
        raise ValueError("%s: float32, float16 or bfloat16, not %s" % (what, x.dtype))
    n, v = x.shape
    if not 1 <= v <= MAX_VOCAB:
        raise ValueError("%s: a vocabulary of 1 to %d tokens" % (what, MAX_VOCAB))
    step, one = x.stride()
    if (v > 1 and one != 1) or (n > 1 and step < v):
        raise ValueError("%s: rows must be contiguous and must not overlap" % what)
    return x.get_device(), n, v, code, max(step, v)


def _packed(x, rows):
    return _pack_logits(x.data_ptr(), rows[3], rows[2], rows[1], rows[4])


def _device(x, what):
    """The index of a CUDA tensor's device.  (Host tensors share -1: without this
    they would all be "on one device".)"""
    dev = x.get_device() if isinstance(x, torch.Tensor) else -1
    if dev < 0:
        raise ValueError("%s: a CUDA tensor" % what)
    return dev


def _tensor(x, dtype, shape, dev, what):
    """The address of a contiguous CUDA tensor of this type and shape on device
    `dev` (an index)."""
    if not isinstance(x, torch.Tensor) or x.dtype is not dtype or x.get_device() != dev or \
            not x.is_contiguous() or (shape is not None and x.shape != shape):
        raise ValueError("%s: a contiguous %s tensor%s on cuda:%d" % (
            what, dtype, "" if shape is None else " of shape %s" % (tuple(shape),), dev))
    return x.data_ptr()


def _written(*tensors):
    """Tells autograd that a call wrote to the caller's tensors, as torch's own
    in-place operations do: a backward pass that had saved one of them then
    raises, where it would use what stands there now."""
    torch.autograd.graph.increment_version(tensors)


def new_status(device="cuda"):
    """A status word for the calls below (the first device error stays in it
    until rans_get_status reads it)."""
    return torch.zeros(32, dtype=torch.int64, device=device)


def _status(status, dev):
    """The call's status word.  Like every tensor whose address goes to the
    library, it has to be held by a name until the call returns: the calls
    release the interpreter's lock, and memory that another thread was given
    meanwhile would be written to."""
    if status is None:
        return new_status(dev)
    if not isinstance(status, torch.Tensor) or status.get_device() != dev or \
            not status.is_contiguous() or status.numel() * status.element_size() < 256:
        raise ValueError("status: from new_status() on cuda:%d" % dev)
    return status


# ---------------------------------------------------------- C entry points --
def _ref(adjust, rows):
    return None if adjust is None else adjust.bind(rows)


def rans_adjust_logits(logits, adjust, out, stream=None):
    rows = _rows(logits)
    with _place(rows[0], stream):
        result = _adjust(rows, logits, adjust, out)
    _written(out)
    return result


def _adjust(rows, logits, adjust, out):
    o = _rows(out, "out")
    if o[:3] != rows[:3]:
        raise ValueError("out: a tensor of the logits' shape on their device")
    return L.lib().rans_adjust_logits(_packed(logits, rows), _ref(adjust, rows),
                                      out.data_ptr(), o[3], o[4], _raw_stream(rows[0]))


def rans_token_intervals(logits, adjust, tokens, starts, freqs, status, stream=None):
    rows = _rows(logits)
    with _place(rows[0], stream):
        result = _intervals(rows, logits, adjust, tokens, starts, freqs, status)
    _written(starts, freqs)
    return result


def _intervals(rows, logits, adjust, tokens, starts, freqs, status):
    dev, n = rows[:2]
    t = _tensor(tokens, torch.int32, (n,), dev, "tokens")
    s = _tensor(starts, torch.int32, (n,), dev, "starts")
    f = _tensor(freqs, torch.int32, (n,), dev, "freqs")
    status = _status(status, dev)
    return L.lib().rans_token_intervals(_packed(logits, rows), _ref(adjust, rows), t, s, f,
                                        status.data_ptr(), _raw_stream(dev))


def rans_encode_intervals(starts, freqs, n, chunking, out, stream_offsets, workspace,
                          stream=None):
    dev = _device(starts, "starts")
    S = L.rans_num_streams(chunking, n)
    with _place(dev, stream):
        result = _encode(dev, starts, freqs, n, S, chunking, out, stream_offsets, workspace)
    _written(out, stream_offsets, workspace)
    return result


def _encode(dev, starts, freqs, n, S, chunking, out, stream_offsets, workspace):
    # (the chunking's own tensor: explicit stream starts)
    if chunking._keep is not None and chunking._keep.get_device() != dev:
        raise ValueError("chunking on %s, starts on cuda:%d" % (chunking._keep.device, dev))
    s = _tensor(starts, torch.int32, (n,), dev, "starts")
    f = _tensor(freqs, torch.int32, (n,), dev, "freqs")
    o = _tensor(out, torch.uint8, None, dev, "out")
    w = _tensor(workspace, torch.uint8, None, dev, "workspace")
    offs = _tensor(stream_offsets, torch.int64, (S + 1,) if S >= 0 else None, dev,
                   "stream_offsets")
    return L.lib().rans_encode_intervals(s, f, n, ctypes.byref(chunking.c), o, out.numel(),
                                         offs, w, workspace.numel(), _raw_stream(dev))


def _streams(data, stream_offsets):
    """(device index, S, the two addresses)."""
    dev = _device(data, "data")
    d = _tensor(data, torch.uint8, None, dev, "data")
    o = _tensor(stream_offsets, torch.int64, None, dev, "stream_offsets")
    S = stream_offsets.numel() - 1
    if S < 0:
        raise ValueError("stream_offsets: S + 1 offsets")
    return dev, S, d, o


def rans_token_states(data, stream_offsets, states, status, stream=None):
    dev, S, d, o = _streams(data, stream_offsets)
    s = _tensor(states, torch.int64, (S, 2), dev, "states")
    with _place(dev, stream):
        status = _status(status, dev)
        result = L.lib().rans_token_states(d, data.numel(), o, S, s, status.data_ptr(),
                                           _raw_stream(dev))
    _written(states)
    return result


def rans_decode_tokens(logits, adjust, data, stream_offsets, stream_ids, states_in, states_out,
                       tokens, status, stream=None):
    rows = _rows(logits)
    with _place(rows[0], stream):
        result = _decode(rows, logits, adjust, data, stream_offsets, stream_ids, states_in,
                         states_out, tokens, status)
    _written(states_out, tokens)
    return result


def _decode(rows, logits, adjust, data, stream_offsets, stream_ids, states_in, states_out,
            tokens, status):
    dev, S, d, o = _streams(data, stream_offsets)
    if dev != rows[0]:
        raise ValueError("data on cuda:%d, logits on cuda:%d" % (dev, rows[0]))
    n = rows[1]
    ids = None if stream_ids is None else _tensor(stream_ids, torch.int32, (n,), dev,
                                                  "stream_ids")
    a = _tensor(states_in, torch.int64, (S, 2), dev, "states")
    b = _tensor(states_out, torch.int64, (S, 2), dev, "states_out")
    t = _tensor(tokens, torch.int32, (n,), dev, "tokens")
    status = _status(status, dev)
    return L.lib().rans_decode_tokens(
        _packed(logits, rows), _ref(adjust, rows), d, data.numel(), o, S, ids, a, b, t,
        status.data_ptr(), _raw_stream(dev))


def rans_token_states_finish(stream_offsets, states, status, stream=None):
    dev = _device(states, "states")
    o = _tensor(stream_offsets, torch.int64, None, dev, "stream_offsets")
    S = stream_offsets.numel() - 1
    s = _tensor(states, torch.int64, (S, 2), dev, "states")
    with _place(dev, stream):
        status = _status(status, dev)
        return L.lib().rans_token_states_finish(o, S, s, status.data_ptr(), _raw_stream(dev))


def _teacher(logits, ids, logprobs, rows=None):
    """(rows of the logits, K, the teacher's two addresses)."""
    rows = rows or _rows(logits)
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or not 1 <= ids.shape[1] <= MAX_TOP:
        raise ValueError("ids: a tensor [rows, K], K from 1 to %d" % MAX_TOP)
    K = ids.shape[1]
    i = _tensor(ids, torch.int32, (rows[1], K), rows[0], "ids")
    return rows, K, i, _tensor(logprobs, torch.float32, (rows[1], K), rows[0], "logprobs")


def rans_distill_forward(logits, ids, logprobs, inv_temperature, tail, losses, stats, status,
                         stream=None):
    rows, K, i, lp = _teacher(logits, ids, logprobs)
    dev, n = rows[:2]
    o = _tensor(losses, torch.float32, (n,), dev, "losses")
    s = _tensor(stats, torch.float32, (n, 8), dev, "stats")
    with _place(dev, stream):
        status = _status(status, dev)
        result = L.lib().rans_distill_forward(
            _packed(logits, rows), i, lp, K, inv_temperature, int(tail), o, s,
            status.data_ptr(), _raw_stream(dev))
    _written(losses, stats)
    return result


def _grad_of(rows, grad):
    """(address, row stride) of a gradient of these rows."""
    o = _rows(grad, "grad")
    if o[:4] != rows[:4]:
        raise ValueError("grad: a tensor of the logits' shape and type on their device")
    return grad.data_ptr(), o[4]


def rans_distill_backward(logits, ids, logprobs, inv_temperature, stats, grad_losses, grad,
                          stream=None):
    rows, K, i, lp = _teacher(logits, ids, logprobs)
    dev, n = rows[:2]
    s = _tensor(stats, torch.float32, (n, 8), dev, "stats")
    w = _tensor(grad_losses, torch.float32, (n,), dev, "grad_losses")
    g, step = _grad_of(rows, grad)
    with _place(dev, stream):
        result = L.lib().rans_distill_backward(_packed(logits, rows), i, lp, K, inv_temperature,
                                               s, w, g, step, _raw_stream(dev))
    _written(grad)
    return result


def rans_distill(logits, ids, logprobs, inv_temperature, tail, grad_losses, losses, grad, status,
                 stream=None):
    rows = _rows(logits)
    with _place(rows[0], stream):
        result = _both(rows, logits, ids, logprobs, inv_temperature, tail, grad_losses, losses,
                       grad, status)
    _written(losses, grad)
    return result


def _both(rows, logits, ids, logprobs, inv_temperature, tail, grad_losses, losses, grad, status):
    _, K, i, lp = _teacher(logits, ids, logprobs, rows)
    dev, n = rows[:2]
    w = _tensor(grad_losses, torch.float32, (n,), dev, "weights")
    o = _tensor(losses, torch.float32, (n,), dev, "losses")
    g, step = _grad_of(rows, grad)
    status = _status(status, dev)
    return L.lib().rans_distill(_packed(logits, rows), i, lp, K, inv_temperature, int(tail),
                                w, o, g, step, status.data_ptr(), _raw_stream(dev))


# ----------------------------------------------------------------- helpers --
def _positive(x, what):
    x = float(x)
    if not 0.0 < x < float("inf"):
        raise ValueError("%s must be positive and finite" % what)
    return x


def _finite(x, what):
    x = float(x)
    if x - x != 0.0:
        raise ValueError("%s must be finite" % what)
    return x


def _in_float32(x, check, what):
    """A number as float32 has it, checked there (where 1e-50 is not positive
    and 1e39 not finite)."""
    return check(ctypes.c_float(float(x)).value, what)


def _inverse(temperature):
    """1 / T of a number, as the per-row form has it: T rounded to float32 and
    its reciprocal rounded once more.  (A double reciprocal of the number itself
    is another float32 for 0.85 or 1.1, and other intervals.)"""
    t = _in_float32(temperature, _positive, "temperature")
    return _in_float32(1.0 / t, _positive, "1 / temperature")


def pack_mask(allowed):
    """Words of a bool tensor [rows, vocab] (or [vocab]) of allowed tokens, as
    LogitAdjust takes them: bit v & 31 of word v >> 5.  For rules that are packed
    once: in torch operations, with 16 bytes a token of temporary memory.  A
    grammar that changes with every token should keep its words itself."""
    flat = allowed if allowed.dim() == 2 else allowed[None]
    n, v = flat.shape
    bits = torch.nn.functional.pad(flat, (0, -v % 32)).view(n, -1, 32).to(torch.int64)
    words = (bits << torch.arange(32, device=flat.device)).sum(2)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    return words if allowed.dim() == 2 else words[0]


class LogitAdjust:
    """What is done to rows of logits before they are used.

    temperature, repetition, frequency, presence: numbers for all rows, or
        float32 CUDA tensors [rows] (any of them).  A number is rounded to
        float32, and the logits are multiplied by the temperature's reciprocal,
        rounded to float32: a number and rows that hold it code alike.
    history: (tokens int32, begin int64 [rows], end int64 [rows]): row r's
        history is tokens[begin[r]:end[r]].
    bias: (ids int32, values float32, begin int64 [rows], end int64 [rows]);
        a token's last entry in its row's window counts.
    mask: int32 [rows, words] or [words] (for all rows) with 1 bits where
        tokens are allowed; see pack_mask.

    The tensors of history, bias and mask are read by each call, so a program
    may keep one LogitAdjust and update them in place between steps (per-row
    numbers are copied when it is made, on the stream current then; calls on
    other streams wait for the copy, captured calls not.  A captured call reads
    that copy at every replay: keep the LogitAdjust as long as the graph).
    """

    def __init__(self, temperature=1.0, repetition=1.0, frequency=0.0, presence=0.0,
                 history=None, bias=None, mask=None):
        self._n, self._words, self._dev = None, 0, None
        self._keep = (history, bias, mask)
        self._made = None
        params = 0
        scalars = (1.0, 0.0, 0.0, 1.0)
        tensor = torch.Tensor
        if isinstance(temperature, tensor) or isinstance(repetition, tensor) or \
                isinstance(frequency, tensor) or isinstance(presence, tensor):
            params = self._per_row((repetition, frequency, presence, temperature))
        else:
            # rounded to float32 at once; one by one, to say which, if one is bad
            r, f, p, t = _float4.unpack(_float4.pack(repetition, frequency, presence, temperature))
            if 0.0 < r < _INF and f - f == 0.0 and p - p == 0.0 and 1e-38 < t < _INF:
                scalars = (r, f, p, 1.0 / t)
            else:
                scalars = (_in_float32(repetition, _positive, "repetition"),
                           _in_float32(frequency, _finite, "frequency"),
                           _in_float32(presence, _finite, "presence"), _inverse(temperature))
        hist = (0, 0, 0, 0)
        if history is not None:
            tokens, begin, end = history
            n = begin.shape
            dev = self._on(begin, n[0])
            hist = (_tensor(tokens, torch.int32, tokens.shape, dev, "history tokens"),
                    _tensor(begin, torch.int64, n, dev, "history begin"),
                    _tensor(end, torch.int64, n, dev, "history end"), tokens.numel())
            if hist[3] == 0:
                hist = (0, 0, 0, 0)
        extra = (0, 0, 0, 0, 0)
        if bias is not None:
            ids, values, begin, end = bias
            k, n = ids.shape, begin.shape
            dev = self._on(begin, n[0])
            extra = (_tensor(ids, torch.int32, k, dev, "bias ids"),
                     _tensor(values, torch.float32, k, dev, "bias values"),
                     _tensor(begin, torch.int64, n, dev, "bias begin"),
                     _tensor(end, torch.int64, n, dev, "bias end"), ids.numel())
            if extra[4] == 0:
                extra = (0, 0, 0, 0, 0)
        allowed = (0, 0)
        if mask is not None:
            if mask.dtype is not torch.int32 or mask.dim() not in (1, 2) or \
                    (mask.shape[-1] > 1 and mask.stride(-1) != 1):
                raise ValueError("mask: int32 words [rows, words] or [words], from pack_mask")
            self._words = mask.shape[-1]
            if self._words < 1:
                raise ValueError("mask: no words")
            if mask.dim() == 2:
                n, step = mask.shape[0], mask.stride(0)
                if n > 1 and step < self._words:
                    raise ValueError("mask: rows must not overlap")
                self._on(mask, n)
                allowed = (mask.data_ptr(), max(step, self._words))
            else:
                self._on(mask, self._n)
                allowed = (mask.data_ptr(), 0)
        self._c = _pack_adjust(*scalars, params, *hist, *extra, *allowed)

    def _per_row(self, parts):
        """Address of the parameters [rows, 4], numbers checked and widened to
        all rows."""
        one = [x for x in parts if isinstance(x, torch.Tensor)][0]
        dev, n = self._on(one, one.numel()), one.numel()
        cols = []
        for x, check, what in zip(parts, (_positive, _finite, _finite, _positive),
                                  ("repetition", "frequency", "presence", "temperature")):
            if isinstance(x, torch.Tensor):
                _tensor(x, torch.float32, (n,), dev, "per-row " + what)
            else:
                if what == "temperature":
                    _inverse(x)  # (it has to have one)
                x = torch.full((n,), _in_float32(x, check, what), dtype=torch.float32,
                               device=one.device)
            cols.append(x)
        # (a float32's reciprocal in double, rounded to float32, is correctly rounded)
        cols[3] = cols[3].double().reciprocal().float()
        rows = torch.stack(cols, 1)
        self._keep += (rows,)
        with _place(dev, None):
            self._made = _MadeOn(rows, dev)
        return rows.data_ptr()

    def _on(self, x, n):
        """The device of a part for n rows, which all parts share."""
        dev = x.get_device()
        if dev < 0 or (self._dev is not None and self._dev != dev):
            raise ValueError("LogitAdjust takes CUDA tensors on one device")
        if self._n is not None and n is not None and self._n != n:
            raise ValueError("parts for %d and for %d rows" % (self._n, n))
        self._dev = dev
        if n is not None:
            self._n = n
        return dev

    def bind(self, rows):
        """The C struct's bytes, checked against the rows it is to be used on
        (as _rows has them), for a call on the device's current stream."""
        dev, n, v = rows[:3]
        if self._dev is not None and self._dev != dev:
            raise ValueError("LogitAdjust on cuda:%d, logits on cuda:%d" % (self._dev, dev))
        if self._n is not None and self._n != n:
            raise ValueError("LogitAdjust for %d rows, logits of %d" % (self._n, n))
        if self._words and self._words < (v + 31) // 32:
            raise ValueError("mask: %d words for %d tokens" % (self._words, v))
        if self._made is not None:
            self._made.use()
        return self._c


def adjust_logits(logits, adjust, out=None, dtype=None, stream=None):
    """Adjusted logits (penalties, biases, temperature, mask) for a sampler, in
    the logits' type or `dtype`; out may be the logits themselves.  No gradient
    flows through the result, whether the logits require one or not."""
    rows = _rows(logits)
    given = out is not None
    with _place(rows[0], stream):
        if not given:
            out = logits.new_empty(rows[1:3], dtype=dtype)
        L.check(_adjust(rows, logits, adjust, out), "adjust_logits")
    if given:
        _written(out)
    return out


def token_intervals(logits, tokens, adjust=None, starts=None, freqs=None, status=None,
                    stream=None):
    """(starts, freqs), int32 [rows]: each row's interval of its token at
    TOKEN_PRECISION bits.  Rows with token -1 are skipped: what stands in
    starts and freqs stays (nothing useful, where they are not given)."""
    rows = _rows(logits)
    given = starts is not None or freqs is not None
    with _place(rows[0], stream):
        if starts is None:
            starts = logits.new_empty(rows[1], dtype=torch.int32)
        if freqs is None:
            freqs = logits.new_empty(rows[1], dtype=torch.int32)
        L.check(_intervals(rows, logits, adjust, tokens, starts, freqs, status),
                "token_intervals")
    if given:
        _written(starts, freqs)
    return starts, freqs


def encode_intervals(starts, freqs, chunking, out=None, ws=None, stream=None):
    """(buffer, stream_offsets[S + 1], workspace): like encode_with_indexes;
    the coded bytes are buffer[:stream_offsets[-1]], device errors
    rans_get_status(workspace).  ws: a workspace to reuse."""
    dev = _device(starts, "starts")
    n = starts.numel()
    S = L.rans_num_streams(chunking, n)
    if S < 0:
        L.check(int(S), "num_streams")
    given = out is not None or ws is not None
    with _place(dev, stream):
        if ws is None:
            # torch's blocks are aligned to 512 bytes, as the workspace has to be to 256
            ws = starts.new_empty(L.rans_encode_workspace_bytes(chunking, n), dtype=torch.uint8)
        if out is None:
            out = starts.new_empty(L.rans_max_compressed_bytes(chunking, n), dtype=torch.uint8)
        offsets = starts.new_empty(S + 1, dtype=torch.int64)
        L.check(_encode(dev, starts, freqs, n, S, chunking, out, offsets, ws), "encode_intervals")
    if given:
        _written(out, ws)
    return out, offsets, ws


def token_states(data, stream_offsets, status=None, stream=None):
    """Decoder states of the streams, int64 [S, 2]: state and words taken."""
    dev, S = _streams(data, stream_offsets)[:2]
    with _place(dev, stream):
        states = torch.empty(S, 2, dtype=torch.int64, device=data.device)
        status = _status(status, dev)
    L.check(rans_token_states(data, stream_offsets, states, status, stream), "token_states")
    return states


def decode_tokens(logits, data, stream_offsets, states, adjust=None, stream_ids=None,
                  out_states=None, tokens=None, status=None, stream=None):
    """One decoding step: (tokens int32 [rows], new states).  Row r is the next
    position of stream stream_ids[r] (default r); out_states may be `states`.
    Rows with stream id -1 are skipped; without `tokens` they read -1."""
    rows = _rows(logits)
    n = rows[1]
    given = out_states is not None or tokens is not None
    with _place(rows[0], stream):
        if out_states is None:
            every = stream_ids is None and n == stream_offsets.numel() - 1
            out_states = torch.empty_like(states) if every else states.clone()
        if tokens is None:
            tokens = logits.new_empty(n, dtype=torch.int32) if stream_ids is None else \
                logits.new_full((n,), -1, dtype=torch.int32)
        L.check(_decode(rows, logits, adjust, data, stream_offsets, stream_ids, states,
                        out_states, tokens, status), "decode_tokens")
    if given:
        _written(out_states, tokens)
    return tokens, out_states


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, logprobs, inv_temperature, tail, status):
        rows, K, i, lp = _teacher(logits, ids, logprobs)
        dev, n = rows[:2]
        losses = logits.new_empty(n, dtype=torch.float32)
        stats = logits.new_empty((n, 8), dtype=torch.float32)
        status = _status(status, dev)
        L.check(L.lib().rans_distill_forward(
            _packed(logits, rows), i, lp, K, inv_temperature, int(tail), losses.data_ptr(),
            stats.data_ptr(), status.data_ptr(), _raw_stream(dev)), "distill_forward")
        ctx.save_for_backward(logits, ids, logprobs, stats)
        ctx.inv_temperature = inv_temperature
        return losses

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_losses):
        # (hooks on saved tensors may give back others than were saved)
        logits, ids, logprobs, stats = ctx.saved_tensors
        rows, K, i, lp = _teacher(logits, ids, logprobs)
        dev, n, v = rows[:3]
        s = _tensor(stats, torch.float32, (n, 8), dev, "stats")
        with _place(dev, None):
            grad = logits.new_empty((n, v))
            grad_losses = grad_losses.contiguous()
            g = _tensor(grad_losses, torch.float32, (n,), dev, "grad_losses")
            L.check(L.lib().rans_distill_backward(
                _packed(logits, rows), i, lp, K, ctx.inv_temperature, s, g, grad.data_ptr(), v,
                _raw_stream(dev)), "distill_backward")
        return grad, None, None, None, None, None


def distill_loss(logits, ids, logprobs, temperature=1.0, tail=True, status=None):
    """Rate of a teacher's listed tokens (ids int32, log probabilities float32,
    both [rows, K]) under the logits, less the teacher's entropy: float32
    [rows], in nats, differentiable in the logits.  tail: the teacher's
    remaining mass is one more bucket; else its list is renormalised.  The
    teacher's probabilities take no gradient."""
    inv = _positive(1.0 / _positive(temperature, "temperature"), "1 / temperature")
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise ValueError("logits: a CUDA tensor [rows, vocab]")
    with _place(logits.get_device(), None):
        return _Distill.apply(logits, ids, logprobs.detach(), inv, tail, status)


def distill_loss_and_grad(logits, ids, logprobs, weights, temperature=1.0, tail=True, grad=None,
                          status=None, stream=None):
    """(losses, gradient of sum(weights * losses) in the logits) in one call, for
    training loops that know the rows' weights; no autograd graph is built.
    grad may be the logits themselves."""
    inv = _positive(1.0 / _positive(temperature, "temperature"), "1 / temperature")
    rows = _rows(logits)
    given = grad is not None
    with _place(rows[0], stream):
        losses = logits.new_empty(rows[1], dtype=torch.float32)
        if not given:
            grad = logits.new_empty(rows[1:3])
        L.check(_both(rows, logits, ids, logprobs, inv, tail, weights, losses, grad, status),
                "distill")
    if given:
        _written(grad)
    return losses, grad
