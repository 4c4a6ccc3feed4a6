"""Tokens under a language model's logits (include/rans_b200.h, "tokens under
a model's logits"): logit adjustment, intervals of tokens, streams of
intervals, decoding steps and the distillation loss.

Argument checks and marshalling only, as in ``_lib``; every step runs in the
library's kernels.  Logits are CUDA tensors [rows, vocab] of float32, float16
or bfloat16 whose rows are contiguous (a column slice of a wider buffer is
fine).  Calls run on the tensors' device, on ``stream`` or that device's
current stream.  ``status`` is a CUDA tensor from ``new_status()``; pass one to
learn of device errors (``check(rans_get_status(status))``).
"""
import contextlib
import ctypes

import torch

from . import _lib as L

_LOGITS_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
MAX_VOCAB = (1 << 19) - 8
MAX_TOP = 4096
TOKEN_PRECISION = 24

_no_context = contextlib.nullcontext()


def _place(device, stream):
    """Context in which to allocate and launch: the tensors' device and the
    caller's stream, where either is not the current one."""
    if stream is not None:
        return torch.cuda.stream(stream)
    if device.index != torch.cuda.current_device():
        return torch.cuda.device(device)
    return _no_context


def _launch_stream(device, stream):
    s = torch.cuda.current_stream(device) if stream is None else stream
    if s.device != device:
        raise ValueError("stream on %s, tensors on %s" % (s.device, device))
    return ctypes.c_void_p(s.cuda_stream)


def _logits(x, what="logits"):
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 2:
        raise ValueError("%s: a CUDA tensor [rows, vocab]" % what)
    if x.dtype not in _LOGITS_CODE:
        raise ValueError("%s: float32, float16 or bfloat16, not %s" % (what, x.dtype))
    n, v = x.shape
    if not 1 <= v <= MAX_VOCAB:
        raise ValueError("%s: a vocabulary of 1 to %d tokens" % (what, MAX_VOCAB))
    if (v > 1 and x.stride(1) != 1) or (n > 1 and x.stride(0) < v):
        raise ValueError("%s: rows must be contiguous and must not overlap" % what)
    c = L.rans_logits()
    c.data, c.dtype, c.vocab = x.data_ptr(), _LOGITS_CODE[x.dtype], v
    c.rows, c.row_stride = n, max(x.stride(0), v)
    return c


def _tensor(x, dtype, shape, device, what):
    """A contiguous CUDA tensor of this type and shape on this device."""
    if not isinstance(x, torch.Tensor) or x.dtype != dtype or x.device != device or \
            not x.is_contiguous() or (shape is not None and tuple(x.shape) != tuple(shape)):
        raise ValueError("%s: a contiguous %s tensor%s on %s" % (
            what, dtype, "" if shape is None else " of shape %s" % (tuple(shape),), device))
    return x


def new_status(device="cuda"):
    """A status word for the calls below (the first device error stays in it
    until rans_get_status reads it)."""
    return torch.zeros(32, dtype=torch.int64, device=device)


def _status(status, device):
    if status is None:
        return new_status(device)
    if not isinstance(status, torch.Tensor) or status.device != device or \
            not status.is_contiguous() or status.numel() * status.element_size() < 256:
        raise ValueError("status: from new_status() on %s" % device)
    return status


# ---------------------------------------------------------- C entry points --
def _ref(adjust, logits):
    return None if adjust is None else ctypes.byref(adjust.bind(logits))


def rans_adjust_logits(logits, adjust, out, stream=None):
    c, o = _logits(logits), _logits(out, "out")
    if out.shape != logits.shape or out.device != logits.device:
        raise ValueError("out: a tensor of the logits' shape on their device")
    with _place(logits.device, stream):
        return L.lib().rans_adjust_logits(
            ctypes.byref(c), _ref(adjust, logits), L._ptr(out), o.dtype, o.row_stride,
            _launch_stream(logits.device, stream))


def rans_token_intervals(logits, adjust, tokens, starts, freqs, status, stream=None):
    c, n, dev = _logits(logits), logits.shape[0], logits.device
    for x, what in ((tokens, "tokens"), (starts, "starts"), (freqs, "freqs")):
        _tensor(x, torch.int32, (n,), dev, what)
    with _place(dev, stream):
        return L.lib().rans_token_intervals(
            ctypes.byref(c), _ref(adjust, logits), L._ptr(tokens), L._ptr(starts),
            L._ptr(freqs), L._ptr(_status(status, dev)), _launch_stream(dev, stream))


def rans_encode_intervals(starts, freqs, n, chunking, out, stream_offsets, workspace,
                          stream=None):
    dev = starts.device
    _tensor(starts, torch.int32, (n,), dev, "starts")
    _tensor(freqs, torch.int32, (n,), dev, "freqs")
    _tensor(out, torch.uint8, None, dev, "out")
    _tensor(workspace, torch.uint8, None, dev, "workspace")
    S = L.rans_num_streams(chunking, n)
    if S >= 0:
        _tensor(stream_offsets, torch.int64, (S + 1,), dev, "stream_offsets")
    with _place(dev, stream):
        return L.lib().rans_encode_intervals(
            L._ptr(starts), L._ptr(freqs), n, ctypes.byref(chunking.c), L._ptr(out), out.numel(),
            L._ptr(stream_offsets), L._ptr(workspace), workspace.numel(),
            _launch_stream(dev, stream))


def _streams(data, stream_offsets):
    dev = data.device
    _tensor(data, torch.uint8, None, dev, "data")
    _tensor(stream_offsets, torch.int64, None, dev, "stream_offsets")
    if stream_offsets.numel() < 1:
        raise ValueError("stream_offsets: S + 1 offsets")
    return dev, stream_offsets.numel() - 1


def rans_token_states(data, stream_offsets, states, status, stream=None):
    dev, S = _streams(data, stream_offsets)
    _tensor(states, torch.int64, (S, 2), dev, "states")
    with _place(dev, stream):
        return L.lib().rans_token_states(
            L._ptr(data), data.numel(), L._ptr(stream_offsets), S, L._ptr(states),
            L._ptr(_status(status, dev)), _launch_stream(dev, stream))


def rans_decode_tokens(logits, adjust, data, stream_offsets, stream_ids, states_in, states_out,
                       tokens, status, stream=None):
    c, n = _logits(logits), logits.shape[0]
    dev, S = _streams(data, stream_offsets)
    if dev != logits.device:
        raise ValueError("data on %s, logits on %s" % (dev, logits.device))
    if stream_ids is not None:
        _tensor(stream_ids, torch.int32, (n,), dev, "stream_ids")
    _tensor(states_in, torch.int64, (S, 2), dev, "states")
    _tensor(states_out, torch.int64, (S, 2), dev, "states_out")
    _tensor(tokens, torch.int32, (n,), dev, "tokens")
    with _place(dev, stream):
        return L.lib().rans_decode_tokens(
            ctypes.byref(c), _ref(adjust, logits), L._ptr(data), data.numel(),
            L._ptr(stream_offsets), S, L._ptr(stream_ids), L._ptr(states_in),
            L._ptr(states_out), L._ptr(tokens), L._ptr(_status(status, dev)),
            _launch_stream(dev, stream))


def rans_token_states_finish(stream_offsets, states, status, stream=None):
    dev, S = _streams(torch.empty(0, dtype=torch.uint8, device=states.device), stream_offsets)
    _tensor(states, torch.int64, (S, 2), dev, "states")
    with _place(dev, stream):
        return L.lib().rans_token_states_finish(
            L._ptr(stream_offsets), S, L._ptr(states), L._ptr(_status(status, dev)),
            _launch_stream(dev, stream))


def _teacher(logits, ids, logprobs):
    c, n, dev = _logits(logits), logits.shape[0], logits.device
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or not 1 <= ids.shape[1] <= MAX_TOP:
        raise ValueError("ids: a tensor [rows, K], K from 1 to %d" % MAX_TOP)
    _tensor(ids, torch.int32, (n, ids.shape[1]), dev, "ids")
    _tensor(logprobs, torch.float32, (n, ids.shape[1]), dev, "logprobs")
    return c, n, ids.shape[1], dev


def rans_distill_forward(logits, ids, logprobs, inv_temperature, tail, losses, stats, status,
                         stream=None):
    c, n, K, dev = _teacher(logits, ids, logprobs)
    _tensor(losses, torch.float32, (n,), dev, "losses")
    _tensor(stats, torch.float32, (n, 8), dev, "stats")
    with _place(dev, stream):
        return L.lib().rans_distill_forward(
            ctypes.byref(c), L._ptr(ids), L._ptr(logprobs), K, inv_temperature, int(tail),
            L._ptr(losses), L._ptr(stats), L._ptr(_status(status, dev)),
            _launch_stream(dev, stream))


def _grad_of(logits, grad):
    o = _logits(grad, "grad")
    if grad.shape != logits.shape or grad.dtype != logits.dtype or grad.device != logits.device:
        raise ValueError("grad: a tensor of the logits' shape and type on their device")
    return o.row_stride


def rans_distill_backward(logits, ids, logprobs, inv_temperature, stats, grad_losses, grad,
                          stream=None):
    c, n, K, dev = _teacher(logits, ids, logprobs)
    _tensor(stats, torch.float32, (n, 8), dev, "stats")
    _tensor(grad_losses, torch.float32, (n,), dev, "grad_losses")
    stride = _grad_of(logits, grad)
    with _place(dev, stream):
        return L.lib().rans_distill_backward(
            ctypes.byref(c), L._ptr(ids), L._ptr(logprobs), K, inv_temperature, L._ptr(stats),
            L._ptr(grad_losses), L._ptr(grad), stride, _launch_stream(dev, stream))


def rans_distill(logits, ids, logprobs, inv_temperature, tail, grad_losses, losses, grad, status,
                 stream=None):
    c, n, K, dev = _teacher(logits, ids, logprobs)
    _tensor(grad_losses, torch.float32, (n,), dev, "weights")
    _tensor(losses, torch.float32, (n,), dev, "losses")
    stride = _grad_of(logits, grad)
    with _place(dev, stream):
        return L.lib().rans_distill(
            ctypes.byref(c), L._ptr(ids), L._ptr(logprobs), K, inv_temperature, int(tail),
            L._ptr(grad_losses), L._ptr(losses), L._ptr(grad), stride,
            L._ptr(_status(status, dev)), _launch_stream(dev, stream))


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


def pack_mask(allowed):
    """Words of a bool tensor [rows, vocab] (or [vocab]) of allowed tokens, as
    LogitAdjust takes them: bit v & 31 of word v >> 5."""
    flat = allowed if allowed.dim() == 2 else allowed[None]
    n, v = flat.shape
    bits = torch.nn.functional.pad(flat, (0, -v % 32)).view(n, -1, 32).to(torch.int64)
    words = (bits << torch.arange(32, device=flat.device)).sum(2)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    return words if allowed.dim() == 2 else words[0]


class LogitAdjust:
    """What is done to rows of logits before they are used.

    temperature, repetition, frequency, presence: numbers for all rows, or
        float32 CUDA tensors [rows] (any of them).
    history: (tokens int32, begin int64 [rows], end int64 [rows]): row r's
        history is tokens[begin[r]:end[r]].
    bias: (ids int32, values float32, begin int64 [rows], end int64 [rows]);
        a token's last entry in its row's window counts.
    mask: int32 [rows, words] or [words] (for all rows) with 1 bits where
        tokens are allowed; see pack_mask.

    The tensors are read by each call, so a program may keep one LogitAdjust
    and update them in place between steps.
    """

    def __init__(self, temperature=1.0, repetition=1.0, frequency=0.0, presence=0.0,
                 history=None, bias=None, mask=None):
        c = L.rans_adjust()
        self.c, self._rows, self._words, self._keep, self._device = c, None, 0, [], None
        parts = (repetition, frequency, presence, temperature)
        if any(isinstance(x, torch.Tensor) for x in parts):
            rows = {x.numel() for x in parts if isinstance(x, torch.Tensor)}
            dev = [x.device for x in parts if isinstance(x, torch.Tensor)][0]
            if len(rows) != 1:
                raise ValueError("per-row parameters of different lengths")
            n = rows.pop()
            cols = [x if isinstance(x, torch.Tensor) else
                    torch.full((n,), float(x), device=dev) for x in parts]
            for x in cols:
                _tensor(x, torch.float32, (n,), dev, "per-row parameters")
            cols[3] = 1.0 / cols[3]
            c.params = self._hold(torch.stack(cols, 1), n)
        else:
            c.repetition = _positive(repetition, "repetition")
            c.frequency = _finite(frequency, "frequency")
            c.presence = _finite(presence, "presence")
            c.inv_temperature = _positive(1.0 / _positive(temperature, "temperature"),
                                          "1 / temperature")
        if history is not None:
            tokens, begin, end = history
            dev, n = tokens.device, begin.numel()
            _tensor(tokens, torch.int32, (tokens.numel(),), dev, "history tokens")
            _tensor(begin, torch.int64, (n,), dev, "history begin")
            _tensor(end, torch.int64, (n,), dev, "history end")
            if tokens.numel() > 0:
                c.history, c.history_len = self._hold(tokens), tokens.numel()
                c.history_begin, c.history_end = self._hold(begin, n), self._hold(end, n)
        if bias is not None:
            ids, values, begin, end = bias
            dev, n = ids.device, begin.numel()
            _tensor(ids, torch.int32, (ids.numel(),), dev, "bias ids")
            _tensor(values, torch.float32, (ids.numel(),), dev, "bias values")
            _tensor(begin, torch.int64, (n,), dev, "bias begin")
            _tensor(end, torch.int64, (n,), dev, "bias end")
            if ids.numel() > 0:
                c.bias_ids, c.bias_values = self._hold(ids), self._hold(values)
                c.bias_len = ids.numel()
                c.bias_begin, c.bias_end = self._hold(begin, n), self._hold(end, n)
        if mask is not None:
            if mask.dtype != torch.int32 or mask.dim() not in (1, 2) or \
                    (mask.shape[-1] > 1 and mask.stride(-1) != 1):
                raise ValueError("mask: int32 words [rows, words] or [words], from pack_mask")
            self._words = mask.shape[-1]
            if mask.dim() == 2:
                if mask.shape[0] > 1 and mask.stride(0) < mask.shape[1]:
                    raise ValueError("mask: rows must not overlap")
                c.mask = self._hold(mask, mask.shape[0])
                c.mask_stride = max(mask.stride(0), mask.shape[1])
            else:
                c.mask = self._hold(mask)

    def _hold(self, x, rows=None):
        if not x.is_cuda or (self._device is not None and x.device != self._device):
            raise ValueError("LogitAdjust takes CUDA tensors on one device")
        if rows is not None:
            if self._rows is not None and rows != self._rows:
                raise ValueError("parts for %d and for %d rows" % (self._rows, rows))
            self._rows = rows
        self._device = x.device
        self._keep.append(x)
        return x.data_ptr()

    def bind(self, logits):
        """The C struct, checked against the rows it is to be used on."""
        n, v = logits.shape
        if self._device is not None and self._device != logits.device:
            raise ValueError("LogitAdjust on %s, logits on %s" % (self._device, logits.device))
        if self._rows is not None and self._rows != n:
            raise ValueError("LogitAdjust for %d rows, logits of %d" % (self._rows, n))
        if self.c.mask and self._words < (v + 31) // 32:
            raise ValueError("mask: %d words for %d tokens" % (self._words, v))
        return self.c


def adjust_logits(logits, adjust, out=None, dtype=None, stream=None):
    """Adjusted logits (penalties, biases, temperature, mask) for a sampler, in
    the logits' type or `dtype`; out may be the logits themselves."""
    _logits(logits)
    with _place(logits.device, stream):
        if out is None:
            out = torch.empty(logits.shape, dtype=dtype or logits.dtype, device=logits.device)
        L.check(rans_adjust_logits(logits, adjust, out, stream), "adjust_logits")
    return out


def token_intervals(logits, tokens, adjust=None, starts=None, freqs=None, status=None,
                    stream=None):
    """(starts, freqs), int32 [rows]: each row's interval of its token at
    TOKEN_PRECISION bits.  Rows with token -1 are skipped."""
    _logits(logits)
    with _place(logits.device, stream):
        n, dev = logits.shape[0], logits.device
        if starts is None:
            starts = torch.empty(n, dtype=torch.int32, device=dev)
        if freqs is None:
            freqs = torch.empty(n, dtype=torch.int32, device=dev)
        L.check(rans_token_intervals(logits, adjust, tokens, starts, freqs,
                                     _status(status, dev), stream), "token_intervals")
    return starts, freqs


def encode_intervals(starts, freqs, chunking, out=None, ws=None, stream=None):
    """(buffer, stream_offsets[S + 1], workspace): like encode_with_indexes;
    the coded bytes are buffer[:stream_offsets[-1]], device errors
    rans_get_status(workspace).  ws: a workspace to reuse."""
    n, dev = starts.numel(), starts.device
    S = L.rans_num_streams(chunking, n)
    if S < 0:
        L.check(int(S), "num_streams")
    with _place(dev, stream):
        if ws is None:
            ws = L.aligned_empty(L.rans_encode_workspace_bytes(chunking, n), dev)
        if out is None:
            out = torch.empty(L.rans_max_compressed_bytes(chunking, n), dtype=torch.uint8,
                              device=dev)
        offsets = torch.empty(S + 1, dtype=torch.int64, device=dev)
        L.check(rans_encode_intervals(starts, freqs, n, chunking, out, offsets, ws, stream),
                "encode_intervals")
    return out, offsets, ws


def token_states(data, stream_offsets, status=None, stream=None):
    """Decoder states of the streams, int64 [S, 2]: state and words taken."""
    with _place(data.device, stream):
        states = torch.empty(stream_offsets.numel() - 1, 2, dtype=torch.int64,
                             device=data.device)
        L.check(rans_token_states(data, stream_offsets, states, status, stream), "token_states")
    return states


def decode_tokens(logits, data, stream_offsets, states, adjust=None, stream_ids=None,
                  out_states=None, tokens=None, status=None, stream=None):
    """One decoding step: (tokens int32 [rows], new states).  Row r is the next
    position of stream stream_ids[r] (default r); out_states may be `states`.
    Rows with stream id -1 are skipped; without `tokens` they read -1."""
    _logits(logits)
    n, dev = logits.shape[0], logits.device
    with _place(dev, stream):
        if out_states is None:
            every = stream_ids is None and n == stream_offsets.numel() - 1
            out_states = torch.empty_like(states) if every else states.clone()
        if tokens is None:
            tokens = torch.empty(n, dtype=torch.int32, device=dev) if stream_ids is None else \
                torch.full((n,), -1, dtype=torch.int32, device=dev)
        L.check(rans_decode_tokens(logits, adjust, data, stream_offsets, stream_ids, states,
                                   out_states, tokens, _status(status, dev), stream),
                "decode_tokens")
    return tokens, out_states


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, logprobs, inv_temperature, tail, status):
        n, dev = logits.shape[0], logits.device
        losses = torch.empty(n, dtype=torch.float32, device=dev)
        stats = torch.empty(n, 8, dtype=torch.float32, device=dev)
        L.check(rans_distill_forward(logits, ids, logprobs, inv_temperature, tail, losses, stats,
                                     status), "distill_forward")
        ctx.save_for_backward(logits, ids, logprobs, stats)
        ctx.inv_temperature = inv_temperature
        return losses

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_losses):
        logits, ids, logprobs, stats = ctx.saved_tensors
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        L.check(rans_distill_backward(logits, ids, logprobs, ctx.inv_temperature, stats,
                                      grad_losses.contiguous(), grad), "distill_backward")
        return grad, None, None, None, None, None


def distill_loss(logits, ids, logprobs, temperature=1.0, tail=True, status=None):
    """Rate of a teacher's listed tokens (ids int32, log probabilities float32,
    both [rows, K]) under the logits, less the teacher's entropy: float32
    [rows], in nats, differentiable in the logits.  tail: the teacher's
    remaining mass is one more bucket; else its list is renormalised.  The
    teacher's probabilities take no gradient."""
    _teacher(logits, ids, logprobs)
    inv = _positive(1.0 / _positive(temperature, "temperature"), "1 / temperature")
    with _place(logits.device, None):
        return _Distill.apply(logits, ids, logprobs.detach(), inv, bool(tail),
                              _status(status, logits.device))


def distill_loss_and_grad(logits, ids, logprobs, weights, temperature=1.0, tail=True, grad=None,
                          status=None, stream=None):
    """(losses, gradient of sum(weights * losses) in the logits) in one call, for
    training loops that know the rows' weights; no autograd graph is built.
    grad may be the logits themselves."""
    _teacher(logits, ids, logprobs)
    inv = _positive(1.0 / _positive(temperature, "temperature"), "1 / temperature")
    with _place(logits.device, stream):
        losses = torch.empty(logits.shape[0], dtype=torch.float32, device=logits.device)
        if grad is None:
            grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        L.check(rans_distill(logits, ids, logprobs, inv, tail, weights, losses, grad,
                             _status(status, logits.device), stream), "distill")
    return losses, grad
