"""Microscaled 4-bit numbers and a model's output head on them
(include/rans_b200.h, "microscaled 4-bit numbers").

Argument checks and marshalling only, as in ``tokens``: every step runs in the
library's kernels (Mxfp4.from_rows and scale_rows, which lay a checkpoint's
scales out, are torch operations).  Rows are CUDA tensors [rows, cols] of
float32, float16 or bfloat16 whose rows are contiguous.  Calls run on the
tensors' device, on ``stream`` or that device's current stream.  Nothing here
takes part in autograd: results carry no gradient.
"""
import ctypes
import struct

import torch

from . import _lib as L
from . import tokens as T

_pack = struct.Struct("@PPqq").pack
assert struct.calcsize("@PPqq") == ctypes.sizeof(L.rans_mxfp4)
MX_BLOCK = 32
_MAX_ROWS = (1 << 31) - 1


def _sizes(rows, cols):
    """(bytes of a row's codes, bytes of all scales), as the library has them."""
    return (cols + 31) // 32 * 16, (rows + 127) // 128 * ((cols + 127) // 128) * 512


class Mxfp4:
    """Rows of microscaled 4-bit numbers.

    codes: uint8 [rows, 16 * ceil(cols / 32)], two elements to a byte, the lower
        column in the low half; a last block that the columns do not fill is
        filled up with 0.
    scales: uint8, the blocks' scale bytes in tiles of 128 rows by 4 blocks
        (see from_rows for bytes in plain rows); those of blocks past the columns
        must not be 255.
    cols: columns of the matrix; all that the codes hold, if not given.

    The tensors are kept, not copied.
    """

    def __init__(self, codes, scales, cols=None):
        dev = T._device(codes, "codes")
        if codes.dtype is not torch.uint8 or codes.dim() != 2 or not codes.is_contiguous() or \
                codes.shape[1] % 16 != 0:
            raise ValueError("codes: a contiguous uint8 tensor [rows, 16 * blocks]")
        rows = codes.shape[0]
        if cols is None:
            cols = 2 * codes.shape[1]
        if not 1 <= cols <= T.MAX_VOCAB or rows > _MAX_ROWS:
            raise ValueError("1 to %d columns, up to %d rows" % (T.MAX_VOCAB, _MAX_ROWS))
        row, need = _sizes(rows, cols)
        if codes.shape[1] != row:
            raise ValueError("codes: %d bytes a row for %d columns, not %d" % (
                row, cols, codes.shape[1]))
        T._tensor(scales, torch.uint8, None, dev, "scales")
        if scales.numel() != need:
            raise ValueError("scales: %d bytes for %d rows of %d columns, not %d" % (
                need, rows, cols, scales.numel()))
        if (codes.data_ptr() | scales.data_ptr()) & 15:
            raise ValueError("codes and scales: aligned to 16 bytes")
        self._set(codes, scales, rows, cols, dev)

    def _set(self, codes, scales, rows, cols, dev):
        self.codes, self.scales, self.rows, self.cols, self.dev = codes, scales, rows, cols, dev
        self._c = _pack(codes.data_ptr(), scales.data_ptr(), rows, cols)
        return self

    @classmethod
    def empty(cls, rows, cols, device="cuda"):
        """Room for rows that a quantisation writes."""
        if not 1 <= cols <= T.MAX_VOCAB or not 0 <= rows <= _MAX_ROWS:
            raise ValueError("1 to %d columns, up to %d rows" % (T.MAX_VOCAB, _MAX_ROWS))
        return cls._room(rows, cols, torch.empty(0, device=device))

    @classmethod
    def _room(cls, rows, cols, like):
        """Room on a tensor's device, of sizes that are known to be good."""
        row, scales = _sizes(rows, cols)
        return cls.__new__(cls)._set(like.new_empty((rows, row), dtype=torch.uint8),
                                     like.new_empty(scales, dtype=torch.uint8), rows, cols,
                                     T._device(like, "device"))

    @classmethod
    def from_rows(cls, codes, scales, cols=None):
        """From scale bytes in rows, uint8 [rows, blocks], as checkpoints hold them."""
        if not isinstance(scales, torch.Tensor) or scales.dim() != 2 or \
                scales.dtype is not torch.uint8:
            raise ValueError("scales: a uint8 tensor [rows, blocks]")
        rows, blocks = scales.shape
        if tuple(codes.shape) != (rows, 16 * blocks):
            raise ValueError("codes: [%d, %d] for these scales" % (rows, 16 * blocks))
        s = torch.nn.functional.pad(scales, (0, -blocks % 4, 0, -rows % 128))
        s = s.view(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
        return cls(codes.contiguous(), s.reshape(-1).contiguous(), cols)

    def scale_rows(self):
        """The scale bytes in rows, uint8 [rows, blocks]."""
        groups = (self.cols + 127) // 128
        s = self.scales.view(-1, groups, 32, 4, 4).permute(0, 3, 2, 1, 4)
        return s.reshape(-1, 4 * groups)[:self.rows, :(self.cols + 31) // 32].contiguous()

    def values(self, dtype=torch.float32, out=None, stream=None):
        """What the codes stand for, [rows, cols], rounded once to `dtype`."""
        with T._place(self.dev, stream):
            if out is None:
                code = _code(dtype)
                out = self.codes.new_empty((self.rows, self.cols), dtype=dtype)
                L.check(L.lib().rans_mxfp4_values(self._c, out.data_ptr(), code, self.cols,
                                                  T._raw_stream(self.dev)), "mxfp4_values")
                return out
            L.check(_values(self, out), "mxfp4_values")
        T._written(out)
        return out


def _code(dtype):
    code = T._LOGITS_CODE.get(dtype)
    if code is None:
        raise ValueError("dtype: float32, float16 or bfloat16, not %s" % dtype)
    return code


# ---------------------------------------------------------- C entry points --
def _numbers(q, what):
    if not isinstance(q, Mxfp4):
        raise ValueError("%s: Mxfp4" % what)
    return q


def rans_mxfp4_codes_bytes(rows, cols):
    return L.lib().rans_mxfp4_codes_bytes(rows, cols)


def rans_mxfp4_scales_bytes(rows, cols):
    return L.lib().rans_mxfp4_scales_bytes(rows, cols)


def rans_mxfp4_logits_workspace_bytes(rows, cols):
    return L.lib().rans_mxfp4_logits_workspace_bytes(rows, cols)


def rans_mxfp4_quantize(x, out, stream=None):
    rows = T._rows(x, "x")
    with T._place(rows[0], stream):
        result = _quantize(rows, x, out)
    T._written(out.codes, out.scales)
    return result


def _quantize(rows, x, out):
    if _numbers(out, "out").dev != rows[0] or out.rows != rows[1] or out.cols != rows[2]:
        raise ValueError("out: %d rows of %d columns on cuda:%d" % (rows[1], rows[2], rows[0]))
    return L.lib().rans_mxfp4_quantize(T._packed(x, rows), out._c, T._raw_stream(rows[0]))


def rans_mxfp4_values(q, out, stream=None):
    with T._place(_numbers(q, "q").dev, stream):
        result = _values(q, out)
    T._written(out)
    return result


def _values(q, out):
    o = T._rows(out, "out")
    if o[:3] != (q.dev, q.rows, q.cols):
        raise ValueError("out: a tensor [%d, %d] on cuda:%d" % (q.rows, q.cols, q.dev))
    return L.lib().rans_mxfp4_values(q._c, out.data_ptr(), o[3], o[4], T._raw_stream(q.dev))


def _result(dev, n, head, out):
    """(dtype code, row stride) of a result, checked."""
    o = T._rows(out, "out")
    if o[:3] != (dev, n, head.rows):
        raise ValueError("out: a tensor [%d, %d] on cuda:%d" % (n, head.rows, dev))
    return o[3], o[4]


def _word(status, dev):
    """A status word's address, or none: nobody would read it."""
    return None if status is None else T._status(status, dev).data_ptr()


def rans_mxfp4_product(a, head, out, status, stream=None):
    with T._place(_numbers(a, "a").dev, stream):
        result = _product(a, head, out, status)
    T._written(out)
    return result


def _product(a, head, out, status):
    _same(a.dev, a.cols, head)
    code, step = _result(a.dev, a.rows, head, out)
    return L.lib().rans_mxfp4_product(a._c, head._c, out.data_ptr(), code, step,
                                      _word(status, a.dev), T._raw_stream(a.dev))


def _same(dev, cols, head):
    if _numbers(head, "head").dev != dev:
        raise ValueError("head on cuda:%d, rows on cuda:%d" % (head.dev, dev))
    if head.cols != cols:
        raise ValueError("head of %d columns, rows of %d" % (head.cols, cols))
    if not 1 <= head.rows <= T.MAX_VOCAB:
        raise ValueError("head: a vocabulary of 1 to %d tokens" % T.MAX_VOCAB)


def rans_mxfp4_logits(hidden, head, out, workspace, status, stream=None):
    rows = T._rows(hidden, "hidden")
    with T._place(rows[0], stream):
        result = _logits(rows, hidden, head, out, workspace, status)
    T._written(out, workspace)
    return result


def _logits(rows, hidden, head, out, workspace, status):
    dev, n, k = rows[:3]
    _same(dev, k, head)
    code, step = _result(dev, n, head, out)
    w = T._tensor(workspace, torch.uint8, None, dev, "workspace")
    return L.lib().rans_mxfp4_logits(T._packed(hidden, rows), head._c, out.data_ptr(), code, step,
                                     w, workspace.numel(), _word(status, dev),
                                     T._raw_stream(dev))


# ----------------------------------------------------------------- helpers --
def quantize_mxfp4(x, out=None, stream=None):
    """Rows [rows, cols] as microscaled 4-bit numbers (Mxfp4), every block of 32
    columns with a scale of its own."""
    rows = T._rows(x, "x")
    given = out is not None
    with T._place(rows[0], stream):
        if not given:
            out = Mxfp4._room(rows[1], rows[2], x)
        L.check(_quantize(rows, x, out), "quantize_mxfp4")
    if given:
        T._written(out.codes, out.scales)
    return out


def mxfp4_logits(hidden, head, out=None, dtype=None, status=None, stream=None):
    """Logits [rows, vocab] of hidden rows under a head (Mxfp4 [vocab, cols]).

    hidden: rows of floats, which are quantised first, or Mxfp4.  The result is
    of `dtype` (by default the hidden rows' own, float32 for Mxfp4).  A row's logits are
    the same, bit for bit, in every batch, which is what TokenCoder asks for: of the same
    hidden row.  One whose numbers differ in a last place (computed in another batch, by
    libraries that split sums by it) may quantise to other codes, and then has other
    logits.  Against the float product, quantisation moves logits by some 16% of their
    spread for rows of even numbers, 20% with a few large channels.
    """
    given = out is not None
    quantised = isinstance(hidden, Mxfp4)
    rows = (hidden.dev, hidden.rows, hidden.cols) if quantised else T._rows(hidden, "hidden")
    dev, n, k = rows[:3]
    _same(dev, k, head)
    with T._place(dev, stream):
        if given:
            code, step = _result(dev, n, head, out)
        else:
            dtype = dtype or (torch.float32 if quantised else hidden.dtype)
            code, step = _code(dtype), head.rows
            out = head.codes.new_empty((n, step), dtype=dtype)
        word = None if status is None else T._status(status, dev).data_ptr()
        if quantised:
            done = L.lib().rans_mxfp4_product(hidden._c, head._c, out.data_ptr(), code, step, word,
                                              T._raw_stream(dev))
        else:
            row, scales = _sizes(n, k)
            size = ((n * row + 255) & ~255) + scales
            # (torch's blocks are aligned to 512 bytes)
            ws = head.codes.new_empty(size)
            done = L.lib().rans_mxfp4_logits(T._packed(hidden, rows), head._c, out.data_ptr(), code,
                                             step, ws.data_ptr(), size, word, T._raw_stream(dev))
        L.check(done, "mxfp4_logits")
    if given:
        T._written(out)
    return out
