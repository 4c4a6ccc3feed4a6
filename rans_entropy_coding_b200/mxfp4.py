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
        (see from_rows for bytes in plain rows).
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
        c, s = codes.data_ptr(), scales.data_ptr()
        if (c | s) & 15:
            raise ValueError("codes and scales: aligned to 16 bytes")
        self.codes, self.scales, self.rows, self.cols, self.dev = codes, scales, rows, cols, dev
        self._c = _pack(c, s, rows, cols)

    @classmethod
    def empty(cls, rows, cols, device="cuda"):
        """Room for rows that a quantisation writes."""
        row, scales = _sizes(rows, cols)
        return cls(torch.empty((rows, row), dtype=torch.uint8, device=device),
                   torch.empty(scales, dtype=torch.uint8, device=device), cols)

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
        given = out is not None
        with T._place(self.dev, stream):
            if not given:
                if dtype not in T._LOGITS_CODE:
                    raise ValueError("dtype: float32, float16 or bfloat16, not %s" % dtype)
                out = torch.empty((self.rows, self.cols), dtype=dtype, device=self.codes.device)
            L.check(_values(self, out), "mxfp4_values")
        if given:
            T._written(out)
        return out


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
            out = Mxfp4.empty(rows[1], rows[2], x.device)
        L.check(_quantize(rows, x, out), "quantize_mxfp4")
    if given:
        T._written(out.codes, out.scales)
    return out


def mxfp4_logits(hidden, head, out=None, dtype=None, status=None, stream=None):
    """Logits [rows, vocab] of hidden rows under a head (Mxfp4 [vocab, cols]).

    hidden: rows of floats, which are quantised first, or Mxfp4.  The result is
    of `dtype` (by default the hidden rows' own, float32 for Mxfp4).  A row's logits are
    the same, bit for bit, in every batch, which is what TokenCoder asks for.
    """
    given = out is not None
    if isinstance(hidden, Mxfp4):
        dev, n = hidden.dev, hidden.rows
        _same(dev, hidden.cols, head)
        with T._place(dev, stream):
            if not given:
                out = torch.empty((n, head.rows), dtype=dtype or torch.float32,
                                  device=hidden.codes.device)
            L.check(_product(hidden, head, out, status), "mxfp4_logits")
    else:
        rows = T._rows(hidden, "hidden")
        dev, n, k = rows[:3]
        _same(dev, k, head)
        with T._place(dev, stream):
            if not given:
                out = hidden.new_empty((n, head.rows), dtype=dtype)
            row, scales = _sizes(n, k)
            # (torch's blocks are aligned to 512 bytes)
            ws = hidden.new_empty(((n * row + 255) & ~255) + scales, dtype=torch.uint8)
            L.check(_logits(rows, hidden, head, out, ws, status), "mxfp4_logits")
    if given:
        T._written(out)
    return out
