"""Microscaled 4-bit numbers, without a GPU: refusals at the C entry points and
in the Python layer, sizes, and the order of scales."""
import ctypes

import pytest
import torch

import rans_entropy_coding_b200 as rb
from rans_entropy_coding_b200 import build as rbuild
from rans_entropy_coding_b200 import mxfp4 as M

P = 1 << 20  # an address that nothing reads: every call here is refused on the host


def A(k):
    """Addresses far from P and from one another."""
    return P + (k << 24)


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rb.lib()


def floats(data=P, dtype=0, vocab=100, rows=4, stride=100):
    c = rb.rans_logits()
    c.data, c.dtype, c.vocab, c.rows, c.row_stride = data, dtype, vocab, rows, stride
    return ctypes.byref(c)


def numbers(codes=A(1), scales=A(2), rows=4, cols=100):
    c = rb.rans_mxfp4()
    c.codes, c.scales, c.rows, c.cols = codes, scales, rows, cols
    return ctypes.byref(c)


BAD = [dict(codes=None), dict(scales=None), dict(codes=A(1) + 8), dict(scales=A(2) + 8),
       dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=rb.MAX_VOCAB + 1)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_bad_numbers_are_refused(lib, bad):
    q = numbers(**bad)
    cols = bad.get("cols", 100)
    S = rb.ERR_ARG
    assert lib.rans_mxfp4_quantize(floats(rows=bad.get("rows", 4)), q, None) == S
    assert lib.rans_mxfp4_values(q, A(3), 0, 100, None) == S
    assert lib.rans_mxfp4_product(q, numbers(A(4), A(5), 50, cols), A(3), 0, 50, None, None) == S
    assert lib.rans_mxfp4_product(numbers(A(4), A(5), 50, cols), q, A(3), 0, 50, None, None) == S
    assert lib.rans_mxfp4_logits(floats(), q, A(3), 0, 50, A(6), 1 << 20, None, None) == S


def test_bad_products_are_refused(lib):
    S = rb.ERR_ARG
    a, w = numbers(A(1), A(2), 4, 100), numbers(A(3), A(4), 50, 100)

    def product(out=A(5), dtype=0, stride=50, status=None, a=a, w=w):
        return lib.rans_mxfp4_product(a, w, out, dtype, stride, status, None)

    assert product(out=None) == S
    assert product(out=A(5) + 2) == S
    assert product(dtype=3) == S
    assert product(stride=49) == S
    assert product(status=A(6) + 8) == S
    assert product(status=A(5) + 256) == S               # the result over the status word
    assert product(w=numbers(A(3), A(4), 50, 99)) == S    # other columns
    assert product(w=numbers(A(3), A(4), 0, 100)) == S
    assert product(w=numbers(A(3), A(4), rb.MAX_VOCAB + 1, 100), stride=rb.MAX_VOCAB + 1) == S
    for at in (1, 2, 3, 4):                              # the result over what is read
        assert product(out=A(at)) == S
        assert product(out=A(at) - 4) == S
    x = floats(A(1))

    def logits(x=x, w=w, out=A(5), ws=A(6), size=1 << 20, status=None):
        return lib.rans_mxfp4_logits(x, w, out, 0, 50, ws, size, status, None)

    need = rb.rans_mxfp4_logits_workspace_bytes(4, 100)
    assert need == 256 + 512
    assert logits(size=need - 1) == rb.ERR_CAPACITY
    assert logits(ws=None) == S
    assert logits(ws=A(6) + 128) == S
    assert logits(x=floats(A(1), vocab=99)) == S
    assert logits(x=floats(A(1), stride=99)) == S
    assert logits(x=floats(None)) == S
    assert logits(out=A(1)) == S                         # over the hidden rows
    assert logits(ws=A(1)) == S
    assert logits(ws=A(5)) == S
    assert logits(ws=A(4)) == S
    assert logits(ws=A(6), status=A(6)) == S


def test_bad_quantisations_are_refused(lib):
    S = rb.ERR_ARG
    q = numbers(A(1), A(2))
    assert lib.rans_mxfp4_quantize(floats(rows=5), q, None) == S
    assert lib.rans_mxfp4_quantize(floats(vocab=99), q, None) == S
    assert lib.rans_mxfp4_quantize(floats(A(1)), q, None) == S
    assert lib.rans_mxfp4_quantize(floats(A(2) + 16), q, None) == S
    assert lib.rans_mxfp4_quantize(floats(), numbers(A(1), A(1) + 16), None) == S
    assert lib.rans_mxfp4_values(q, None, 0, 100, None) == S
    assert lib.rans_mxfp4_values(q, A(3) + 1, 0, 100, None) == S
    assert lib.rans_mxfp4_values(q, A(3), 5, 100, None) == S
    assert lib.rans_mxfp4_values(q, A(3), 0, 99, None) == S
    assert lib.rans_mxfp4_values(q, A(1), 0, 100, None) == S
    assert lib.rans_mxfp4_values(q, A(2), 0, 100, None) == S


def test_no_rows_do_nothing(lib):
    none, w = numbers(None, None, 0, 100), numbers(A(3), A(4), 50, 100)
    assert lib.rans_mxfp4_quantize(floats(None, rows=0), none, None) == rb.OK
    assert lib.rans_mxfp4_values(none, None, 0, 0, None) == rb.OK
    assert lib.rans_mxfp4_product(none, w, None, 0, 0, None, None) == rb.OK
    assert lib.rans_mxfp4_logits(floats(None, rows=0), w, None, 0, 0, None, 0, None,
                                 None) == rb.OK


def test_sizes(lib):
    for rows, cols in ((0, 1), (1, 1), (1, 32), (1, 33), (128, 128), (129, 129), (131072, 4096),
                       ((1 << 31) - 1, rb.MAX_VOCAB)):
        row, scales = M._sizes(rows, cols)
        assert rb.rans_mxfp4_codes_bytes(rows, cols) == rows * row
        assert rb.rans_mxfp4_scales_bytes(rows, cols) == scales
    for rows, cols in ((-1, 1), (1, 0), (1 << 31, 1), (1, rb.MAX_VOCAB + 1)):
        assert rb.rans_mxfp4_codes_bytes(rows, cols) == 0
        assert rb.rans_mxfp4_scales_bytes(rows, cols) == 0


def test_host_tensors_and_bad_parts_are_refused(lib):
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    for call in (lambda: rb.Mxfp4(codes, scales), lambda: rb.Mxfp4(None, scales),
                 lambda: rb.quantize_mxfp4(torch.zeros(2, 32)),
                 lambda: rb.Mxfp4.from_rows(codes, scales),
                 lambda: rb.Mxfp4.from_rows(codes, torch.zeros(4, 3, dtype=torch.uint8)),
                 lambda: rb.Mxfp4.from_rows(codes, torch.zeros(4, 4, dtype=torch.uint8)),
                 lambda: rb.mxfp4_logits(torch.zeros(2, 32), None)):
        with pytest.raises(ValueError):
            call()
