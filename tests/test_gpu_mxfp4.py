"""Microscaled 4-bit numbers on the GPU: quantisation, values and products
against plain versions in 64 bits (numpy), at the sizes where they can go
wrong, and the promise that a row's logits do not depend on its batch."""
import math

import numpy as np
import pytest
import torch

import rans_entropy_coding_b200 as rb

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def host(x):
    return x.float().cpu().numpy().astype(np.float64)


def blocks_of(x):
    n, k = x.shape
    out = np.zeros((n, -(-k // 32) * 32))
    out[:, :k] = x
    return out.reshape(n, -1, 32)


def quantised(x):
    """(codes [rows, blocks, 32], scale bytes [rows, blocks]) from the definition."""
    b = blocks_of(x)
    top = np.abs(b).max(2)
    bad = ~np.isfinite(top)
    with np.errstate(all="ignore"):
        e = np.where((top > 0) & ~bad, np.frexp(np.where(bad, 1, top))[1] - 1 - 2, -127)
        e = np.maximum(e, -127)
        a = np.abs(b) / np.exp2(e)[:, :, None]
        # the nearest of the grid, ties to the even place
        d = np.abs(np.where(np.isfinite(a), a, 0)[..., None] - GRID)
        near = d.min(3, keepdims=True)
        first = (d == near).argmax(3)
        last = 7 - (d == near)[..., ::-1].argmax(3)
        code = np.where(first % 2 == 0, first, last)
    return code + 8 * np.signbit(b), np.where(bad, 255, e + 127)


def numbers(code, byte, cols):
    with np.errstate(all="ignore"):
        scale = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
        v = GRID[code & 7] * np.where(code >= 8, -1.0, 1.0) * scale[..., None]
    return v.reshape(code.shape[0], -1)[:, :cols]


def unpack(q):
    c = q.codes.cpu().numpy().astype(np.int64)
    code = np.stack([c & 15, c >> 4], 2).reshape(q.rows, -1, 32)
    return code, q.scale_rows().cpu().numpy().astype(np.int64)


def wide(n, k, dtype, pad=0, offset=0, fill=math.nan):
    """Rows inside a wider, possibly misaligned buffer of NaN."""
    flat = torch.full((offset + n * (k + pad),), fill, device="cuda", dtype=dtype)
    return flat[offset:].view(n, k + pad)[:, :k]


def rows(n, k, dtype, pad=0, offset=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + 7 * k + n)
    x = torch.randn(n, k, device="cuda", generator=g)
    x *= torch.exp2(torch.randint(-12, 12, (n, k), device="cuda", generator=g).float())
    out = wide(n, k, dtype, pad, offset)
    out.copy_(x)
    return out


# ----------------------------------------------------------- quantisation --
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n,k,pad,offset", [
    (1, 1, 0, 0), (3, 31, 0, 0), (5, 32, 0, 1), (2, 33, 1, 3), (129, 127, 0, 0), (130, 128, 8, 0),
    (7, 129, 3, 2), (4, 1000, 0, 5), (3, 1024, 0, 0), (2, 1025, 7, 1), (257, 2053, 3, 0)])
def test_quantise(n, k, pad, offset, dtype):
    x = rows(n, k, dtype, pad, offset)
    q = rb.quantize_mxfp4(x)
    code, byte = unpack(q)
    want, scale = quantised(host(x))
    assert np.array_equal(byte, scale)
    assert np.array_equal(code, want)
    # bytes of blocks past the columns are 0
    groups = -(-k // 128)
    tiles = q.scales.view(-1, groups, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * groups)
    assert bool((tiles[:n, -(-k // 32):] == 0).all())
    for out_dtype in TYPES:
        got = wide(n, k, out_dtype, pad, offset, fill=77.0)
        q.values(out=got)
        exact = numbers(code, byte, k)
        assert torch.equal(got.cpu(), torch.from_numpy(exact).to(out_dtype))
        if pad:
            assert bool((got.as_strided((n, pad), (k + pad, 1), offset + k)[:-1] == 77).all())
        assert torch.equal(q.values(out_dtype), got)


def test_quantise_every_value_and_edges():
    """All bfloat16 and float16 numbers, in blocks of one; blocks of zeros,
    subnormals, ties, the largest numbers, infinities and NaN."""
    for dtype in (BF16, F16):
        every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype).cuda()
        x = torch.zeros(65536, 32, device="cuda", dtype=dtype)
        x[:, 5] = every
        q = rb.quantize_mxfp4(x)
        code, byte = unpack(q)
        want, scale = quantised(host(x))
        assert np.array_equal(byte, scale)
        ok = byte[:, 0] != 255
        assert np.array_equal(code[ok], want[ok])
        back = q.values(F32).cpu().numpy()
        assert np.isnan(back[~ok]).all() and np.isfinite(back[ok]).all()
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0, 6.0, 7.0, 7.99, 0.2499, 0.2501, -0.25,
            -0.75, -5.0, 0.0, -0.0]
    base = torch.tensor(ties + [0.0] * (32 - len(ties)))
    scales = torch.exp2(torch.tensor([-149.0, -140, -129, -128, -127, -126, -125, -124, 0, 1, 60,
                                      124, 125]).double())
    x = (base.double() * scales[:, None]).float().cuda()
    code, byte = unpack(rb.quantize_mxfp4(x))
    want, scale = quantised(host(x))
    assert np.array_equal(byte, scale) and np.array_equal(code, want)


# --------------------------------------------------------------- products --
def check_product(out, a, w):
    """Against 64-bit sums of the same numbers.  Products of 4-bit numbers and
    powers of two are exact; each step of 64 columns rounds its sum and its
    addition by at most an ulp each of a number no larger than S, the sum of
    magnitudes: 2 (K / 64 + 1) 2^-23 S, then the output's own rounding."""
    exact = a @ w.T
    size = np.abs(a) @ np.abs(w.T)
    steps = -(-a.shape[1] // 64) + 1
    err = 2 * steps * 2.0 ** -23 * size
    eps = torch.finfo(out.dtype).eps / 2
    tiny = torch.finfo(out.dtype).smallest_normal * eps
    got = host(out)
    assert (np.abs(got - exact) <= err + eps * (np.abs(exact) + err) + tiny).all()


def head_of(v, k, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed + k)
    return rb.quantize_mxfp4(torch.randn(v, k, device="cuda", generator=g) / math.sqrt(k))


def dense(q):
    return q.values(F32).cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("n,v,k", [
    (1, 1, 1), (1, 128, 64), (1, 129, 32), (2, 300, 96), (16, 127, 128), (17, 257, 160),
    (33, 1000, 256), (48, 515, 257), (64, 640, 1000), (100, 300, 512), (128, 384, 2048),
    (129, 200, 300), (200, 1025, 640), (256, 259, 4096), (257, 300, 288), (300, 128, 64),
    (513, 1500, 1100)])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_product(n, v, k, dtype):
    w, x = head_of(v, k), rows(n, k, F32, seed=2)
    a = rb.quantize_mxfp4(x)
    out = wide(n, v, dtype, pad=3, offset=1, fill=77.0)
    status = rb.new_status()
    rb.mxfp4_logits(a, w, out=out, status=status)
    rb.check(rb.rans_get_status(status))
    check_product(out, dense(a), dense(w))
    edge = out.as_strided((n, 3), (v + 3, 1), 1 + v)
    assert bool((edge[:-1] == 77).all())
    assert torch.equal(rb.mxfp4_logits(x, w, dtype=dtype), out)


@pytest.mark.parametrize("n,k", [(129, 64), (160, 96), (200, 320), (256, 512), (257, 1056),
                                 (300, 288), (385, 640), (520, 128)])
def test_product_of_many_head_rows(n, k):
    """Blocks in pairs (more than 128 tokens, head rows for every SM)."""
    v = 148 * 128 + 301
    w, x = head_of(v, k), rows(n, k, F32, seed=6)
    a = rb.quantize_mxfp4(x)
    out = wide(n, v, F32, pad=3, offset=1, fill=77.0)
    status = rb.new_status()
    rb.mxfp4_logits(a, w, out=out, status=status)
    rb.check(rb.rans_get_status(status))
    check_product(out, dense(a), dense(w))
    assert bool((out.as_strided((n, 3), (v + 3, 1), 1 + v)[:-1] == 77).all())
    for m in (1, 100, 128):  # the same rows in batches that blocks take alone
        assert torch.equal(rb.mxfp4_logits(x[:m], w, dtype=F32), out[:m])
    assert torch.equal(rb.mxfp4_logits(x, w, dtype=BF16), out.bfloat16())


def test_rows_do_not_depend_on_their_batch():
    v, k = 1201, 1056
    w = head_of(v, k)
    x = rows(700, k, BF16, seed=3)
    whole = rb.mxfp4_logits(x, w, dtype=F32)
    for n in (1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 144, 255, 256, 257, 400):
        for at in (0, 3, 700 - n):
            assert torch.equal(rb.mxfp4_logits(x[at:at + n], w, dtype=F32), whole[at:at + n]), n
    order = torch.randperm(700, device="cuda")
    assert torch.equal(rb.mxfp4_logits(x[order], w, dtype=F32), whole[order])


def test_numbers_that_are_none_stay_in_their_rows():
    n, v, k = 40, 300, 320
    x = rows(n, k, F32, seed=4)
    x[7, 100] = math.nan
    x[9, 319] = math.inf
    wv = torch.randn(v, k, device="cuda")
    wv[200, 0] = math.nan
    out = rb.mxfp4_logits(x, rb.quantize_mxfp4(wv))
    bad = torch.zeros(n, v, dtype=torch.bool, device="cuda")
    bad[7] = bad[9] = True
    bad[:, 200] = True
    assert torch.equal(out.isnan(), bad)


def test_texts_coded_under_a_head():
    """Whole texts in, one row per stream and step out, hidden rows alone
    shared; and the intervals are those of the head's logits."""
    v, k, lengths = 5003, 416, [37, 0, 5, 64]
    w, n = head_of(v, k), sum([37, 0, 5, 64])
    hidden = rows(n, k, BF16, seed=5)
    tokens = torch.randint(0, v, (n,), device="cuda")
    for dtype in (F32, BF16):
        coder = rb.TokenCoder(head=w, logits_dtype=dtype)
        coder.add(hidden[:50], tokens[:50]).add(rb.quantize_mxfp4(hidden[50:]), tokens[50:])
        data, offsets = coder.streams(lengths)
        plain = rb.TokenCoder().add(rb.mxfp4_logits(hidden, w, dtype=dtype), tokens)
        assert torch.equal(plain.streams(lengths)[0], data)
        coder.begin(data, offsets)
        first = [0, 37, 37, 42]
        for t in range(max(lengths)):
            ids = [i for i, m in enumerate(lengths) if t < m]
            got = coder.step(torch.stack([hidden[first[i] + t] for i in ids]),
                             stream_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"))
            assert got.tolist() == [int(tokens[first[i] + t]) for i in ids]
        coder.finish()
