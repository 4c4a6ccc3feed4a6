"""The 4-bit product's bounded waits: blocks whose tokens' copies stop give up with
RANS_ERR_TIMEOUT, whatever they were doing, and the next call is as if nothing had been.
(Copies in flight and products issued are waited for; no access goes out of range.)"""
import pytest
import torch

import rans_entropy_coding_b200 as rb
from test_gpu_mxfp4 import head_of, rows

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TRIES = 2000


def product(a, w, out, status, stages, tries=TRIES):
    code = {F32: 0, BF16: 2}[out.dtype]
    return rb.lib().rans_debug_product_timeout(
        a._c, w._c, out.data_ptr(), code, out.stride(0), status.data_ptr(), stages, tries,
        torch.cuda.current_stream().cuda_stream)


# few tokens, a narrow tile, a wide one, pairs; heads of several tiles a block
@pytest.mark.parametrize("n,v,k", [(8, 300, 256), (8, 40000, 1024), (100, 40000, 1024),
                                   (200, 1500, 4096), (256, 148 * 128 + 300, 1024),
                                   (300, 3 * 148 * 128, 1024)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_waits_that_give_up(n, v, k, dtype):
    w, a = head_of(v, k), rb.quantize_mxfp4(rows(n, k, F32, seed=8))
    want = rb.mxfp4_logits(a, w, dtype=dtype)
    status = rb.new_status()
    guard = torch.full((n + 2, v + 8), 77.0, device="cuda", dtype=dtype)
    out = guard[1:-1, :v]
    # nothing copied; the middle of a tile; between tiles; the middle of a later one
    for stages in (0, 1, k // 256 - 1, k // 256, k // 256 + 1, 2 * (k // 256)):
        rb.check(product(a, w, out, status, stages))
        err = rb.rans_get_status(status)
        blocks_need = -(-k // 256)  # of a block's first tile
        if stages < blocks_need:
            assert err == rb.ERR_TIMEOUT, stages
        else:
            assert err in (rb.OK, rb.ERR_TIMEOUT)
        assert bool((guard[0] == 77).all()) and bool((guard[-1] == 77).all())
        assert bool((guard[:, v:] == 77).all())
        assert torch.equal(rb.mxfp4_logits(a, w, dtype=dtype, status=status), want)
        assert rb.rans_get_status(status) == rb.OK
    # with all its copies the same call is a product
    rb.check(product(a, w, out, status, (1 << 32) - 1))
    assert rb.rans_get_status(status) == rb.OK and torch.equal(out, want)


def test_refusals():
    w, a = head_of(300, 64), rb.quantize_mxfp4(rows(8, 64, F32))
    out, status = torch.empty(8, 300, device="cuda"), rb.new_status()
    assert product(a, w, out, status, 0, 999) == rb.ERR_ARG
    assert product(a, w, out, status, 0, (1 << 21) + 1) == rb.ERR_ARG
    assert rb.lib().rans_debug_product_timeout(a._c, w._c, out.data_ptr(), 0, 300, None, 0, TRIES,
                                               None) == rb.ERR_ARG
