"""A row's logits have the same bits in a pair of blocks and in a single one, wherever the
row lies: the second half of a tile of tokens, the second block's, later tiles."""
import pytest
import torch

import rans_entropy_coding_b200 as rb
from test_gpu_mxfp4 import head_of, rows

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("n,k", [(129, 320), (200, 1056), (256, 512), (257, 640), (385, 1056),
                                 (385, 4096), (700, 300)])
def test_rows_of_a_pair_are_those_of_single_blocks(n, k):
    v = 148 * 128 + 301
    w, x = head_of(v, k), rows(n, k, F32, seed=9)
    out = rb.mxfp4_logits(x, w)
    for m in (1, 2, 17, 64, 128):  # batches that blocks take alone
        for at in (0, 64, 100, 127, 128, 200, 255, 256, n - 128, n - 1):
            if 0 <= at and at + m <= n:
                assert torch.equal(rb.mxfp4_logits(x[at:at + m], w), out[at:at + m]), (m, at)
    for at in (1, 37):  # and pairs at other places of their tiles
        assert torch.equal(rb.mxfp4_logits(x[at:], w), out[at:])
    # a head of fewer rows than a pair is taken for
    few = rb.quantize_mxfp4(w.values(F32)[:1500])
    assert torch.equal(rb.mxfp4_logits(x, few), out[:, :1500])
    for dtype in (F16, BF16):
        assert torch.equal(rb.mxfp4_logits(x, w, dtype=dtype), out.to(dtype))
