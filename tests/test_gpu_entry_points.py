"""The entry points under the helpers (rb.rans_*) of 4-bit numbers and searches give
what the helpers give, on results and workspaces of the caller's."""
import pytest
import torch

import rans_entropy_coding_b200 as rb
from test_gpu_mxfp4 import head_of, rows

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("own_stream", [False, True])
def test_numbers_and_products(own_stream):
    stream = torch.cuda.Stream() if own_stream else None
    x, head = rows(37, 300, BF16), head_of(1001, 300)
    want = rb.quantize_mxfp4(x)
    logits = rb.mxfp4_logits(x, head, dtype=F32)
    torch.cuda.synchronize()
    q = rb.Mxfp4.empty(37, 300)
    assert q.codes.numel() == rb.rans_mxfp4_codes_bytes(37, 300)
    assert q.scales.numel() == rb.rans_mxfp4_scales_bytes(37, 300)
    rb.check(rb.rans_mxfp4_quantize(x, q, stream=stream))
    values = torch.empty(37, 300, device="cuda")
    rb.check(rb.rans_mxfp4_values(q, values, stream=stream))
    out, again = torch.empty(2, 37, 1001, device="cuda")
    status = rb.new_status()
    rb.check(rb.rans_mxfp4_product(q, head, out, status, stream=stream))
    size = rb.rans_mxfp4_logits_workspace_bytes(37, 300)
    ws = torch.empty(size, device="cuda", dtype=torch.uint8)
    rb.check(rb.rans_mxfp4_logits(x, head, again, ws, status, stream=stream))
    assert rb.rans_mxfp4_logits(x, head, again, ws[:-1], status, stream=stream) == rb.ERR_CAPACITY
    torch.cuda.synchronize()
    rb.check(rb.rans_get_status(status))
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scale_rows(), want.scale_rows())
    assert torch.equal(values, want.values())
    assert torch.equal(out, logits) and torch.equal(again, logits)
    for call in (lambda: rb.rans_mxfp4_quantize(x, want.codes),
                 lambda: rb.rans_mxfp4_values(x, values),
                 lambda: rb.rans_mxfp4_product(q, x, out, None),
                 lambda: rb.rans_mxfp4_logits(x, head, out[:1], ws, None),
                 lambda: rb.rans_mxfp4_logits(x, head, out, ws.cpu(), None)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("own_stream", [False, True])
def test_searches(own_stream):
    stream = torch.cuda.Stream() if own_stream else None
    texts, beams, v, count = 3, 4, 5003, 9
    n = texts * beams
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(n, v, device="cuda", generator=g)
    rules = rb.LogitAdjust(temperature=0.8)
    plain, search = (rb.BeamSearch(texts, beams, 3, ends=[7]) for _ in range(2))
    best = rb.beam_select(x, plain.scores, beams, count, rules)
    state = torch.randn(n, 6, device="cuda", generator=g)
    torch.cuda.synchronize()
    scores, tokens = torch.empty(texts, count, device="cuda"), best[1].new_empty(texts, count)
    parents = torch.empty_like(tokens)
    ws = torch.empty(rb.rans_beam_workspace_bytes(F32, n, v, count), device="cuda",
                     dtype=torch.uint8)
    status = rb.new_status()
    rb.check(rb.rans_beam_select(x, rules, search.scores, beams, count, scores, tokens, parents, ws,
                                 status, stream=stream))
    assert rb.rans_beam_select(x, rules, search.scores, beams, count, scores, tokens, parents,
                               ws[:-1], status, stream=stream) == rb.ERR_CAPACITY
    rb.check(rb.rans_beam_advance(scores, tokens, parents, search, stream=stream))
    moved, copied = state.clone(), state.clone()
    torch.cuda.synchronize()
    for a, b in zip(best, (scores, tokens, parents)):
        assert torch.equal(a, b)
    assert search.lengths.tolist() == [1] * texts
    assert torch.equal(search.tokens.view(texts, beams).sort().values,
                       torch.where(search.scores.view(texts, beams) > -float("inf"),
                                   search.tokens.view(texts, beams), 0).sort().values)
    rb.check(rb.rans_reorder_states([moved], search.parents, None, None, status, stream=stream))
    rb.reorder_states(copied, search.parents)
    torch.cuda.synchronize()
    assert torch.equal(moved, copied)
    rb.check(rb.rans_get_status(status))
    for call in (lambda: rb.rans_beam_select(x, rules, search.scores, 5, count, scores, tokens,
                                             parents, ws, None),
                 lambda: rb.rans_beam_advance(scores[:1], tokens, parents, search),
                 lambda: rb.rans_reorder_states([moved], search.parents.long(), None, None, None)):
        with pytest.raises(ValueError):
            call()
