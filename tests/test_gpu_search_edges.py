"""The 4-bit head, selection, searches and states where a program is not alone on
the stream: captured graphs, other streams, calls at once, empty and very large
arguments, outputs that autograd had saved."""
import math

import pytest
import torch

import rans_entropy_coding_b200 as rb
from test_gpu_beams import plain_reorder
from test_gpu_mxfp4 import head_of, rows

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def test_captured_heads():
    """Two graphs with their own workspaces, replayed in turn with new rows; a pair's
    sizes and a single block's."""
    small, big = head_of(1000, 320), head_of(148 * 128 + 5, 96)
    x, y = rows(5, 320, BF16), rows(200, 96, F32)
    rb.mxfp4_logits(x, small), rb.mxfp4_logits(y, big)  # kernels are set up outside
    graphs, outs = [], []
    for hidden, head in ((x, small), (y, big)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(rb.mxfp4_logits(hidden, head))
        graphs.append(g)
    for seed in (3, 4):
        x.copy_(rows(5, 320, BF16, seed=seed))
        y.copy_(rows(200, 96, F32, seed=seed))
        for g in graphs:
            g.replay()
        for g in graphs[::-1]:
            g.replay()
        assert torch.equal(outs[0], rb.mxfp4_logits(x, small))
        assert torch.equal(outs[1], rb.mxfp4_logits(y, big))


def test_a_captured_search():
    """One captured step, replayed, against a search that is not captured."""
    texts, beams, v, steps = 3, 4, 3001, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    every = torch.randn(steps, texts * beams, v, device="cuda", generator=g)
    o = dict(temperature=0.9, repetition=1.3)

    def make():
        return rb.BeamSearch(texts, beams, steps, ends=[7], length_penalty=0.5), \
            torch.arange(texts * beams * 6, device="cuda", dtype=F32).view(-1, 2, 3)

    plain, state = make()
    search, moved = make()
    warm, scratch = make()
    logits = every[0].clone()
    warm.step(logits, rb.LogitAdjust(history=warm.window, **o), [scratch])
    rules = rb.LogitAdjust(history=search.window, **o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens = search.step(logits, rules, [moved])
    assert int(search.lengths.sum()) == 0  # (captured, not run)
    for step in range(steps):
        want = plain.step(every[step], rb.LogitAdjust(history=plain.window, **o), [state])
        logits.copy_(every[step])
        graph.replay()
        assert torch.equal(tokens, want)
        assert torch.equal(search.scores, plain.scores) and torch.equal(moved, state)
    for a, b in zip(search.results(3), plain.results(3)):
        assert torch.equal(a, b)


def test_other_streams_and_calls_at_once():
    w, x = head_of(20000, 512), rows(300, 512, BF16)
    z = torch.randn(8, 30000, device="cuda")
    s = torch.zeros(8, device="cuda")
    state = torch.randn(8, 1000, device="cuda")
    parents = torch.tensor([[1, 0, 3, 3], [0, 0, 0, 0]], device="cuda", dtype=torch.int32)
    want = (rb.mxfp4_logits(x, w), *rb.beam_select(z, s, 4))
    moved = plain_reorder(state.cpu(), parents.cpu(), None, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(9):
        st = streams[i % 3]
        copy = state.clone()
        st.wait_stream(torch.cuda.current_stream())
        got.append((rb.mxfp4_logits(x, w, stream=st), *rb.beam_select(z, s, 4, stream=st),
                    rb.reorder_states(copy, parents, stream=st)))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g[:4], want):
            assert torch.equal(a, b)
        assert torch.equal(g[4].cpu(), moved)


def test_empty_calls():
    w = head_of(300, 64)
    none = torch.empty(0, 64, device="cuda")
    q = rb.quantize_mxfp4(none)
    assert q.values().shape == (0, 64) and q.scale_rows().shape == (0, 2)
    assert rb.mxfp4_logits(none, w).shape == (0, 300) == rb.mxfp4_logits(q, w).shape
    best, tokens, parents = rb.beam_select(torch.empty(0, 9, device="cuda"),
                                           torch.empty(0, device="cuda"), 4)
    assert best.shape == tokens.shape == parents.shape == (0, 8)
    rb.reorder_states([], torch.zeros(2, 3, dtype=torch.int32, device="cuda"))
    rb.reorder_states(torch.empty(0, 5, device="cuda"),
                      torch.zeros(0, 3, dtype=torch.int32, device="cuda"))
    rb.reorder_states(torch.empty(6, 0, device="cuda"),
                      torch.ones(2, 3, dtype=torch.int32, device="cuda"))
    search = rb.BeamSearch(0, 2, 5)
    assert search.step(torch.empty(0, 50, device="cuda")).numel() == 0


def test_results_given_by_the_caller_raise_versions():
    """A backward pass that had saved what a call then wrote to raises."""
    x = torch.randn(4, 64, device="cuda", requires_grad=True)
    w = head_of(32, 64)
    saved = x[:, :32] * 1.0
    y = (saved * saved).sum()
    rb.mxfp4_logits(x.detach(), w, out=saved.detach())
    with pytest.raises(RuntimeError):
        y.backward()
    saved = x * 1.0
    y = (saved * saved).sum()
    rb.reorder_states(saved.detach(), torch.ones(1, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(RuntimeError):
        y.backward()
    saved = x * 1.0
    y = (saved * saved).sum()
    rb.quantize_mxfp4(x.detach()).values(out=saved.detach())
    with pytest.raises(RuntimeError):
        y.backward()
    assert not rb.mxfp4_logits(x, w).requires_grad


def test_offsets_past_31_and_32_bits():
    # logits: 2.2e9 of them, 4.3 GB
    v, n, k = rb.MAX_VOCAB, 4200, 32
    w, x = head_of(v, k), rows(n, k, BF16)
    out = rb.mxfp4_logits(x, w)
    for r in (0, 2048, 4095, 4096, 4199):
        assert torch.equal(out[r:r + 1], rb.mxfp4_logits(x[r:r + 1], w))
    del out
    # many tiles of tokens on few head rows
    w, x = head_of(130, 96), rows(200001, 96, F16)
    out = rb.mxfp4_logits(x, w)
    for at in (0, 255, 256, 131071, 199936, 200000):
        assert torch.equal(out[at:at + 1], rb.mxfp4_logits(x[at:at + 1], w))
    assert torch.equal(out[1000:1100], rb.mxfp4_logits(x[1000:1100], w))
    del out
    # quantisation: 2.3e9 elements
    big = torch.empty(70000, 32800, device="cuda", dtype=BF16).normal_()
    q = rb.quantize_mxfp4(big)
    for r in (0, 65472, 69999):
        one = rb.quantize_mxfp4(big[r:r + 1])
        assert torch.equal(q.codes[r], one.codes[0])
        assert torch.equal(q.values(BF16)[r] if r == 69999 else one.values(BF16)[0],
                           one.values(BF16)[0])
    del big, q
    # states: 6 GB, rows of 1.5 GB
    state = torch.empty(4, 3, 1 << 28, device="cuda", dtype=F16)
    for b in range(4):
        state[b] = float(b)
    lengths = torch.tensor([(1 << 28) - 3], dtype=torch.int32, device="cuda")
    rb.reorder_states(state, torch.tensor([[1, 2, 3, 0]], dtype=torch.int32, device="cuda"),
                      lengths, axis=2)
    for b in range(4):
        assert bool((state[b, :, :-3] == (b + 1) % 4).all())
        assert bool((state[b, :, -3:] == b).all())


def test_search_rows_that_share_everything_tie_to_the_lower_beam():
    """Equal beams at rows of every alignment, under penalties too."""
    v, beams = 10007, 6
    row = torch.randn(v, device="cuda")
    for dtype in (F32, F16, BF16):
        flat = torch.full((1 + beams * (v + 3),), math.nan, device="cuda", dtype=dtype)
        x = flat[1:].view(beams, v + 3)[:, :v]
        x.copy_(row)
        s = torch.full((beams,), -3.0, device="cuda")
        n = torch.arange(beams, device="cuda")
        history = torch.randint(0, v, (500,), device="cuda", dtype=torch.int32)
        rules = rb.LogitAdjust(repetition=1.3, frequency=0.2, history=(
            history, torch.zeros_like(n), torch.full_like(n, 500)))
        for adjust in (None, rules):
            best, tokens, parents = rb.beam_select(x, s, beams, 2 * beams, adjust)
            assert parents[0].tolist() == [i % beams for i in range(2 * beams)]
            assert torch.equal(best[0, :beams], best[0, :1].expand(beams))
            assert torch.equal(tokens[0, :beams], tokens[0, :1].expand(beams))
