"""Beam search on the GPU: selection, bookkeeping and reordered states against
plain versions in 64 bits (numpy and Python), at the sizes, masks and maps where
they can go wrong."""
import math

import numpy as np
import pytest
import torch

import rans_entropy_coding_b200 as rb
import token_oracle as TO
from test_gpu_tokens import make_adjust, make_logits, numpy_rows

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
# A sum of exponentials: each is off by 2 units of 2^-24 (series, rounding of the
# difference), a thread's sum by 2 more, and each of at most 8 raised maxima by 1.5:
# under 16 units of a share of the sum, hence 2^-20 in its logarithm.
SUM = 2.0 ** -20


def exact_rows(x, o):
    """Adjusted logits of all rows by the library's float32 steps, in 64 bits."""
    z = numpy_rows(x)
    out = np.empty(z.shape)
    for r in range(z.shape[0]):
        if o is None:
            out[r] = z[r]
            continue
        with np.errstate(all="ignore"):
            y, _ = TO.adjusted(z[r], o, r, np.float32)
            t = TO.param(o, "temperature", r, 1.0)
            y = y * (np.float32(1) / np.float32(t))
        y[~TO.allowed(o, r, y.size)] = -np.inf
        out[r] = y
    return out


def host_rows(x):
    return numpy_rows(x).astype(np.float64)


def totals(x, scores):
    with np.errstate(all="ignore"):
        m = x.max(1, keepdims=True)
        lse = m + np.log(np.exp(x - m).sum(1, keepdims=True))
        t = scores[:, None] + (x - lse)
    t[~(x > -np.inf)] = -np.inf
    t[scores == -np.inf] = -np.inf
    return t


def check_selection(got, total, beams, count):
    """total: [texts * beams, vocab] in 64 bits."""
    best, tokens, parents = (g.cpu().numpy() for g in got)
    texts, v = total.shape[0] // beams, total.shape[1]
    for t in range(texts):
        flat = total[t * beams:(t + 1) * beams].reshape(-1)
        order = np.argsort(-flat, kind="stable")[:count]
        order = order[flat[order] > -np.inf]
        n = order.size
        assert (tokens[t, n:] == -1).all() and (parents[t, n:] == -1).all()
        assert (best[t, n:] == -np.inf).all()
        assert (tokens[t, :n] >= 0).all() and (parents[t, :n] >= 0).all()
        mine = parents[t, :n].astype(np.int64) * v + tokens[t, :n]
        assert np.unique(mine).size == n
        gap = np.abs(flat[mine] - flat[order])
        assert (gap <= 2 * SUM).all()
        # what is as good to the bit, and what no error reaches, is in order
        assert (mine[gap == 0] == order[gap == 0]).all()
        assert (gap == 0).sum() >= 0.9 * n
        want = flat[mine]
        assert (np.abs(best[t, :n] - want) <= SUM + 2.0 ** -24 * np.abs(want)).all()


def make_scores(n, seed, beams):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = -9.0 * torch.rand(n, device="cuda", generator=g) - 1.0
    if n > 2:
        s[2] = -math.inf  # a dead beam
    return s


# --------------------------------------------------------------- selection --
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v,pad", [(1, 0), (7, 1), (33, 0), (1000, 3), (8185, 7), (20011, 5),
                                   (70000, 0)])
def test_select(v, pad, dtype):
    for texts, beams, count in ((1, 1, 1), (1, 4, 8), (3, 5, 10), (2, 2, 128)):
        n = texts * beams
        x = make_logits(n, v, dtype, pad, seed=beams, offset=pad)
        s = make_scores(n, v, beams)
        status = rb.new_status()
        got = rb.beam_select(x, s, beams, count, status=status)
        rb.check(rb.rans_get_status(status))
        check_selection(got, totals(exact_rows(x, None), s.cpu().numpy().astype(float)), beams,
                        count)
        for a, b in zip(got, rb.beam_select(x, s, beams, count)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v,pad", [(33, 0), (1000, 3), (20011, 5)])
def test_select_adjusted(v, pad, dtype):
    texts, beams, count = 3, 4, 8
    n = texts * beams
    x = make_logits(n, v, dtype, pad, seed=7, offset=pad)
    s = make_scores(n, v, beams)
    for parts in (dict(), dict(mask=False), dict(history=False, bias=False),
                  dict(history=False, per_row=True), dict(bias=False, mask=False),
                  dict(long=9000)):
        a, o = make_adjust(n, v, seed=v + len(parts), **parts)
        got = rb.beam_select(x, s, beams, count, a)
        check_selection(got, totals(exact_rows(x, o), s.cpu().numpy().astype(float)), beams,
                        count)


@pytest.mark.parametrize("beams", [1, 7, 16, 64])
def test_select_many_beams(beams):
    x = make_logits(2 * beams, 9001, BF16, 1, seed=beams)
    s = make_scores(2 * beams, 1, beams)
    count = min(2 * beams, 128)
    check_selection(rb.beam_select(x, s, beams, count),
                    totals(exact_rows(x, None), s.cpu().numpy().astype(float)), beams, count)


def test_select_large():
    """More parts than one, tables past their span and more touched tokens than
    a table holds."""
    v, beams = 300007, 2
    x = make_logits(beams, v, F16, 1, seed=3)
    s = make_scores(beams, 5, beams)
    a, o = make_adjust(beams, v, seed=3, long=30000)
    check_selection(rb.beam_select(x, s, beams, 16, a),
                    totals(exact_rows(x, o), s.cpu().numpy().astype(float)), beams, 16)
    x = make_logits(600, 40000, BF16, 0, seed=4)  # a block takes a row
    s = make_scores(600, 6, 8)
    check_selection(rb.beam_select(x, s, 8, 16),
                    totals(exact_rows(x, None), s.cpu().numpy().astype(float)), 8, 16)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v", [5, 1000, 30000])
def test_ties(v, dtype):
    """Equal logits, a few levels, equal beams: lower beams and tokens first."""
    beams, count = 3, 12
    x = torch.zeros(2 * beams, v, device="cuda", dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(v)
    x[beams:] = torch.randint(0, 3, (v,), device="cuda", generator=g).to(dtype)
    s = torch.full((2 * beams,), -2.0, device="cuda")
    best, tokens, parents = rb.beam_select(x, s, beams, count)
    n = min(count, v)
    assert tokens[0, :n].tolist() == list(range(n)) and parents[0, :n].tolist() == [0] * n
    z = numpy_rows(x[beams:])
    total = np.concatenate([z[b] for b in range(beams)])
    order = np.argsort(-total, kind="stable")[:count]
    assert (tokens[1].cpu().numpy()[:order.size] == order % v).all()
    assert (parents[1].cpu().numpy()[:order.size] == order // v).all()
    # a mask that leaves a few, and one that leaves none
    allowed = torch.zeros(2 * beams, v, dtype=torch.bool, device="cuda")
    allowed[1, v - 1] = allowed[4, 0] = True
    out = rb.beam_select(x, s, beams, count, rb.LogitAdjust(mask=rb.pack_mask(allowed)))
    assert out[1][:, 0].tolist() == [v - 1, 0] and out[2][:, 0].tolist() == [1, 1]
    assert bool((out[0][:, 0] == -2).all()) and bool((out[1][:, 1:] == -1).all())
    none = rb.beam_select(x, s, beams, count,
                          rb.LogitAdjust(mask=rb.pack_mask(torch.zeros_like(allowed))))
    assert bool((none[0] == -math.inf).all()) and bool((none[2] == -1).all())


def test_ties_of_zeros_and_under_penalties():
    """Zeros of both signs are equal; more equal logits than a block keeps, some of
    them touched; a mask that leaves single tokens in whole tiles of nothing."""
    v, beams, count = 30000, 2, 10
    x = torch.zeros(beams, v, device="cuda")
    x[:, ::2] = -0.0
    s = torch.tensor([-1.0, -1.0], device="cuda")
    best, tokens, parents = rb.beam_select(x, s, beams, count)
    assert tokens[0].tolist() == list(range(count)) and parents[0].tolist() == [0] * count
    n = torch.zeros(beams, dtype=torch.int64, device="cuda")
    history = torch.tensor([0, 3, 5, 29999], dtype=torch.int32, device="cuda")
    for bias, want in ((1.0, [4, 29998, 0, 1]), (-1.0, [0, 1, 2, 3])):
        ids = torch.tensor([4, 29998], dtype=torch.int32, device="cuda")
        values = torch.full((2,), bias, device="cuda")
        rules = rb.LogitAdjust(history=(history[:0], n, n), bias=(ids, values, n, n + 2))
        tokens = rb.beam_select(x[:1], s[:1], 1, 4, rb.LogitAdjust(
            bias=(ids, values, n[:1], n[:1] + 2)))[1]
        assert tokens[0].tolist() == want
        assert rb.beam_select(x, s, beams, 2, rules)[1][0].tolist() == (
            [4, 29998] if bias > 0 else [0, 1])
    tokens = rb.beam_select(x[:1], s[:1], 1, 4, rb.LogitAdjust(
        presence=1.0, history=(history, n[:1], n[:1] + 4)))[1]
    assert tokens[0].tolist() == [1, 2, 4, 6]
    allowed = torch.zeros(beams, v, dtype=torch.bool, device="cuda")
    for at in (9000, 9777, 17000, 29000):
        allowed[0, at] = True
    x[0, 17000] = 2.0
    got = rb.beam_select(x, s, beams, 6, rb.LogitAdjust(mask=rb.pack_mask(allowed)))
    assert got[1][0].tolist() == [17000, 9000, 9777, 29000, -1, -1]
    check_selection(got, totals(np.where(allowed.cpu().numpy(), host_rows(x), -np.inf),
                                np.array([-1.0, -np.inf])), beams, 6)


def test_low_values_and_infinities():
    v, beams = 5000, 2
    x = make_logits(2 * beams, v, F32, 0, seed=1)
    x[0, 100:] = torch.finfo(F32).min   # a mask by the type's lowest value
    x[1, ::2] = -math.inf
    s = torch.tensor([-1.0, -2.0, -math.inf, -math.inf], device="cuda")
    status = rb.new_status()
    got = rb.beam_select(x, s, beams, 6, status=status)
    rb.check(rb.rans_get_status(status))
    check_selection(got, totals(exact_rows(x, None), s.cpu().numpy().astype(float)), beams, 6)
    # what a mask covers, and dead beams' rows, may be anything
    y = x.clone()
    allowed = torch.ones(2 * beams, v, dtype=torch.bool, device="cuda")
    allowed[0, 7], allowed[1, 8] = False, False
    y[0, 7], y[1, 8], y[2], y[3] = math.nan, math.inf, math.nan, math.inf
    mask = rb.LogitAdjust(mask=rb.pack_mask(allowed))
    x[0, 7] = x[1, 8] = -math.inf
    again = rb.beam_select(y, s, beams, 6, mask, status=status)
    rb.check(rb.rans_get_status(status))
    for a, b in zip(again, rb.beam_select(x, s, beams, 6)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bad", ["nan", "inf", "score nan", "score inf", "temperature"])
def test_bad_beams_are_reported_and_left_out(bad):
    v, beams = 20000, 3
    x = make_logits(2 * beams, v, F32, 0, seed=2)
    s = torch.full((2 * beams,), -1.0, device="cuda")
    adjust = None
    if bad == "nan":
        x[4, 19999] = math.nan
    elif bad == "inf":
        x[4, 3] = math.inf
    elif bad == "temperature":
        adjust = rb.LogitAdjust(temperature=torch.ones(6, device="cuda"))
        adjust._keep[-1][4, 3] = 0.0
    else:
        s[4] = math.nan if bad == "score nan" else math.inf
    status = rb.new_status()
    got = rb.beam_select(x, s, beams, 6, adjust, status=status)
    assert rb.rans_get_status(status) == rb.ERR_RANGE
    total = totals(exact_rows(torch.where(x.isfinite(), x, 0.0), None), np.full(6, -1.0))
    total[4] = -np.inf
    check_selection(got, total, beams, 6)


# ------------------------------------------------------------- bookkeeping --
class Plain:
    """One text's bookkeeping from the header's words."""

    def __init__(self, K, capacity, ends, penalty, early, pad):
        self.K, self.capacity, self.ends, self.penalty = K, capacity, ends, penalty
        self.early, self.pad = early, pad
        self.scores = [0.0] + [-math.inf] * (K - 1)
        self.rows = [[] for _ in range(K)]
        self.done, self.over = [], False

    def norm(self, score, n):
        return score if self.penalty == 0 else score / n ** self.penalty

    def advance(self, cands):
        n = len(self.rows[0]) + 1
        kept, old = [], [list(r) for r in self.rows]
        for j, (v, tok, p) in enumerate(cands):
            if tok < 0 or len(kept) == self.K:
                break
            if tok in self.ends:
                if j < self.K:
                    w = self.norm(v, n)
                    if len(self.done) < self.K:
                        self.done.append((w, old[p] + [tok]))
                    else:
                        worst = min(d[0] for d in self.done)
                        at = max(i for i, d in enumerate(self.done) if d[0] == worst)
                        if w > worst:
                            self.done[at] = (w, old[p] + [tok])
                continue
            kept.append((v, tok, p))
        slot, late = {}, []
        for c in kept:
            if c[2] in slot:
                late.append(c)
            else:
                slot[c[2]] = c
        for c in late:
            slot[min(set(range(self.K)) - set(slot))] = c
        over = not kept
        if len(self.done) == self.K:
            worst = min(d[0] for d in self.done)
            reach = self.capacity if self.penalty > 0 else n
            over |= self.early or not (kept and self.norm(kept[0][0], reach) > worst)
        self.parents = [slot[b][2] if b in slot else b for b in range(self.K)]
        self.tokens = [slot[b][1] if b in slot else self.pad for b in range(self.K)]
        self.rows = [old[self.parents[b]] + [self.tokens[b]] if b in slot
                     else old[b] + [self.pad] for b in range(self.K)]
        self.scores = [slot[b][0] if b in slot and not over else -math.inf
                       for b in range(self.K)]
        self.over = over


@pytest.mark.parametrize("K,penalty,early,ends", [
    (1, 0.0, False, [3]), (3, 0.0, True, [3]), (4, 1.0, False, [0, 3]), (5, -0.5, False, [3]),
    (8, 0.6, True, []), (64, 0.0, False, [1])])
def test_search_against_a_plain_one(K, penalty, early, ends):
    """Searches over a small vocabulary, whose candidates the plain one shares."""
    texts, v, steps = 3, 40, 9
    search = rb.BeamSearch(texts, K, steps, ends, penalty, early, pad=39)
    plain = [Plain(K, steps, ends, penalty, early, 39) for _ in range(texts)]
    state = torch.arange(texts * K, device="cuda", dtype=F32)[:, None].repeat(1, 5)
    count = min(K * max(2, 1 + len(ends)), 128)
    g = torch.Generator(device="cuda").manual_seed(K)
    for step in range(steps):
        x = torch.randn(texts * K, v, device="cuda", generator=g) * 2
        cands = [c.cpu() for c in rb.beam_select(x, search.scores, K, count)]
        before = state.clone()
        tokens = search.step(x, states=[state])
        for t, p in enumerate(plain):
            p.advance(list(zip(*(c[t].tolist() for c in cands))))
            rows = slice(t * K, (t + 1) * K)
            assert search.parents[t].tolist() == p.parents
            assert tokens[rows].tolist() == p.tokens
            assert search.scores[rows].tolist() == p.scores
            assert search._history[t, :, :step + 1].tolist() == p.rows
            assert bool(search.over[t]) == p.over
            assert int(search._done_counts[t]) == len(p.done)
            for b, (w, seq) in enumerate(p.done):
                assert float(search._done_scores[t, b]) == pytest.approx(w, rel=1e-6)
                assert search._done_tokens[t, b, :len(seq)].tolist() == seq
                assert int(search._done_lengths[t, b]) == len(seq)
            want = before[rows][torch.tensor(p.parents, device="cuda")]
            assert torch.equal(state[rows], want)
        tok, begin, end = search.window
        assert ((end - begin) == step + 1).all()
    n = min(K, 3)
    tokens, lengths, scores = search.results(n)
    for t, p in enumerate(plain):
        every = p.done + [(p.norm(s, steps), r) for s, r in zip(p.scores, p.rows)
                          if s > -math.inf]
        every.sort(key=lambda d: -d[0])
        for i, (w, seq) in enumerate(every[:n]):
            assert float(scores[t, i]) == pytest.approx(w, rel=1e-5)
            assert int(lengths[t, i]) == len(seq)
            assert tokens[t, i, :len(seq)].tolist() == seq
    # past the capacity nothing changes
    kept = [p.clone() for p in search._parts]
    moved = state.clone()
    search.step(x, states=[state])
    assert torch.equal(state, moved)
    for a, b, in zip(kept, search._parts):
        assert a is kept[2] or torch.equal(a, b)


# ------------------------------------------------------------------ states --
def plain_reorder(x, parents, lengths, axis):
    out = x.clone()
    t, k = parents.shape
    for i in range(t):
        for b in range(k):
            p = int(parents[i, b])
            if p < 0 or p >= k:
                continue
            a, c = x[i * k + p], out[i * k + b]
            if axis is not None:
                n = min(max(int(lengths[i]), 0), x.shape[axis]) if lengths is not None \
                    else x.shape[axis]
                a, c = a.narrow(axis - 1, 0, n), c.narrow(axis - 1, 0, n)
            c.copy_(a)
    return out


@pytest.mark.parametrize("beams", [1, 2, 4, 5, 8, 13, 16, 31, 32, 33, 64])
def test_reorder_any_map(beams):
    """Cycles, one parent for all, rows that stay; several types and axes."""
    texts = 4
    g = torch.Generator().manual_seed(beams)
    parents = torch.randint(0, beams, (texts, beams), generator=g).to(torch.int32)
    parents[0] = torch.randperm(beams, generator=g)
    parents[1] = torch.roll(torch.arange(beams), 1)
    parents[2, ::2] = -1
    lengths = torch.tensor([0, 9, 40, 13], dtype=torch.int32)
    n = texts * beams
    states = [torch.randn(n, 3, 13, 8, generator=g), torch.randn(n, 13, 2, 5, generator=g).half(),
              torch.randint(0, 255, (n, 13, 7), generator=g).to(torch.uint8),
              torch.randint(0, 99, (n, 13), generator=g)]
    axis = [2, 1, 1, 1]
    want = [plain_reorder(x, parents, lengths, a) for x, a in zip(states, axis)]
    up = [x.cuda() for x in states]
    assert rb.reorder_states(up, parents.cuda(), lengths.cuda(), axis) is up
    for a, b in zip(up, want):
        assert torch.equal(a.cpu(), b)
    up = [x.cuda() for x in states]
    rb.reorder_states(up, parents.cuda())
    for a, x in zip(up, states):
        assert torch.equal(a.cpu(), plain_reorder(x, parents, None, None))


def test_reorder_views_and_many():
    """Misaligned bases and strides, halves of one buffer, more states than a
    launch describes; nothing else is written."""
    texts, beams = 3, 4
    n = texts * beams
    parents = torch.tensor([[1, 1, 3, 2], [0, 1, 2, 3], [3, 3, 3, 3]], dtype=torch.int32)
    lengths = torch.tensor([5, 3, 11], dtype=torch.int32)
    both = torch.randn(n, 2, 11, 6)
    flat = torch.randn(1 + n * 50).half()
    odd = flat[1:].view(n, 50)[:, 3:48].view(n, 45)
    many = [torch.randn(n, 11, 3) for _ in range(130)]
    up, flat_up, many_up = both.cuda(), flat.cuda(), [m.cuda() for m in many]
    odd_up = flat_up[1:].view(n, 50)[:, 3:48]
    p, k = parents.cuda(), lengths.cuda()
    rb.reorder_states([up[:, 0], up[:, 1]], p, k, axis=1)
    for h in (0, 1):
        assert torch.equal(up[:, h].cpu(), plain_reorder(both[:, h], parents, lengths, 1))
    rb.reorder_states(odd_up, p)
    want = flat.clone()
    want[1:].view(n, 50)[:, 3:48] = plain_reorder(odd, parents, None, None)
    assert torch.equal(flat_up.cpu(), want)
    rb.reorder_states(many_up, p, k, axis=1)
    for a, m in zip(many_up, many):
        assert torch.equal(a.cpu(), plain_reorder(m, parents, lengths, 1))


def test_reorder_bad_parents_and_refusals():
    x = torch.arange(8.0, device="cuda").view(8, 1)
    parents = torch.tensor([[1, 4, 0, -2], [3, 1, 1, 9]], dtype=torch.int32, device="cuda")
    status = rb.new_status()
    rb.reorder_states(x, parents, status=status)
    assert rb.rans_get_status(status) == rb.ERR_INDEX
    assert x.view(-1).tolist() == [1, 1, 0, 3, 7, 5, 5, 7]
    good = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    y = torch.zeros(8, 6, device="cuda")
    for call in (lambda: rb.reorder_states([y, y], good),
                 lambda: rb.reorder_states([y[:, :4], y[:, 3:]], good),
                 lambda: rb.reorder_states(good.view(8, 1), good)):
        with pytest.raises((rb.RansError, ValueError)):
            call()
    for call in (lambda: rb.reorder_states(y[:7], good),
                 lambda: rb.reorder_states(y, good, axis=2),
                 lambda: rb.reorder_states(y, good, torch.zeros(2, dtype=torch.int32, device="cuda")),
                 lambda: rb.reorder_states(torch.zeros(6, 8, device="cuda").t(), good),
                 lambda: rb.reorder_states(y.cpu(), good),
                 lambda: rb.reorder_states(y, good.long())):
        with pytest.raises(ValueError):
            call()
    rb.reorder_states([y[:, :3], y[:, 3:]], good)


def test_a_search_on_a_head_under_rules():
    """Hidden rows, the 4-bit head, rules over the search's own tokens, beams and
    states: against the same steps in plain form."""
    texts, beams, v, k, steps = 2, 3, 700, 96, 6
    n = texts * beams
    g = torch.Generator(device="cuda").manual_seed(9)
    head = rb.quantize_mxfp4(torch.randn(v, k, device="cuda", generator=g) * 0.4)
    embed = torch.randn(v, k, device="cuda", generator=g)
    search = rb.BeamSearch(texts, beams, steps, ends=[5], length_penalty=0.7)
    state = torch.zeros(n, 2, steps, k, device="cuda")
    hidden = embed[torch.arange(n, device="cuda")]
    lengths = torch.zeros(texts, dtype=torch.int32, device="cuda")
    o = dict(temperature=0.8, repetition=1.2, frequency=0.1, presence=0.2)
    for step in range(steps):
        state[:, :, step] = hidden[:, None]
        lengths += 1
        logits = rb.mxfp4_logits(hidden, head, dtype=F32)
        window = search.window
        rules = rb.LogitAdjust(history=window, **o)
        plain = dict(o, history=tuple(w.cpu().numpy().copy() for w in window))
        total = totals(exact_rows(logits, plain), search.scores.cpu().numpy().astype(float))
        check_selection(rb.beam_select(logits, search.scores, beams, adjust=rules), total, beams,
                        2 * beams)
        before = state.clone()
        tokens = search.step(logits, rules, [state], lengths, axis=2)
        assert torch.equal(state.cpu(), plain_reorder(before.cpu(), search.parents.cpu(),
                                                      lengths.cpu(), 2))
        hidden = embed[tokens.long()] + 0.5 * state[:, 0, step]
    tokens, lengths, scores = search.results(beams)
    assert bool((lengths[:, 0] > 0).all()) and bool((scores[:, 0] > -math.inf).all())
