"""Tokens under a model's logits on the GPU, where the two sides of a call
meet: numbers against rows that hold them, lists and logits at the ends of
float32, streams other than the tensors' own, rows of several tables and rings
that refill, and decoders under offsets that lie."""
import math

import numpy as np
import pytest
import torch

import rans_entropy_coding_b200 as rb
import token_oracle as TO
from test_gpu_tokens import (BF16, F16, F32, TYPES, U, check_adjusted, check_distill, coded,
                             make_adjust, make_logits, numpy_rows, status_ok, teacher)

pytestmark = pytest.mark.gpu


def rows32(n, x):
    return torch.full((n,), x, device="cuda", dtype=F32)


# ------------------------------------------------------------ adjustments --
@pytest.mark.parametrize("T", [0.55, 0.85, 1.1, 1.45, 1.95])
def test_texts_coded_under_a_number_decode_under_rows_of_it(T):
    """A server codes one text under its temperature and decodes it in a batch
    whose rows bring their own."""
    n, v, length = 3, 5000, 12
    x = make_logits(length, v, F32, seed=31)
    tok = torch.randint(0, v, (n, length), device="cuda",
                        generator=torch.Generator("cuda").manual_seed(31))
    c = rb.TokenCoder()
    one = rb.LogitAdjust(temperature=T, repetition=1.1, frequency=0.3, presence=0.2)
    for k in range(n):
        c.add(x, tok[k], one)
    data, offs = c.streams([length] * n)
    many = rb.LogitAdjust(temperature=rows32(n, T), repetition=rows32(n, 1.1),
                          frequency=0.3, presence=rows32(n, 0.2))
    assert torch.equal(rb.adjust_logits(x[:n], one), rb.adjust_logits(x[:n], many))
    every = torch.arange(v, dtype=torch.int32, device="cuda")
    row = x[:1].expand(v, v).contiguous()
    a = rb.token_intervals(row, every, one)
    b = rb.token_intervals(row, every, rb.LogitAdjust(temperature=rows32(v, T)))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.begin(data, offs)
    for t in range(length):
        got = c.step(x[t:t + 1].expand(n, v).contiguous(), many)
        assert got.tolist() == tok[:, t].tolist()
    c.finish()


SLEEP = 50_000_000  # cycles: some 25 ms, far longer than a call takes to arrive


def test_per_row_numbers_on_a_stream_of_their_own():
    """The copy of per-row numbers is waited for by calls on other streams, and
    outlives them, with no synchronisation by the caller."""
    n, v = 6, 3000
    x = make_logits(n, v, F32, seed=37)
    a, _ = make_adjust(n, v, seed=37, per_row=True)
    tok = torch.full((n,), 3, dtype=torch.int32, device="cuda")
    per_row = make_adjust(n, v, seed=37, per_row=True)[1]
    fixed = {k: tuple(torch.from_numpy(t).cuda() for t in per_row[k]) for k in ("history", "bias")}
    fixed["mask"] = torch.from_numpy(per_row["mask"]).cuda()
    numbers = {k: torch.from_numpy(per_row[k]).cuda()
               for k in ("temperature", "repetition", "frequency", "presence")}
    want = [rb.adjust_logits(x, a), *rb.token_intervals(x, tok, a)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    # the copy is late
    torch.cuda._sleep(SLEEP)
    b = rb.LogitAdjust(**fixed, **numbers)
    got = [rb.adjust_logits(x, b, stream=s), *rb.token_intervals(x, tok, b, stream=s)]
    s.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    # the call is late, and what it was given gone
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP)
    b = rb.LogitAdjust(**fixed, **numbers)
    got = rb.adjust_logits(x, b, stream=s)
    del b
    junk = [torch.full((n, 4), 1e6, device="cuda") for _ in range(64)]
    s.synchronize()
    assert torch.equal(got, want[0]) and len(junk) == 64


def test_per_row_numbers_in_a_captured_call():
    """Made before a capture and used in it, on torch's capture stream."""
    n, v = 4, 500
    x = make_logits(n, v, F32, seed=38)
    a, _ = make_adjust(n, v, seed=38, per_row=True)
    out, want = torch.empty_like(x), rb.adjust_logits(x, a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rb.adjust_logits(x, a, out=out)
    g.replay()
    assert torch.equal(out, want)
    # made in the capture: its numbers are read at every replay, on a stream
    # that joins as any other
    t, side = torch.full((n,), 0.5, device="cuda"), torch.cuda.Stream()
    g, other = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(g):
        b = rb.LogitAdjust(temperature=t)
        rb.adjust_logits(x, b, out=out)
        side.wait_stream(torch.cuda.current_stream())
        rb.adjust_logits(x, b, out=other, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for temperature in (2.0, 0.25):
        t.fill_(temperature)
        g.replay()
        want = rb.adjust_logits(x, rb.LogitAdjust(temperature=temperature))
        assert torch.equal(out, want) and torch.equal(other, want)


# ----------------------------------------------------------- distillation --
def both_ways(x, ids, lp, w, T=1.0, tail=True, st=None):
    """(losses, gradient) in one call, and by autograd."""
    ti, tl, tw = (torch.from_numpy(np.ascontiguousarray(a)).cuda() if isinstance(a, np.ndarray)
                  else a for a in (ids, lp, w))
    yield rb.distill_loss_and_grad(x, ti, tl, tw, T, tail, status=st)
    y = x.detach().requires_grad_()
    losses = rb.distill_loss(y, ti, tl, T, tail, status=st)
    (grad,) = torch.autograd.grad(losses, y, tw)
    yield losses.detach(), grad


@pytest.mark.parametrize("shift", [0.0, 64.0, -64.0, 128.0, -128.0, -1024.0, 1e30, -1e30])
@pytest.mark.parametrize("K", [3, 128, 300])
def test_lists_without_a_tail_count_by_their_differences(K, shift):
    """Log probabilities moved as a whole, as unnormalised scores are.  The
    multiples of 2^-10 here stay exact under the shift (to 1024 + 16: 21 bits),
    so moved and unmoved lists are the same teacher; at 1e30 all entries
    are equal."""
    n, v = 4, 3001
    x = make_logits(n, v, F32, 3, seed=32)
    ids, lp = teacher(n, v, K, K, False)
    if K == 3:
        ids[0], lp[0] = -1, -np.inf     # a row without entries
    lp = (np.round(lp * 1024) / 1024).astype(np.float32)
    moved = (lp + np.float32(shift)).astype(np.float32)
    if abs(shift) <= 1024:
        assert np.array_equal(moved - np.float32(shift), lp)
    else:
        lp = np.where(np.isinf(lp), lp, np.float32(0))
    g = np.array([1.0, -0.5, 2.0, 1.0], np.float32)
    st = rb.new_status()
    same = list(both_ways(x, ids, lp, g, tail=False, st=st))
    for a, b in zip(both_ways(x, ids, moved, g, tail=False, st=st), same):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        check_distill(x, ids, lp, 1.0, False, g, *a)
    status_ok(st)


def test_rows_without_entries_add_nothing_at_all():
    """Padding of a batch, whatever its logits are (but for NaN and +inf)."""
    n, v = 4, 900
    x = make_logits(n, v, BF16, 1, seed=33)
    x[2] = -math.inf
    x[3, 5:] = -math.inf
    w = torch.ones(n, device="cuda")
    none = np.full((n, 2), -1, np.int32), np.full((n, 2), -0.5, np.float32)
    gone = np.full((n, 2), 3, np.int32), np.full((n, 2), -np.inf, np.float32)
    for tail in (True, False):
        for ids, lp in (none, gone):
            for losses, grad in both_ways(x, ids, lp, w, tail=tail):
                assert losses.tolist() == [0.0] * n and not bool(grad.any())
                assert not bool(grad.isnan().any())
    # entries that are there, however unlikely, are not absent
    far = np.array([[7, 9]] * n, np.int32), np.full((n, 2), -2000.0, np.float32)
    for losses, grad in both_ways(x[:2], far[0][:2], far[1][:2], w[:2], tail=False):
        check_distill(x[:2], far[0][:2], far[1][:2] + 2000, 1.0, False, np.ones(2), losses, grad)
        assert float(losses.min()) > 0


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("absent", [True, False])
@pytest.mark.parametrize("dtype,low", [(F32, -1e4), (F32, -1e9), (F32, -1e10), (F32, -1e30),
                                       (F32, torch.finfo(F32).min), (F16, -65504.0),
                                       (BF16, -1e10), (BF16, torch.finfo(BF16).min)], ids=str)
def test_masked_students_whose_list_holds_all_that_is_left(dtype, low, absent, tail):
    """A mask written as a low value, on every token outside the list (`absent`:
    but for the ids of entries that are absent): the mass there is 0 in
    any type, and its logarithm finite."""
    n, v, K, T = 3, 3001, 40, 2.0
    x = make_logits(n, v, dtype, 3, seed=34)
    ids, lp = teacher(n, v, K, 9, tail)
    out = torch.ones(n, v, dtype=torch.bool, device="cuda")
    for r in range(n):
        some = (ids[r] >= 0) & (absent | (lp[r] > -np.inf))
        out[r, torch.from_numpy(ids[r][some].astype(np.int64)).cuda()] = False
    x[out] = low
    x[0] = low                          # (row 0 has no entries: all equal)
    x[0, 5] = 1.0
    g = np.array([1.0, -0.5, 2.0], np.float32)

    def lse(z):
        return z.max() + math.log(np.exp(z - z.max()).sum())

    for losses, grad in both_ways(x, ids, lp, g, T, tail):
        if not tail:
            check_distill(x, ids, lp, T, tail, g, losses, grad)
            continue
        rows, eps = numpy_rows(x).astype(np.float64), torch.finfo(grad.dtype).eps
        G = grad.double().cpu().numpy()
        assert float(losses[0]) == 0.0 and not G[0].any()
        for r in range(1, n):
            # in logarithms: the tail's mass may have no double
            keep = (ids[r] >= 0) & (lp[r] > -np.inf)
            p, z = np.exp(lp[r][keep].astype(np.float64)), rows[r] / T
            others = np.ones(v, bool)
            others[ids[r][keep]] = False
            lz, lr, pt = lse(z), lse(z[others]), 1 - p.sum()
            want = (p * (np.log(p) - z[ids[r][keep]] + lz)).sum() + pt * (math.log(pt) + lz - lr)
            # float32's log probabilities, the loss's own rounding
            assert abs(float(losses[r]) - want) <= 1e-5 + 2 * U * abs(want)
            dz = np.exp(z - lz)
            dz[ids[r][keep]] -= p
            share = np.exp(z[others] - z[others].max())  # (lr has no room for log v at 1e30)
            dz[others] -= pt * share / share.sum()
            dz *= g[r] / T
            tol = 1e-5 * abs(g[r]) + np.abs(dz) * eps
            assert (np.abs(G[r] - dz) <= tol).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_students_at_the_ends_of_their_type(dtype):
    """Logits of both signs up to the largest, -inf rows, small temperatures:
    against 64 bits, where every sum of these is held."""
    v = 2000
    x = make_logits(7, v, dtype, 1, seed=35)
    top = torch.finfo(dtype).max
    x[0, 100:] = -top
    x[1, ::2], x[1, 7] = top, -math.inf
    x[2] = top
    x[3] = -top
    x[4, :900], x[4, 900:] = -top, -top / 2
    x[5] = -math.inf
    ids = np.tile(np.array([[7, 9, 1500]], np.int32), (7, 1))
    lp = np.log(np.tile(np.array([[0.25, 0.125, 0.5]], np.float32), (7, 1)))
    g = np.ones(7, np.float32)
    for T in (1.0, 0.01, 4.0):              # (with reciprocals that float32 holds)
        for tail in (True, False):
            for losses, grad in both_ways(x, ids, lp, g, T, tail):
                assert bool(losses[5].isnan()) and bool(grad[5].isnan().all())
                assert losses[1] == math.inf        # token 7 has no mass at all
                assert bool(grad[:5].isfinite().all())
                for r in (0, 2, 3, 4, 6):
                    one = slice(r, r + 1)
                    if TO.distill(numpy_rows(x)[r], ids[r], lp[r], 1.0 / T, tail)[0] > 3.4e38:
                        assert losses[r] == math.inf
                    else:
                        check_distill(x[one], ids[one], lp[one], T, tail, g[one], losses[one],
                                      grad[one])
    # the whole list far below the rest: the listed have no mass, the others all
    y = make_logits(1, v, dtype, 1, seed=36)
    y[0, torch.tensor([7, 9, 1500], device="cuda")] = -1e4
    for losses, grad in both_ways(y, ids[:1], lp[:1], g[:1]):
        check_distill(y, ids[:1], lp[:1], 1.0, True, g[:1], losses, grad)


@pytest.mark.parametrize("shift", [-20000.0, 20000.0, 1e7])
def test_distillation_counts_differences_to_their_last_bit(shift):
    """Logits far from zero: their differences are exact, so the error is
    that of rows near zero."""
    n, v = 3, 5000
    x = make_logits(n, v, F32, seed=16) + shift
    x[1, 2500:] -= 30000.0                 # a row whose ends lie far apart
    x[2, :2500] -= 30000.0
    ids, lp = teacher(n, v, 30, 7, True)
    g = np.array([1.0, -0.5, 2.0], np.float32)
    for losses, grad in both_ways(x, ids, lp, g):
        check_distill(x, ids, lp, 1.0, True, g, losses, grad)


def test_a_backward_pass_whose_logits_were_written_over_raises():
    n, v = 3, 200
    x = make_logits(n, v, F32, seed=39).contiguous()
    ids, lp = (torch.from_numpy(t).cuda() for t in teacher(n, v, 5, 1, True))
    w = torch.ones(n, device="cuda")
    for write in (lambda z: rb.adjust_logits(z, rb.LogitAdjust(temperature=0.5), out=z),
                  lambda z: rb.distill_loss_and_grad(z, ids, lp, w, grad=z)):
        y = x.clone().requires_grad_()
        z = y * 1.0
        loss = rb.distill_loss(z, ids, lp).sum()
        write(z.detach())
        with pytest.raises(RuntimeError, match="inplace operation"):
            loss.backward()
    # what is not saved may be written to
    loss = rb.distill_loss(y, ids, lp).sum()
    rb.adjust_logits(y.detach(), None, out=torch.empty_like(x))
    loss.backward()
    with torch.inference_mode():
        z = x.clone()
        rb.adjust_logits(z, None, out=z)
    rb.adjust_logits(z, None, out=z)
    assert torch.equal(z, x)


# ------------------------------------------------------- the coder object --
def test_a_coder_starts_afresh_after_an_error():
    x, tok, (data, offs) = coded(1, 60, 4, seed=40)
    c = rb.TokenCoder()
    with pytest.raises(RuntimeError):
        c.step(x[:1])
    with pytest.raises(RuntimeError):
        c.finish()
    c.begin(data[:4], offs)             # streams that are not there, given up
    c.begin(data, offs)
    for t in range(4):
        assert int(c.step(x[t:t + 1])) == int(tok[0, t])
    c.finish()
    c.begin(data[:4], offs)             # nor do they spoil texts that are coded
    again, _ = c.add(x, tok[0]).streams([4])
    assert torch.equal(again, data)
    with pytest.raises(rb.RansError):   # and an error is told once
        c.finish()
    c.add(x, torch.tensor([1, 2, 60, 3]))
    with pytest.raises(rb.RansError):
        c.streams([4])
    again, _ = c.add(x, tok[0]).streams([4])
    assert torch.equal(again, data)
    c.add(x[:1], tok[0, :1])
    with pytest.raises(ValueError):     # (the call's own mistake drops nothing)
        c.streams([4])
    again, _ = c.add(x[1:], tok[0, 1:]).streams([4])
    assert torch.equal(again, data)


def test_wide_token_ids_are_refused():
    x = make_logits(3, 50, F32, seed=41)
    for bad in (2**32 + 5, 2**31, -2**32 + 7):
        c = rb.TokenCoder()
        c.add(x, torch.tensor([1, bad, 2], device="cuda"))
        with pytest.raises(rb.RansError) as e:
            c.streams([3])
        assert e.value.status == rb.ERR_INDEX


# ------------------------------------------------- decoders that are lied to --
def test_a_refill_is_read_inside_its_stream_or_not_at_all():
    """Every row needs a word, and whether its offsets allow one is decided on
    the host: the oracle's step where they do; else no token, the state as it
    was, and an error."""
    x, _, (data, offs) = coded(4, 50, 3)
    st = rb.new_status()
    rows = x[:4].contiguous() if x.shape[0] >= 4 else x[:1].expand(4, 50).contiguous()
    bounds = [TO.bounds(r, {}, 0) for r in numpy_rows(rows)]
    words = np.frombuffer(data.cpu().numpy().tobytes(), np.uint32)
    total, seen = data.numel(), set()
    for lie in (offs.tolist(), [0, 10, 20, 30, 40], [64, 48, 32, 16, 0], [0] * 4 + [1 << 40],
                [0] * 5, [-8, 16, 32, 48, 64], [0, total, total, total, total + 4],
                [0, total, 0, total, 0], [total - 12, total, total + 4, 8, total]):
        for taken in (2, 0, 1 << 40, (1 << 62) - 1):
            states = torch.tensor([[(1 << 31) + 3 * r, taken] for r in range(4)], device="cuda")
            tok, new = rb.decode_tokens(rows, data, torch.tensor(lie, device="cuda"), states,
                                        status=st)
            ok = []
            for r in range(4):
                off, lim = lie[r] % (1 << 64), lie[r + 1] % (1 << 64)
                ok.append(off % 4 == 0 and off <= lim <= total and taken < (lim - off) // 4)
                if not ok[r]:
                    assert int(tok[r]) == -1 and torch.equal(new[r], states[r])
                    continue
                b, slot = bounds[r], 3 * r
                t = int(np.searchsorted(np.array(b), slot, side="right")) - 1
                y = (b[t + 1] - b[t]) * ((1 << 31) >> 24) + slot - b[t]
                assert y < 1 << 31 and int(tok[r]) == t
                assert new[r].tolist() == [y << 32 | int(words[off // 4 + taken]), taken + 1]
            seen.update(ok)
            assert rb.rans_get_status(st) == (rb.OK if all(ok) else rb.ERR_CORRUPT)
    assert seen == {True, False}


# ------------------------------------------ rows of several tables and tiles --
def check_token_rows(x, a, o, sample, seed):
    """Adjusted logits, intervals and decoding steps of some of the rows."""
    n, rng, st = x.shape[0], np.random.default_rng(seed), rb.new_status()
    rows = {r: numpy_rows(x[r:r + 1])[0] for r in sample}
    b = {r: TO.bounds(rows[r], o, r) for r in sample}
    tok = np.full(n, -1, np.int32)
    slots = rng.integers(0, 1 << 24, n)
    for r in sample:
        alive = np.flatnonzero(np.diff(b[r]))
        tok[r] = alive[-1 - len(alive) // 7] if r % 2 else rng.choice(alive)
    s, f = rb.token_intervals(x, torch.from_numpy(tok).cuda(), a, status=st)
    states = torch.stack([torch.from_numpy(slots).cuda() + (1 << 62),
                          torch.full((n,), 2, device="cuda")], 1)
    got, _ = rb.decode_tokens(x, torch.zeros(8 * n, dtype=torch.uint8, device="cuda"),
                              torch.arange(n + 1, device="cuda") * 8, states, a, status=st)
    out = rb.adjust_logits(x, a, dtype=F32)
    for r in sample:
        assert int(s[r]) == b[r][tok[r]] and int(f[r]) == b[r][tok[r] + 1] - b[r][tok[r]]
        assert int(got[r]) == int(np.searchsorted(np.array(b[r]), slots[r], side="right")) - 1
        want, err = TO.adjust(rows[r], o, r)
        z, dead = out[r].double().cpu().numpy(), np.isinf(want)
        assert np.array_equal(z[dead], want[dead])
        assert (np.abs(z[~dead] - want[~dead]) <=
                err[~dead] + U * (np.abs(want[~dead]) + err[~dead]) + 2.0 ** -149).all()
    status_ok(st)
    y = x.clone()
    assert torch.equal(rb.adjust_logits(y, a, out=y), rb.adjust_logits(x, a))


@pytest.mark.parametrize("dtype,v,pad", [(BF16, 131072, 0), (F16, 131071, 2), (F32, 150001, 1)],
                         ids=str)
def test_rows_of_many_tables_in_one_block(dtype, v, pad):
    """Enough rows that a block has one to itself, histories of more distinct
    tokens than a hash takes: a table for every 8,192 tokens, walked twice, and
    once more for the decoded token."""
    n = 150
    x = make_logits(n, v, dtype, pad, seed=42, offset=pad)
    a, o = make_adjust(n, v, seed=42, long=120000)
    assert np.unique(o["history"][0]).size > 50000
    check_token_rows(x, a, o, [0, 1, 2, 71, 149], 42)


@pytest.mark.parametrize("parts", [dict(history=False, bias=False), dict(bias=False), dict()],
                         ids=str)
@pytest.mark.parametrize("dtype,v,n", [(BF16, 150001, 900), (F32, 140000, 150),
                                       (F16, rb.MAX_VOCAB, 150)], ids=str)
def test_masks_past_a_tables_span(dtype, v, n, parts):
    """More tokens than a table's bitmap and hash cover, in one block: the mask
    alone, and with few touched tokens.  (At 900 rows adjust_logits has one
    block a row too.)"""
    x = make_logits(n, v, dtype, v % 2, seed=43)
    a, o = make_adjust(n, v, seed=43, **parts)
    check_token_rows(x, a, o, [1, n - 2], 43)


def check_rows(x, ids, lp, T, tail, g, losses, grad, sample, rescales):
    """As check_distill, with the 2^-22 of each exponential that a sum is
    rescaled by when its maximum rises (`rescales` times at most)."""
    L, G, inv, fi = (losses.double().cpu().numpy(), grad.cpu(), 1.0 / T, torch.finfo(grad.dtype))
    v = x.shape[1]
    for r in sample:
        row = numpy_rows(x[r:r + 1])[0]
        want, dz, parts = TO.distill(row, ids[r], lp[r], inv, tail)
        arg = np.abs(row.astype(np.float64) - row.max()) * inv
        eps = 2.0 ** -22 * (1 + rescales) + U * (3 * 0.7 * (math.log2(v) + 1) + v / 512 + 20)
        assert abs(L[r] - want) <= 2 * eps + U * abs(want), (r, L[r], want)
        tol = abs(g[r]) * parts * (2 * eps + U * (8 + 4 * arg)) + \
            np.abs(dz * g[r]) * (fi.eps / 2 + 2 * U) + fi.smallest_normal * fi.eps / 2 + 2.0 ** -126
        assert (np.abs(G[r].double().numpy() - dz * g[r]) <= tol).all(), r


@pytest.mark.parametrize("n", [3, 300])
@pytest.mark.parametrize("dtype,v,pad", [(BF16, 131072, 0), (F16, 150001, 3), (F32, 150001, 0),
                                         (F32, 131072, 5)], ids=str)
def test_distillation_of_rows_longer_than_their_ring(dtype, v, pad, n):
    """Many tiles a warp: stages that are filled again while others are read, in
    both walks, with one block a row (300) and several (3); in place, where
    later tiles are on their way while earlier ones are written.  Row 2's logits
    rise, so that every tile raises the maximum."""
    T, tail, K = 1.5, n > 3, 60 if n > 3 else 300
    x = make_logits(n, v, dtype, pad, seed=44, offset=pad)
    x[2] = x[2].float().sort().values.to(dtype)
    ids, lp = teacher(n, v, K, 44, tail)
    g = np.random.default_rng(44).uniform(0.5, 2.0, n).astype(np.float32)
    if dtype == F16:
        g *= 1024                       # (gradients above the type's smallest)
    sample = sorted({0, 1, 2, n // 2, n - 1})
    st = rb.new_status()
    # a warp's tiles are kStep tokens apart
    rescales = -(-v // (8 * 32 * 4 * (16 // x.element_size())))
    both = list(both_ways(x, ids, lp, g, T, tail, st))
    for losses, grad in both:
        check_rows(x, ids, lp, T, tail, g, losses, grad, sample, rescales)
    ti, tl, tg = (torch.from_numpy(t).cuda() for t in (ids, lp, g))
    wide = torch.empty(n * (v + 16), device="cuda", dtype=dtype).view(n, v + 16)[:, 8:v + 8]
    y = wide.copy_(x) if pad == 0 else x.clone()
    losses, _ = rb.distill_loss_and_grad(y, ti, tl, tg, T, tail, grad=y, status=st)
    # (a clone of padded rows is packed: other vectors, the same to rounding)
    check_rows(x, ids, lp, T, tail, g, losses, y, sample, rescales)
    y = make_logits(n, v, dtype, pad, seed=44, offset=pad)
    y[2] = x[2]
    losses, _ = rb.distill_loss_and_grad(y, ti, tl, tg, T, tail, grad=y, status=st)
    assert torch.equal(losses, both[0][0]) and torch.equal(y, both[0][1])
    status_ok(st)


@pytest.mark.parametrize("n", [2, 300])
def test_distillation_memory_that_may_be_shared(n):
    """Losses over the weights that they were asked for with; lists that lie
    between a result's rows."""
    v, K = 20011, 8
    x = make_logits(n, v, F32, seed=45)
    ids, lp = teacher(n, v, K, 45, True)
    ti, tl = torch.from_numpy(ids).cuda(), torch.from_numpy(lp).cuda()
    w = torch.linspace(0.5, 2.0, n, device="cuda")
    st = rb.new_status()
    want, grad = rb.distill_loss_and_grad(x, ti, tl, w, status=st)
    out, again = w.clone(), torch.empty_like(grad)
    rb.check(rb.rans_distill(x, ti, tl, 1.0, True, out, out, again, st))
    assert torch.equal(out, want) and torch.equal(again, grad)
    wide = torch.zeros(n, v + 2 * n * K + 1, device="cuda")
    wide[0, v:v + n * K].view(torch.int32).copy_(ti.view(-1))
    wide[1, v + n * K:v + 2 * n * K].copy_(tl.view(-1))
    got, g = rb.distill_loss_and_grad(x, wide[0, v:v + n * K].view(torch.int32).view(n, K),
                                      wide[1, v + n * K:v + 2 * n * K].view(n, K), w,
                                      grad=wide[:, :v], status=st)
    assert torch.equal(got, want) and torch.equal(g, grad)
    status_ok(st)


@pytest.mark.parametrize("dtype,n", [(BF16, 3), (BF16, 300), (F32, 2)], ids=str)
def test_distillation_at_its_largest_sizes(dtype, n):
    """The largest vocabulary and the longest list, in one block a row and in
    several: the most shared memory that a launch asks for."""
    v, K, T = rb.MAX_VOCAB, rb.MAX_TOP, 0.8
    x = make_logits(n, v, dtype, 0, seed=46)
    few = min(n, 4)
    ids, lp = teacher(few, v, K, 46, True)
    ids, lp = (np.concatenate([a] * (-(-n // few)))[:n] for a in (ids, lp))
    g = np.linspace(0.5, 2.0, n).astype(np.float32)
    st = rb.new_status()
    rescales = -(-v // (8 * 32 * 4 * (16 // x.element_size())))
    for losses, grad in both_ways(x, ids, lp, g, T, True, st):
        check_rows(x, ids, lp, T, True, g, losses, grad, sorted({1, n // 2, n - 1}), rescales)
    status_ok(st)
