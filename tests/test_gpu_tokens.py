"""Tokens under a model's logits on the GPU: logit adjustment, intervals,
streams, decoding steps and distillation against plain versions in 64 bits
(tests/token_oracle.py), at the sizes and masks where they can go wrong."""
import math

import numpy as np
import pytest
import torch

import rans_entropy_coding_b200 as rb
import token_oracle as TO

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
U = 2.0 ** -24
# one token, around a vector, around a word of mask bits, around a span of the
# touched-token tables, and the largest vocabulary of a block's first pass
SIZES = [(1, 0), (7, 1), (8, 0), (33, 0), (1000, 3), (8185, 7), (8193, 0), (20011, 5)]


def numpy_rows(x):
    return x.float().cpu().numpy()


def make_logits(n, v, dtype, pad=0, seed=0, offset=0):
    """Rows inside a wider, possibly misaligned buffer whose other elements are
    NaN: nothing outside the rows may be used."""
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + v)
    flat = torch.full((offset + n * (v + pad),), math.nan, device="cuda", dtype=dtype)
    x = flat[offset:].view(n, v + pad)[:, :v]
    body = torch.randn(n, v, device="cuda", generator=g) * 3
    few = torch.randint(0, v, (n, 4), device="cuda", generator=g)
    body.scatter_add_(1, few, torch.rand(n, 4, device="cuda", generator=g) * 9)
    x.copy_(body)
    return x


def make_adjust(n, v, seed, history=True, bias=True, mask=True, per_row=False, long=700):
    """(LogitAdjust, the oracle's dict): windows that overlap, repeat ids, are
    empty, run past the arrays' ends or hold ids outside the vocabulary.
    `long`: the history array's length (row 1's window is all of it)."""
    rng = np.random.default_rng(seed)
    o = dict(temperature=0.8, repetition=1.25, frequency=0.1, presence=0.35)
    if per_row:
        o = dict(temperature=rng.uniform(0.5, 1.5, n).astype(np.float32),
                 repetition=rng.uniform(0.8, 1.5, n).astype(np.float32),
                 frequency=rng.uniform(-0.2, 0.5, n).astype(np.float32),
                 presence=rng.uniform(-0.2, 0.5, n).astype(np.float32))

    def spans(total):
        b = rng.integers(-3, total, n)
        e = b + rng.integers(0, total, n)
        e[0] = b[0]                         # an empty window
        if n > 1:
            b[1], e[1] = 0, total + 5       # all of it and past its end
        if n > 2:
            b[2], e[2] = total, total - 2   # end before begin
        return b.astype(np.int64), e.astype(np.int64)

    if history:
        toks = np.minimum(rng.integers(-2, v + 2, long), rng.integers(0, v + 2, long))
        o["history"] = (toks.astype(np.int32), *spans(long))
    if bias:
        ids = rng.integers(-1, v + 1, 60).astype(np.int32)
        o["bias"] = (ids, rng.normal(0, 3, 60).astype(np.float32), *spans(60))
    if mask:
        m = rng.integers(-2**31, 2**31, (n, (v + 31) // 32)).astype(np.int32)
        m[:, 0] |= 1
        o["mask"] = m

    def up(x):
        return torch.from_numpy(x).cuda() if isinstance(x, np.ndarray) else x

    kw = {k: tuple(up(t) for t in x) if isinstance(x, tuple) else up(x) for k, x in o.items()}
    return rb.LogitAdjust(**kw), o


def check_adjusted(out, x, o, n):
    rows, got = numpy_rows(x), out.float().cpu().numpy().astype(np.float64)
    eps = torch.finfo(out.dtype).eps / 2
    tiny = torch.finfo(out.dtype).smallest_normal * eps
    for r in range(n):
        want, err = TO.adjust(rows[r], o, r)
        same = np.isinf(want)
        assert np.array_equal(got[r][same], want[same])
        tol = err + eps * (np.abs(want) + err) + tiny
        assert (np.abs(got[r] - want)[~same] <= tol[~same]).all(), r


# ------------------------------------------------------------- adjustment --
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v,pad", SIZES)
def test_adjust(v, pad, dtype):
    n = 5
    x = make_logits(n, v, dtype, pad, offset=pad)
    for parts in (dict(), dict(mask=False), dict(history=False, bias=False),
                  dict(history=False, per_row=True), dict(bias=False, mask=False)):
        a, o = make_adjust(n, v, seed=v + len(parts), **parts)
        check_adjusted(rb.adjust_logits(x, a), x, o, n)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("out_dtype", TYPES, ids=str)
def test_adjust_into_other_types_and_strides(dtype, out_dtype):
    n, v = 4, 1001
    x = make_logits(n, v, dtype, 3)
    a, o = make_adjust(n, v, seed=5)
    wide = torch.full((n, v + 6), 77.0, device="cuda", dtype=out_dtype)
    rb.adjust_logits(x, a, out=wide[:, 1:v + 1])
    check_adjusted(wide[:, 1:v + 1], x, o, n)
    assert bool((wide[:, 0] == 77).all()) and bool((wide[:, v + 1:] == 77).all())
    assert torch.equal(rb.adjust_logits(x, a, dtype=out_dtype), wide[:, 1:v + 1])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_adjust_in_place_and_neutral(dtype):
    n, v = 3, 9001
    x = make_logits(n, v, dtype, 1)
    a, _ = make_adjust(n, v, seed=6)
    want = rb.adjust_logits(x, a)
    y = x.clone()
    assert rb.adjust_logits(y, a, out=y) is y and torch.equal(y, want)
    assert torch.equal(rb.adjust_logits(x, None), x)
    assert torch.equal(rb.adjust_logits(x, rb.LogitAdjust()), x)
    a, _ = make_adjust(n, v, seed=6, long=30000)     # too many touched tokens for a hash
    want = rb.adjust_logits(x, a)
    y = x.clone()
    rb.adjust_logits(y, a, out=y)
    assert torch.equal(y, want)
    # penalties that are neutral change no bit
    (h, b, e) = torch.arange(50, dtype=torch.int32, device="cuda"), *torch.tensor(
        [[0] * n, [50] * n], device="cuda")
    assert torch.equal(rb.adjust_logits(x, rb.LogitAdjust(history=(h, b, e))), x)


def test_adjust_masks_hide_anything_and_may_hide_everything():
    v = 70
    x = make_logits(4, v, BF16)
    x[:, 5], x[:, 6], x[:, 7] = math.nan, math.inf, -math.inf
    x[:, 8] = torch.finfo(BF16).min
    ok = torch.ones(4, v, dtype=torch.bool, device="cuda")
    ok[0, 5] = ok[0, 6] = False
    ok[1] = False
    ok[2] = False
    ok[2, 69] = True
    out = rb.adjust_logits(x, rb.LogitAdjust(mask=rb.pack_mask(ok)))
    assert not bool(out[0].isnan().any()) and not bool((out[0] == math.inf).any())
    assert bool((out[1] == -math.inf).all())
    assert int((out[2] > -math.inf).sum()) == 1 and out[2, 69] == x[2, 69]
    assert bool(out[3, 5].isnan()) and out[3, 6] == math.inf and out[3, 7] == -math.inf
    assert out[3, 8] == x[3, 8]
    shared = rb.adjust_logits(x, rb.LogitAdjust(mask=rb.pack_mask(ok[0])))
    assert torch.equal(shared[0], out[0]) and bool((shared[:, 5] == -math.inf).all())


# -------------------------------------------------------------- intervals --
def status_ok(st):
    assert rb.rans_get_status(st) == rb.OK


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v,pad", SIZES)
def test_intervals(v, pad, dtype):
    n = 6
    x = make_logits(n, v, dtype, pad, seed=2, offset=pad)
    rows, rng = numpy_rows(x), np.random.default_rng(v)
    st = rb.new_status()
    for parts in (None, dict(), dict(mask=False, per_row=True), dict(history=False, bias=False)):
        a, o = (None, {}) if parts is None else make_adjust(n, v, seed=v, **parts)
        want = [TO.bounds(rows[r], o, r) for r in range(n)]
        tok = np.array([rng.choice(np.flatnonzero(np.diff(b))) for b in want], np.int32)
        tok[0] = np.flatnonzero(np.diff(want[0]))[0]        # the first and the last alive one
        tok[1] = np.flatnonzero(np.diff(want[1]))[-1]
        s, f = rb.token_intervals(x, torch.from_numpy(tok).cuda(), a, status=st)
        assert s.tolist() == [b[t] for b, t in zip(want, tok)]
        assert f.tolist() == [b[t + 1] - b[t] for b, t in zip(want, tok)]
    status_ok(st)


@pytest.mark.parametrize("v", [1, 5, 700])
def test_intervals_of_all_tokens_tile_the_range(v):
    x = make_logits(1, v, BF16, seed=3)
    every = x.expand(v, v).contiguous()
    st = rb.new_status()
    s, f = rb.token_intervals(every, torch.arange(v, dtype=torch.int32, device="cuda"), status=st)
    ends = (s + f).tolist()
    assert s.tolist() == [0] + ends[:-1] and ends[-1] == 1 << 24 and int(f.min()) >= 1
    status_ok(st)


def test_interval_of_a_row_does_not_depend_on_its_batch():
    n, v = 40, 30011
    x = make_logits(n, v, F16, seed=4, pad=1)
    a, o = make_adjust(n, v, seed=9)
    st = rb.new_status()
    b = [TO.bounds(r, o, i) for i, r in enumerate(numpy_rows(x))]
    tok = torch.tensor([int(np.flatnonzero(np.diff(q))[-1 - i]) for i, q in enumerate(b)],
                       dtype=torch.int32, device="cuda")
    s, f = rb.token_intervals(x, tok, a, status=st)
    assert s.tolist() == [q[t] for q, t in zip(b, tok.tolist())]
    for i in (0, 17, 39):
        one = {k: (w if not isinstance(w, tuple) else (*w[:-2], w[-2][i:i + 1], w[-1][i:i + 1]))
               for k, w in o.items()}
        one["mask"] = o["mask"][i:i + 1]
        kw = {k: tuple(torch.from_numpy(t).cuda() for t in w) if isinstance(w, tuple) else
              torch.from_numpy(w).cuda() if isinstance(w, np.ndarray) else w
              for k, w in one.items()}
        s1, f1 = rb.token_intervals(x[i:i + 1].clone(), tok[i:i + 1], rb.LogitAdjust(**kw),
                                    status=st)
        assert int(s1) == int(s[i]) and int(f1) == int(f[i])
    status_ok(st)


def test_intervals_errors_and_skipped_rows():
    v = 100
    st = rb.new_status()

    def one(row, token, a=None):
        x = row[None].cuda()
        s = torch.full((1,), 7, dtype=torch.int32, device="cuda")
        f = s.clone()
        rb.token_intervals(x, torch.tensor([token], dtype=torch.int32, device="cuda"), a, s, f, st)
        return int(s), int(f), rb.rans_get_status(st)

    base = torch.randn(v, generator=torch.Generator().manual_seed(1))
    assert one(base, -1) == (7, 7, rb.OK)
    assert one(base, v) == (0, 0, rb.ERR_INDEX)
    assert one(base, -2) == (0, 0, rb.ERR_INDEX)
    for bad in (math.nan, math.inf, 3.4e38):
        row = base.clone()
        row[3] = bad
        assert one(row, 5) == (0, 0, rb.ERR_RANGE)
        hidden = torch.ones(v, dtype=torch.bool, device="cuda")
        hidden[3] = False
        s, f, code = one(row, 5, rb.LogitAdjust(mask=rb.pack_mask(hidden)))
        assert code == rb.OK and f > 0
    row = base.clone()
    row[5] = -math.inf
    assert one(row, 5) == (0, 0, rb.ERR_ZERO_FREQ)
    assert one(torch.full((v,), -math.inf), 5) == (0, 0, rb.ERR_ZERO_FREQ)
    none = torch.zeros(v, dtype=torch.bool, device="cuda")
    assert one(base, 5, rb.LogitAdjust(mask=rb.pack_mask(none))) == (0, 0, rb.ERR_ZERO_FREQ)
    # the type's lowest value is finite: a token of weight 0, still codable
    row = base.clone()
    row[5] = torch.finfo(F32).min
    b = TO.bounds(row.numpy(), {}, 0)
    assert one(row, 5) == (b[5], 1, rb.OK)
    # per-row parameters that are no temperature
    for bad in (0.0, -1.0, math.nan, math.inf):
        p = rb.LogitAdjust(temperature=torch.full((1,), bad, device="cuda"))
        assert one(base, 5, p) == (0, 0, rb.ERR_RANGE)
    # and where a row has nothing else, its tokens weigh the same
    low = torch.full((v,), torch.finfo(F32).min)
    low[0] = -math.inf
    b = TO.bounds(low.numpy(), {}, 0)
    assert one(low, 5) == (b[5], b[6] - b[5], rb.OK)


@pytest.mark.parametrize("long", [1700, 6000, 30000])
@pytest.mark.parametrize("v", [40, 1000, 20011])
def test_long_histories(v, long):
    """Windows full of repeats in a small vocabulary, and with more touched
    tokens than a hash table takes (3,584 in a block's share of the row) in a
    large one."""
    n = 4
    x = make_logits(n, v, BF16, 1, seed=14)
    a, o = make_adjust(n, v, seed=long + v, long=long)
    check_adjusted(rb.adjust_logits(x, a, dtype=F32), x, o, n)
    rng, st = np.random.default_rng(v), rb.new_status()
    b = [TO.bounds(row, o, r) for r, row in enumerate(numpy_rows(x))]
    tok = np.array([rng.choice(np.flatnonzero(np.diff(q))) for q in b], np.int32)
    s, f = rb.token_intervals(x, torch.from_numpy(tok).cuda(), a, status=st)
    assert s.tolist() == [q[t] for q, t in zip(b, tok)]
    assert f.tolist() == [q[t + 1] - q[t] for q, t in zip(b, tok)]
    slots = rng.integers(0, 1 << 24, n)
    states = torch.tensor([[(1 << 62) + int(k), 2] for k in slots], device="cuda")
    tok, _ = rb.decode_tokens(x, torch.zeros(8 * n, dtype=torch.uint8, device="cuda"),
                              torch.arange(n + 1, device="cuda") * 8, states, a, status=st)
    assert tok.tolist() == [int(np.searchsorted(q, k, side="right")) - 1
                            for q, k in zip(b, slots)]
    status_ok(st)


@pytest.mark.parametrize("dtype,v,n", [(F16, 150001, 160), (BF16, 131072, 150), (F32, 70003, 75),
                                       (BF16, rb.MAX_VOCAB, 3)])
def test_many_rows_and_large_vocabularies(dtype, v, n):
    """The split of a row over blocks follows the number of rows: the same rows
    in another batch give the same intervals, tokens and states."""
    x = make_logits(n, v, dtype, 3 if v % 2 else 0, seed=15)
    a, o = make_adjust(n, v, seed=15, mask=False)
    st = rb.new_status()
    g = torch.Generator("cuda").manual_seed(1)
    tok = torch.randint(0, v, (n,), device="cuda", generator=g).to(torch.int32)
    words = torch.randint(-2**31, 2**31, (4 * n,), device="cuda", generator=g).to(torch.int32)
    data, offs = words.view(torch.uint8), torch.arange(n + 1, device="cuda") * 16
    states = torch.stack([torch.randint(1 << 31, 1 << 55, (n,), device="cuda", generator=g),
                          torch.full((n,), 2, device="cuda")], 1)

    def one(r, adj):
        p = {k: (tuple(torch.from_numpy(q).cuda() for q in (*w[:-2], w[-2][r:r + 1],
                                                             w[-1][r:r + 1]))
                 if isinstance(w, tuple) else w) for k, w in o.items()}
        return rb.LogitAdjust(**p) if adj else None

    for adj in (None, a):
        s, f = rb.token_intervals(x, tok, adj, status=st)
        t, new = rb.decode_tokens(x, data, offs, states, adj, status=st)
        for r in sorted({0, 1, n // 2, n - 1}):
            s1, f1 = rb.token_intervals(x[r:r + 1], tok[r:r + 1], one(r, adj), status=st)
            assert (int(s1), int(f1)) == (int(s[r]), int(f[r]))
            t1, n1 = rb.decode_tokens(x[r:r + 1], data, offs[r:r + 2], states[r:r + 1],
                                      one(r, adj), status=st)
            assert int(t1) == int(t[r]) and torch.equal(n1[0], new[r])
        r = n // 2
        b = TO.bounds(numpy_rows(x[r:r + 1])[0], {} if adj is None else o, r)
        assert int(s[r]) == b[int(tok[r])]
        slot = int(states[r, 0]) & ((1 << 24) - 1)
        assert int(t[r]) == int(np.searchsorted(b, slot, side="right")) - 1
    status_ok(st)


# ---------------------------------------------------------------- streams --
def random_intervals(n, rng):
    f = np.minimum(1 << rng.integers(0, 25, n), (1 << 24) - rng.integers(0, 2, n) * 12345)
    f = np.maximum(f - rng.integers(0, 3, n), 1)
    s = (rng.random(n) * ((1 << 24) - f + 1)).astype(np.int64)
    return s, f


def cuda32(x):
    return torch.from_numpy(np.asarray(x, np.int64).astype(np.int32)).cuda()


@pytest.mark.parametrize("cuts", [[0, 1], [0, 0, 3, 3], [0, 31, 63, 96, 128],
                                  [5, 38, 38, 200, 333, 1500], list(range(0, 90, 9))])
def test_streams_of_intervals(cuts):
    rng = np.random.default_rng(len(cuts))
    n = cuts[-1] + 4
    s, f = random_intervals(n, rng)
    ch = rb.Chunking.explicit(torch.tensor(cuts, device="cuda"))
    out, offs, ws = rb.encode_intervals(cuda32(s), cuda32(f), ch)
    status_ok(ws)
    got = rb.to_byte_strings(out, offs)
    assert got == [TO.encode(s[a:b], f[a:b]) for a, b in zip(cuts, cuts[1:])]


@pytest.mark.parametrize("S", [1, 16, 17, 40])
def test_long_streams(S):
    """Thousands of divisors, on both sides of the one-block form's 16 streams;
    reusing a workspace that holds an old error."""
    n = 6000
    s, f = random_intervals(n, np.random.default_rng(S))
    f[::7] = np.random.default_rng(1).integers(1, 1 << 24, f[::7].size)
    s = np.minimum(s, (1 << 24) - f)
    ch = rb.Chunking.contig(S)
    bad = f.copy()
    bad[5] = 0
    _, _, ws = rb.encode_intervals(cuda32(s), cuda32(bad), ch)
    out, offs, ws = rb.encode_intervals(cuda32(s), cuda32(f), ch, ws=ws)
    status_ok(ws)
    per = -(-n // S)
    assert rb.to_byte_strings(out, offs) == [
        TO.encode(s[k * per:(k + 1) * per], f[k * per:(k + 1) * per]) for k in range(S)]


def test_streams_extremes_and_contiguous_chunks():
    for f0 in (1, 2, 3, (1 << 24) - 1, 1 << 24):
        s, f = np.zeros(100, np.int64), np.full(100, f0)
        s[::2] = (1 << 24) - f0
        for S in (1, 3, 7):
            out, offs, ws = rb.encode_intervals(cuda32(s), cuda32(f), rb.Chunking.contig(S))
            status_ok(ws)
            per = -(-100 // S)
            assert rb.to_byte_strings(out, offs) == [
                TO.encode(s[k * per:(k + 1) * per], f[k * per:(k + 1) * per]) for k in range(S)]
    out, offs, ws = rb.encode_intervals(cuda32([]), cuda32([]), rb.Chunking.contig(2))
    status_ok(ws)
    assert rb.to_byte_strings(out, offs) == [TO.encode([], [])] * 2


def test_streams_errors():
    s, f = random_intervals(64, np.random.default_rng(8))
    one = rb.Chunking.contig(2)

    def code(s, f, ch=one, **kw):
        _, _, ws = rb.encode_intervals(cuda32(s), cuda32(f), ch, **kw)
        return rb.rans_get_status(ws)

    assert code(s, f) == rb.OK
    g = f.copy()
    g[40] = 0
    assert code(s, g) == rb.ERR_ZERO_FREQ
    t = s.copy()
    t[3] = (1 << 24) - f[3] + 1
    assert code(t, f) == rb.ERR_RANGE
    g = f.copy()
    g[3] = (1 << 24) + 1
    assert code(s, g) == rb.ERR_RANGE
    assert code(s, f, out=torch.empty(16, dtype=torch.uint8, device="cuda")) == rb.ERR_CAPACITY
    for cuts in ([0, 40, 30, 64], [0, 65], [-1, 64], [10, 3, 20]):
        ch = rb.Chunking.explicit(torch.tensor(cuts, device="cuda"))
        assert code(s, f, ch) == rb.ERR_ARG


# --------------------------------------------------------------- decoding --
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v,pad", SIZES)
def test_decode_step(v, pad, dtype):
    """Random words are a stream: states under way against the oracle's."""
    n = 7
    x = make_logits(n, v, dtype, pad, seed=5, offset=pad)
    rng = np.random.default_rng(v + 1)
    st = rb.new_status()
    for parts in (None, dict(), dict(mask=False, per_row=True)):
        a, o = (None, {}) if parts is None else make_adjust(n, v, seed=v + 3, **parts)
        lens = rng.integers(2, 6, n)
        words = rng.integers(0, 1 << 32, lens.sum(), dtype=np.uint64).astype(np.uint32)
        offs = np.concatenate([[0], np.cumsum(lens) * 4])
        state = [int(rng.integers(1 << 31, 1 << int(rng.integers(32, 64)), dtype=np.uint64))
                 for _ in range(n)]
        states = torch.tensor([[q, 1] for q in state], device="cuda")
        before = states.clone()
        data = torch.from_numpy(words.view(np.uint8).copy()).cuda()
        tok, new = rb.decode_tokens(x, data, torch.from_numpy(offs).cuda(), states, a, status=st)
        status_ok(st)
        assert torch.equal(states, before)
        for r, row in enumerate(numpy_rows(x)):
            d = TO.Decoder(words[offs[r] // 4:offs[r + 1] // 4].tobytes())
            d.x, d.at = state[r], 1
            assert int(tok[r]) == d.step(TO.bounds(row, o, r))
            assert new[r].tolist() == [d.x, d.at]
        # in place, the same
        tok2, same = rb.decode_tokens(x, data, torch.from_numpy(offs).cuda(), states, a,
                                      out_states=states, status=st)
        assert same is states and torch.equal(states, new) and torch.equal(tok, tok2)


def coded(n, v, length, dtype=F32, seed=0):
    """n texts of `length` tokens, each position's row the same for all texts."""
    x = make_logits(length, v, dtype, seed=seed)
    tok = torch.randint(0, v, (n, length), device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(seed))
    c = rb.TokenCoder()
    for k in range(n):
        c.add(x, tok[k])
    return x, tok, c.streams([length] * n)


def test_decode_streams_of_different_lengths_and_padded_rows():
    v, lengths = 300, [5, 0, 12, 1, 9]
    x, tok, _ = coded(1, v, sum(lengths), seed=7)
    c = rb.TokenCoder()
    data, offs = c.add(x[:10], tok[0, :10]).add(x[10:], tok[0, 10:]).streams(lengths)
    cut = np.concatenate([[0], np.cumsum(lengths)])
    c.begin(data, offs)
    got = [[] for _ in lengths]
    for t in range(max(lengths)):
        live = [k for k in range(5) if t < lengths[k]][::-1]
        ids = torch.tensor(live + [-1, -1], dtype=torch.int32, device="cuda")
        rows = torch.cat([x[[cut[k] + t for k in live]],
                          torch.full((2, v), math.nan, device="cuda")])
        out = c.step(rows, stream_ids=ids).tolist()
        assert out[-2:] == [-1, -1]
        for k, w in zip(live, out):
            got[k].append(w)
    c.finish()
    assert sum(got, []) == tok[0].tolist()


def test_decode_leaves_what_it_does_not_name():
    x, tok, (data, offs) = coded(4, 50, 3)
    st = rb.new_status()
    states = rb.token_states(data, offs, st)
    ids = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    out = torch.full((4, 2), 99, device="cuda")
    t = torch.full((3,), 55, dtype=torch.int32, device="cuda")
    rb.decode_tokens(x[:1].expand(3, 50).contiguous(), data, offs, states, stream_ids=ids,
                     out_states=out, tokens=t, status=st)
    status_ok(st)
    assert t.tolist() == [int(tok[2, 0]), 55, int(tok[0, 0])]
    assert out[1].tolist() == [99, 99] and out[3].tolist() == [99, 99]
    # fewer rows than streams: the others' states are kept
    t, out = rb.decode_tokens(x[:1].expand(2, 50).contiguous(), data, offs, states, status=st)
    assert t.tolist() == tok[:2, 0].tolist() and torch.equal(out[2:], states[2:])


def test_decode_errors():
    x, tok, (data, offs) = coded(4, 50, 3)
    st = rb.new_status()
    states = rb.token_states(data, offs, st)
    rows = x[:1].expand(4, 50).contiguous()

    def step(ids=None, states=states, rows=rows, offs=offs, data=data, a=None):
        ids = None if ids is None else torch.tensor(ids, dtype=torch.int32, device="cuda")
        t, s = rb.decode_tokens(rows, data, offs, states, a, stream_ids=ids, status=st)
        return t.tolist(), s, rb.rans_get_status(st)

    good, after, code = step()
    assert good == tok[:, 0].tolist() and code == rb.OK
    t, s, code = step([0, 4, -2, 1])
    assert code == rb.ERR_INDEX and t == [good[0], -1, -1, good[1]]
    assert torch.equal(s[2:], states[2:]) and torch.equal(s[:2], after[:2])
    t, s, code = step([3, 1, 3, 0])
    assert code == rb.ERR_INDEX and t == [-1, good[1], -1, good[0]]
    assert torch.equal(s[2:], states[2:])
    bad = states.clone()
    bad[1, 0], bad[2, 0] = (1 << 31) - 1, -1      # below the bound; past 2^63
    t, s, code = step(states=bad)
    assert code == rb.ERR_CORRUPT and t == [good[0], -1, -1, good[3]]
    assert torch.equal(s[1:3], bad[1:3])
    dead = rows.clone()
    dead[1], dead[2, 7] = -math.inf, math.nan
    t, s, code = step(rows=dead)
    assert code in (rb.ERR_ZERO_FREQ, rb.ERR_RANGE) and t == [good[0], -1, -1, good[3]]
    assert torch.equal(s[1:3], states[1:3])
    # past a stream's end: decoding goes on until it would need a word
    c = rb.TokenCoder().begin(data, offs)
    with pytest.raises(rb.RansError):
        for _ in range(40):
            c.step(rows)
        c.finish()
    # offsets that lie
    for lie in ([0, 10, 20, 30, 40], [64, 48, 32, 16, 0], [0] * 4 + [1 << 40], [0] * 5,
                [-8, 16, 32, 48, 64]):
        lie = torch.tensor(lie, device="cuda")
        rb.token_states(data, lie, st)
        assert rb.rans_get_status(st) == rb.ERR_CORRUPT
        low = states.clone()
        low[:, 0] = 1 << 31                       # the next token needs a word
        _, s, code = step(states=low, offs=lie)
        assert code in (rb.ERR_CORRUPT, rb.OK)    # a row may still find its word in bounds
    # truncated and too long streams do not finish
    for cut in (-1, 1):
        o = offs.clone()
        o[-1] += 4 * cut
        d = torch.cat([data, data[:4]])
        c = rb.TokenCoder().begin(d, o)
        with pytest.raises(rb.RansError):
            for t in range(3):
                c.step(x[t:t + 1].expand(4, 50).contiguous())
            c.finish()


# ----------------------------------------------------------- distillation --
def teacher(n, v, K, seed, tail):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(v)[:K] for _ in range(n)]).astype(np.int32)
    lp = rng.normal(0, 2, (n, K))
    mass = rng.uniform(0.3, 0.999, (n, 1)) if tail and K < v else 1.0
    lp = (lp - np.log(np.exp(lp).sum(1, keepdims=True) / mass)).astype(np.float32)
    if K > 2:
        gone = rng.random((n, K)) < 0.2
        gone[0] = True                     # a row without entries
        ids[gone & (rng.random((n, K)) < 0.5)] = -1
        lp[gone] = -np.inf
    return ids, lp


def check_distill(x, ids, lp, T, tail, g, losses, grad):
    rows, L, G = numpy_rows(x), losses.double().cpu().numpy(), grad.double().cpu().numpy()
    v, inv, fi = rows.shape[1], 1.0 / T, torch.finfo(grad.dtype)
    for r in range(rows.shape[0]):
        want, dz, parts = TO.distill(rows[r], ids[r], lp[r], inv, tail)
        arg = np.abs(rows[r].astype(np.float64) - rows[r].max()) * inv
        # sums of 2^a: the exponential's own error 2^-22, three roundings of an
        # argument (weighted by its term: |a| 2^-a stays below log2 v + 1), and
        # at most ceil(v / 512) + 20 float32 additions in a row
        eps = 2.0 ** -22 + U * (3 * 0.7 * (math.log2(v) + 1) + v / 512 + 20)
        assert abs(L[r] - want) <= 2 * eps + U * abs(want), (r, L[r], want)
        rel = 2 * eps + U * (8 + 4 * arg)
        tol = abs(g[r]) * parts * rel + np.abs(dz * g[r]) * (fi.eps / 2 + 2 * U) + \
            fi.smallest_normal * fi.eps / 2 + 2.0 ** -126
        off = np.abs(G[r] - dz * g[r])
        assert (off <= tol).all(), (r, float((off - tol).max()))


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("v,pad", SIZES)
def test_distill(v, pad, dtype, tail):
    n, T = 4, 1.3
    x = make_logits(n, v, dtype, pad, seed=6, offset=pad)
    rng = np.random.default_rng(v)
    for K in sorted({1, min(v, 5), min(v, 700)}):
        ids, lp = teacher(n, v, K, v + K, tail)
        g = rng.uniform(-2, 2, n).astype(np.float32)
        ti, tl, tg = (torch.from_numpy(a).cuda() for a in (ids, lp, g))
        st = rb.new_status()
        y = x.detach().requires_grad_()
        losses = rb.distill_loss(y, ti, tl, T, tail, status=st)
        (grad,) = torch.autograd.grad(losses, y, tg)
        check_distill(x, ids, lp, T, tail, g, losses.detach(), grad)
        losses, grad = rb.distill_loss_and_grad(x, ti, tl, tg, T, tail, status=st)
        check_distill(x, ids, lp, T, tail, g, losses, grad)
        status_ok(st)


@pytest.mark.parametrize("shift", [-20000.0, 20000.0])
def test_distill_and_intervals_far_from_zero(shift):
    """Only differences of logits count, wherever they lie."""
    n, v = 3, 5000
    x = make_logits(n, v, F32, seed=16) + shift
    x[1, 2500:] -= 30000.0                 # a row whose ends lie far apart
    x[2, :2500] -= 30000.0
    ids, lp = teacher(n, v, 30, 7, True)
    g = np.array([1.0, -0.5, 2.0], np.float32)
    ti, tl, tg = (torch.from_numpy(a).cuda() for a in (ids, lp, g))
    # a logit's own place is 2^-10 apart here, and c z - s is one rounding of
    # terms of 2^15: at most 2^-9 off in the exponent, which goes into both R and
    # the gradient; the rest is as near zero
    losses, grad = rb.distill_loss_and_grad(x, ti, tl, tg)
    rows = numpy_rows(x)
    for r in range(n):
        want, dz, parts = TO.distill(rows[r], ids[r], lp[r], 1.0, True)
        assert math.isfinite(want)
        assert abs(float(losses[r]) - want) <= 2.0 ** -7 + 1e-5 * abs(want)
        off = np.abs(grad[r].double().cpu().numpy() - dz * g[r])
        assert (off <= abs(g[r]) * parts * 2.0 ** -6 + 2.0 ** -126).all()
    b = [TO.bounds(row, {}, 0) for row in rows]
    tok = np.array([int(np.argmax(np.diff(q))) for q in b], np.int32)
    st = rb.new_status()
    s, f = rb.token_intervals(x, torch.from_numpy(tok).cuda(), status=st)
    assert s.tolist() == [q[t] for q, t in zip(b, tok)]
    assert f.tolist() == [q[t + 1] - q[t] for q, t in zip(b, tok)]
    status_ok(st)


def test_distill_in_place_and_into_a_wider_buffer():
    n, v = 5, 3001
    x = make_logits(n, v, BF16, 2, seed=8)
    ids, lp = teacher(n, v, 20, 1, True)
    ti, tl = torch.from_numpy(ids).cuda(), torch.from_numpy(lp).cuda()
    w = torch.linspace(0.5, 2, n, device="cuda")
    losses, grad = rb.distill_loss_and_grad(x, ti, tl, w)
    wide = torch.full((n, v + 9), 7.0, device="cuda", dtype=BF16)
    rb.distill_loss_and_grad(x, ti, tl, w, grad=wide[:, 4:v + 4])
    assert torch.equal(wide[:, 4:v + 4], grad)
    assert bool((wide[:, :4] == 7).all()) and bool((wide[:, v + 4:] == 7).all())
    y = x.clone()
    l2, g2 = rb.distill_loss_and_grad(y, ti, tl, w, grad=y)
    assert torch.equal(y, grad) and torch.equal(l2, losses)


def test_distill_against_differences():
    """Central differences of the kernel's own losses.  With steps of 1/8 the
    third derivative (of softmax terms, below 0.2 in sum) adds at most
    h^2 / 6 * 0.2 = 5.3e-4, the losses' own errors (below 4e-6 here) 6.4e-5."""
    v, K = 40, 6
    x = make_logits(1, v, F32, seed=9)
    ids, lp = teacher(1, v, K, 3, True)
    ids, lp = np.abs(ids), np.where(np.isinf(lp), -3.0, lp).astype(np.float32)
    ids = np.array([np.random.default_rng(0).permutation(v)[:K]], np.int32)
    lp -= max(0.0, float(np.log(np.exp(lp.astype(np.float64)).sum() / 0.9)))
    ti, tl = torch.from_numpy(ids).cuda(), torch.from_numpy(lp).cuda()
    for tail in (True, False):
        _, grad = rb.distill_loss_and_grad(x, ti, tl, torch.ones(1, device="cuda"), tail=tail)
        h = 0.125
        eye = torch.eye(v, device="cuda") * h
        many = torch.cat([x + eye, x - eye])
        L = rb.distill_loss(many, ti.expand(2 * v, K).contiguous(),
                            tl.expand(2 * v, K).contiguous(), tail=tail)
        diff = (L[:v] - L[v:]) / (2 * h)
        assert float((diff - grad[0]).abs().max()) <= 5.3e-4 + 6.4e-5


def test_distill_small_tails_keep_their_precision():
    """A student whose mass outside the list is 1e-12: 1 - sum q has no digit
    of it in float32, its own sum all of them."""
    v = 1000
    x = torch.randn(2, v, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    x[:, 3] += 30.0
    x[1] *= 3.0
    ids = np.array([[3], [3]], np.int32)
    lp = np.log(np.array([[0.9], [0.999]])).astype(np.float32)
    g = np.ones(2, np.float32)
    out = rb.distill_loss_and_grad(x, torch.from_numpy(ids).cuda(), torch.from_numpy(lp).cuda(),
                                   torch.from_numpy(g).cuda())
    check_distill(x, ids, lp, 1.0, True, g, *out)


def test_distill_rows_without_mass_and_bad_logits():
    v = 64
    x = make_logits(6, v, F32, seed=10)
    x[0] = -math.inf
    x[0, 5] = 1.0                  # all mass on the listed token, teacher has a tail
    x[1, 9] = -math.inf            # no mass on a listed token
    x[2, 4] = math.nan
    x[3, 4] = math.inf
    ids = np.tile(np.array([[5, 9]], np.int32), (6, 1))
    lp = np.log(np.tile(np.array([[0.5, 0.25]], np.float32), (6, 1)))
    lp[4] = -np.inf
    g = torch.ones(6, device="cuda")
    ti, tl = torch.from_numpy(ids).cuda(), torch.from_numpy(lp).cuda()
    st = rb.new_status()
    losses, grad = rb.distill_loss_and_grad(x, ti, tl, g, status=st)
    assert losses[0] == math.inf and losses[1] == math.inf
    assert bool(losses[2:4].isnan().all())
    assert bool(grad[:2].isfinite().all()) and abs(float(losses[4])) <= 1e-5
    assert float(grad[4].abs().max()) <= 1e-5
    check_distill(x[5:], ids[5:], lp[5:], 1.0, True, np.ones(1), losses[5:], grad[5:])
    # listing the whole vocabulary leaves no tail
    every = np.arange(v, dtype=np.int32)[None]
    p = np.full((1, v), math.log(0.9 / v), np.float32)
    a = rb.distill_loss_and_grad(x[5:], torch.from_numpy(every).cuda(), torch.from_numpy(p).cuda(),
                                 g[:1], status=st)
    check_distill(x[5:], every, p, 1.0, True, np.ones(1), *a)
    status_ok(st)


def test_distill_errors():
    x = make_logits(2, 50, F32)
    lp = torch.full((2, 3), math.log(0.2), device="cuda")
    w = torch.ones(2, device="cuda")
    for bad in ([1, 2, 50], [1, -2, 3], [4, 7, 4]):
        ids = torch.tensor([[1, 2, 3], bad], dtype=torch.int32, device="cuda")
        for call in (lambda s: rb.distill_loss_and_grad(x, ids, lp, w, status=s),
                     lambda s: rb.distill_loss(x, ids, lp, status=s)):
            st = rb.new_status()
            got = call(st)
            assert rb.rans_get_status(st) == rb.ERR_INDEX
            loss = got[0][0] if isinstance(got, tuple) else got[0]
            want = TO.distill(numpy_rows(x)[0], np.array([1, 2, 3]), lp[0].cpu().numpy(), 1.0,
                              True)[0]
            assert abs(float(loss) - want) <= 1e-5
    with pytest.raises(ValueError):
        rb.distill_loss(x, ids.long(), lp)
    with pytest.raises(ValueError):
        rb.distill_loss(x.t(), ids, lp)
    with pytest.raises(ValueError):
        rb.distill_loss_and_grad(x, ids, lp, w[:1])


def test_distill_through_autograd():
    """Broadcast and reduced gradients, a non-leaf student, and repeated
    backward passes."""
    n, v, K = 6, 500, 8
    x = make_logits(n, v, F32, seed=11)
    ids, lp = teacher(n, v, K, 2, True)
    ti, tl = torch.from_numpy(ids).cuda(), torch.from_numpy(lp).cuda()
    _, want = rb.distill_loss_and_grad(x, ti, tl, torch.full((n,), 1.0 / n, device="cuda"))
    y = x.clone().requires_grad_()
    loss = rb.distill_loss(y, ti, tl).mean()
    loss.backward(retain_graph=True)
    assert torch.equal(y.grad, want)
    loss.backward()
    assert torch.equal(y.grad, want * 2)
    # what is saved may come back elsewhere and with other strides
    wide = torch.zeros(n, v + 3, device="cuda")
    wide[:, :v] = x
    y = wide[:, :v].detach().requires_grad_()
    (here,) = torch.autograd.grad(rb.distill_loss(y, ti, tl).mean(), y)
    with torch.autograd.graph.save_on_cpu():
        loss = rb.distill_loss(y, ti, tl).mean()
    (g,) = torch.autograd.grad(loss, y)
    assert torch.equal(g, here)
    z = x.clone().requires_grad_()
    rb.distill_loss(z * 0.5, ti, tl).sum().backward()
    _, half = rb.distill_loss_and_grad(x * 0.5, ti, tl, torch.ones(n, device="cuda"))
    assert torch.equal(z.grad, half * 0.5)


def test_offsets_past_32_bits():
    """Rows that lie 2^30 elements apart."""
    v, step = 1003, (1 << 30) + 3
    flat = torch.zeros(2 * step + v, device="cuda", dtype=F16)
    far = flat.as_strided((3, v), (step, 1))
    x = make_logits(3, v, F16, seed=17)
    far.copy_(x)
    a, _ = make_adjust(3, v, seed=17)
    tok = torch.full((3,), 7, dtype=torch.int32, device="cuda")
    ids, lp = (torch.from_numpy(t).cuda() for t in teacher(3, v, 9, 8, True))
    w = torch.ones(3, device="cuda")
    assert torch.equal(rb.adjust_logits(far, a), rb.adjust_logits(x, a))
    for p, q in zip(rb.token_intervals(far, tok), rb.token_intervals(x, tok)):
        assert torch.equal(p, q)
    want = rb.distill_loss_and_grad(x, ids, lp, w)
    for p, q in zip(rb.distill_loss_and_grad(far, ids, lp, w), want):
        assert torch.equal(p, q)
    rb.distill_loss_and_grad(far, ids, lp, w, grad=far)
    assert torch.equal(far, want[1])


@pytest.mark.parametrize("K", [128, 129, 1000, 4096])
def test_distill_long_lists_and_the_same_bits_twice(K):
    n, v = 3, 6000
    x = make_logits(n, v, BF16, 5, seed=18)
    ids, lp = teacher(n, v, K, K, True)
    g = np.array([1.0, 2.0, -1.0], np.float32)
    args = (x, *(torch.from_numpy(t).cuda() for t in (ids, lp, g)))
    st = rb.new_status()
    one, two = (rb.distill_loss_and_grad(*args, status=st) for _ in range(2))
    check_distill(x, ids, lp, 1.0, True, g, *one)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    y = x.detach().requires_grad_()
    loss = rb.distill_loss(y, *args[1:3], status=st)
    (grad,) = torch.autograd.grad(loss, y, args[3])
    assert torch.equal(loss, one[0])
    check_distill(x, ids, lp, 1.0, True, g, loss.detach(), grad)
    status_ok(st)


def test_a_token_that_was_not_given_is_not_coded():
    x = make_logits(3, 50, F32)
    c = rb.TokenCoder()
    c.add(x, torch.tensor([1, -1, 2]))
    with pytest.raises(rb.RansError):
        c.streams([3])


# -------------------------------------------------- streams, graphs, runs --
def test_on_another_stream():
    n, v = 8, 5003
    x = make_logits(n, v, BF16, 5, seed=12)
    a, _ = make_adjust(n, v, seed=12)
    ids, lp = (torch.from_numpy(t).cuda() for t in teacher(n, v, 9, 4, True))
    w = torch.ones(n, device="cuda")
    tok = torch.zeros(n, dtype=torch.int32, device="cuda")
    want = [rb.adjust_logits(x, a), *rb.token_intervals(x, tok),
            *rb.distill_loss_and_grad(x, ids, lp, w)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [rb.adjust_logits(x, a, stream=s), *rb.token_intervals(x, tok, stream=s),
           *rb.distill_loss_and_grad(x, ids, lp, w, stream=s)]
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_captured_steps_replay_on_new_inputs():
    """A decoding step (updating its states in place, its history window
    growing) and a training step, captured once; both graphs share a status
    word."""
    v, length = 700, 6
    x, tok, (data, offs) = coded(3, v, length, seed=13)
    st = rb.new_status()
    states = rb.token_states(data, offs, st)
    rows, out = torch.empty(3, v, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    ids, lp = (torch.from_numpy(t).cuda() for t in teacher(3, v, 5, 5, True))
    w = torch.ones(3, device="cuda")
    losses, grad = torch.empty(3, device="cuda"), torch.empty(3, v, device="cuda")
    rows.copy_(x[:1].expand(3, v))
    keep = states.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # first calls set kernel attributes
        rb.decode_tokens(rows, data, offs, states, out_states=states, tokens=out, status=st)
        rb.check(rb.rans_distill(rows, ids, lp, 1.0, True, w, losses, grad, st))
    torch.cuda.current_stream().wait_stream(s)
    states.copy_(keep)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        rb.decode_tokens(rows, data, offs, states, out_states=states, tokens=out, status=st)
    with torch.cuda.graph(g2):
        rb.check(rb.rans_distill(rows, ids, lp, 1.0, True, w, losses, grad, st))
    got = []
    for t in range(length):
        rows.copy_(x[t:t + 1].expand(3, v))
        g1.replay()
        g2.replay()
        got.append(out.clone())
        want = rb.distill_loss_and_grad(rows, ids, lp, w)
        assert torch.equal(want[0], losses) and torch.equal(want[1], grad)
    assert torch.equal(torch.stack(got, 1), tok.to(torch.int32))
    rb.check(rb.rans_token_states_finish(offs, states, st))
    status_ok(st)


def test_a_text_under_sampling_rules_from_end_to_end():
    """As used: a model yields rows, texts are drawn under penalties, a bias,
    a temperature and a grammar, coded with the whole text's rows at once
    (each position's history being what came before it), and decoded one
    token per step; the distillation loss gives the streams' rate."""
    n, v, length = 4, 1500, 20
    g = torch.Generator("cuda").manual_seed(21)
    table = torch.randn(v, v, device="cuda", generator=g).mul_(2.5).to(BF16)  # next-token rows
    rules = dict(temperature=0.9, repetition=1.2, frequency=0.2, presence=0.1)
    mask = rb.pack_mask(torch.rand(v, device="cuda", generator=g) < 0.3)
    bias = (torch.tensor([3, 9, 3], dtype=torch.int32, device="cuda"),
            torch.tensor([1.0, 2.0, -1.0], device="cuda"))
    texts = torch.zeros(n, length + 1, dtype=torch.int32, device="cuda")
    base = torch.arange(n, device="cuda") * (length + 1)

    def step_rules(rows, begin, end):
        windows = [torch.full((rows,), k, device="cuda") for k in (0, 3)]
        return rb.LogitAdjust(history=(texts.view(-1), begin, end), bias=(*bias, *windows),
                              mask=mask, **rules)

    for t in range(length):     # draw the texts
        z = rb.adjust_logits(table[texts[:, t].long()], step_rules(n, base, base + t + 1),
                             dtype=F32)
        texts[:, t + 1] = torch.multinomial(torch.softmax(z, 1), 1, generator=g)[:, 0]
    drawn = texts.clone()
    # encode: all positions of all texts
    rows = table[texts[:, :-1].reshape(-1).long()]
    at = base[:, None] + torch.arange(length, device="cuda") + 1
    c = rb.TokenCoder()
    c.add(rows, texts[:, 1:].reshape(-1),
          step_rules(n * length, base.repeat_interleave(length), at.reshape(-1)))
    data, offs = c.streams([length] * n)
    # the rate: one listed token of probability 1, under the adjusted logits
    z = rb.adjust_logits(rows, step_rules(n * length, base.repeat_interleave(length),
                                          at.reshape(-1)), dtype=F32)
    rate = rb.distill_loss(z, texts[:, 1:].reshape(-1, 1), torch.zeros(n * length, 1,
                                                                      device="cuda"))
    bits = rate.view(n, length).sum(1).double() / math.log(2)
    size = (offs[1:] - offs[:-1]) * 8
    # a stream holds its tokens' bits on top of the 31 of the initial state, in
    # whole 32-bit words of a state between 2^31 and 2^63.  Intervals cost at
    # most 0.02 bits a token over the softmax (N ones of 2^24, the weights'
    # 1e-4) for tokens of this probability.
    assert bool((size >= bits + 31 - length * 0.02).all())
    assert bool((size <= bits + 31 + 33 + length * 0.02).all())
    # decode into an empty text
    texts.zero_()
    c.begin(data, offs)
    for t in range(length):
        texts[:, t + 1] = c.step(table[texts[:, t].long()], step_rules(n, base, base + t + 1))
    c.finish()
    assert torch.equal(texts, drawn)
