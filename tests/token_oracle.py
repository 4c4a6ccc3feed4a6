"""Plain versions of the language-model operators, for the tests: logit
adjustment and distillation in 64 bits, token intervals by the format's own
float32 steps (numpy rounds each to nearest) with Python integers for sums and
quotients, and a one-state rANS over Python integers.  numpy only; shares no
code with the library."""
import math

import numpy as np

PREC = 24
LOW = 1 << 31
F = np.float32


def windows(adj, part, r):
    """Row r's slice of a (arrays..., begin, end) part, clipped."""
    *arrays, begin, end = adj[part]
    n = len(arrays[0])
    b = min(max(int(begin[r]), 0), n)
    e = max(b, min(int(end[r]), n))
    return [a[b:e] for a in arrays]


def allowed(adj, r, vocab):
    if adj.get("mask") is None:
        return np.ones(vocab, bool)
    m = adj["mask"]
    words = np.asarray(m[r] if m.ndim == 2 else m).astype(np.uint32)
    v = np.arange(vocab)
    return (words[v >> 5] >> (v & 31).astype(np.uint32) & 1).astype(bool)


def param(adj, name, r, default):
    x = adj.get(name, default)
    return x[r] if isinstance(x, np.ndarray) else x


def adjusted(row, adj, r, dtype):
    """Penalised and biased logits of one row in `dtype` (before temperature
    and mask), and a bound on what float32 steps may add to the error."""
    z = row.astype(dtype)
    v = z.size
    err = np.zeros(v)
    u = 2.0 ** -24
    if adj.get("history") is not None:
        (toks,) = windows(adj, "history", r)
        count = np.zeros(v, np.int64)
        toks = toks[(toks >= 0) & (toks < v)]
        np.add.at(count, toks, 1)
        at = np.flatnonzero(count)
        rho = dtype(F(param(adj, "repetition", r, 1.0)))
        freq = dtype(F(param(adj, "frequency", r, 0.0)))
        pres = dtype(F(param(adj, "presence", r, 0.0)))
        with np.errstate(all="ignore"):
            x = np.where(z[at] > 0, z[at] / rho, z[at] * rho)
            less = count[at].astype(dtype) * freq + pres
            err[at] += u * (np.abs(x) + 2 * np.abs(less) + np.abs(pres))
            z[at] = x - less
            err[at] += u * np.abs(z[at])
    if adj.get("bias") is not None:
        ids, values = windows(adj, "bias", r)
        last = {}
        for i, b in zip(ids, values):
            if 0 <= i < v:
                last[int(i)] = b
        for i, b in last.items():
            z[i] = z[i] + dtype(b)
            err[i] += u * abs(float(z[i]))
    return z, err


def adjust(row, adj, r):
    """(values in 64 bits, error bound before the final rounding)."""
    z, err = adjusted(row, adj, r, np.float64)
    inv = 1.0 / float(param(adj, "temperature", r, 1.0))
    with np.errstate(all="ignore"):
        out = z * inv
        # 1 / T is a float32 of its own, and so is the product
        err = err * inv + np.abs(out) * 3 * 2.0 ** -24
    out[~allowed(adj, r, row.size)] = -np.inf
    return out, err


def weights(row, adj, r):
    """(integer weights, alive) of one row; the row must have an alive token
    and no bad logit."""
    with np.errstate(all="ignore"):
        z, _ = adjusted(row, adj, r, np.float32)
        alive = allowed(adj, r, row.size) & ~(z == -np.inf)
        # the temperature as the library takes it: per row a float32 division,
        # for all rows a double one rounded once
        t = param(adj, "temperature", r, 1.0)
        inv = F(1.0) / F(t) if isinstance(adj.get("temperature"), np.ndarray) else F(1.0 / t)
        scale = F(float.fromhex("0x1.715476p+0")) * inv
        y = z * scale
        top = y[alive].max()
        if top == -np.inf:
            return np.where(alive, 1 << 21, 0).astype(np.int64), alive
        d = np.maximum(y - top, F(-64))
        k = np.rint(d)
        f = d - k
        p = f * F(float.fromhex("0x1.c2a218p-5")) + F(float.fromhex("0x1.f00c4ep-3"))
        p = p * f + F(float.fromhex("0x1.62f5fap-1"))
        p = p * f + F(1)
        w = np.rint(np.ldexp(p, np.where(alive, k, -64).astype(np.int32) + 21))
    return np.where(alive, w, 0).astype(np.int64), alive


def bounds(row, adj, r):
    """Starts of all tokens and the end of the last, as Python integers."""
    w, alive = weights(row, adj, r)
    total, n = int(w.sum()), int(alive.sum())
    c = np.concatenate([[0], np.cumsum(w)])
    a = np.concatenate([[0], np.cumsum(alive)])
    room = (1 << PREC) - n
    return [int(x) * room // total + int(y) for x, y in zip(c, a)]


def encode(starts, freqs):
    """Bytes of one stream."""
    x, words = LOW, []
    for s, f in zip(reversed(list(starts)), reversed(list(freqs))):
        s, f = int(s), int(f)
        if x >= f << 39:
            words.append(x & 0xffffffff)
            x >>= 32
        x = (x // f << PREC) + x % f + s
        assert LOW <= x < 1 << 63
    words += [x >> 32, x & 0xffffffff]
    return np.array(words[::-1], np.uint32).tobytes()


class Decoder:
    def __init__(self, data):
        w = np.frombuffer(data, np.uint32)
        self.words, self.at = [int(v) for v in w], 2
        self.x = self.words[0] | self.words[1] << 32

    def step(self, b):
        slot = self.x & ((1 << PREC) - 1)
        token = int(np.searchsorted(np.array(b), slot, side="right")) - 1
        self.x = (b[token + 1] - b[token]) * (self.x >> PREC) + slot - b[token]
        if self.x < LOW:
            self.x = self.x << 32 | self.words[self.at]
            self.at += 1
        return token


def distill(row, ids, lp, inv_t, tail):
    """(loss, gradient, parts for error bounds) of one row in 64 bits."""
    z = row.astype(np.float64) * inv_t
    v = z.size
    keep = (ids >= 0) & (lp > -np.inf)
    at, l = ids[keep].astype(np.int64), lp[keep].astype(np.float64)
    if not tail and at.size == 0:
        return 0.0, np.zeros(v), np.zeros(v)
    p = np.exp(l)
    if not tail:
        l = l - math.log(p.sum())
        p = np.exp(l)
    pt = max(0.0, 1.0 - p.sum()) if tail and at.size < v else 0.0
    with np.errstate(all="ignore"):
        m = z.max()
        e = np.exp(z - m)
        out = np.ones(v, bool)
        out[at] = False
        Z, R = e.sum(), e[out].sum()
        lq = z - m - math.log(Z)
        loss = float(np.where(p > 0, p * (l - lq[at]), 0.0).sum())
        if pt > 0:
            loss += pt * (math.log(pt) - (math.log(R / Z) if R > 0 else -math.inf))
        mass = p.sum() + pt
        share = np.zeros(v)
        if R > 0:
            share[out] = e[out] / R
        grad = mass * e / Z - pt * share
        grad[at] -= p
        parts = e / Z + share
        parts[at] += p
    return loss, grad * inv_t, parts * inv_t
