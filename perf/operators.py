"""The language-model operators of the library, as cases to measure.

Three families: ``adjust`` (penalties, biases, masks and temperature on
logits), ``encode`` / ``decode`` (coding tokens under a model's logits: whole
texts at once in one direction, one token per stream and step in the other)
and ``distill`` (the coder's rate against a teacher's top probabilities, with
its gradient).  ``run`` computes each in elementary torch operations, or,
where ``own`` is set, through the library's calls.
"""
import math

import torch

own = False

FLOATS = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}

# The token coder's definition: intervals at 24 bits, weights at 21 bits and
# the polynomial for 2^f on [-1/2, 1/2], every operation rounded to float32.
PRECISION = 24
WEIGHT_BITS = 21
LOG2E = 1.4426950216293335
C1, C2, C3 = 0.6932829022407532, 0.2422109693288803, 0.05500893294811249
LOWEST = -64.0
STATE_LOW = 1 << 31


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one request of a server, between two model steps: launch latency
        dict(name="adjust one row", op="adjust", rows=1, vocab=32768, dtype="float32", pad=0,
             history=512, bias=16, mask=False),
        # rows of an odd vocabulary inside a wider buffer, under a grammar
        dict(name="adjust odd rows", op="adjust", rows=61, vocab=50021, dtype="float16", pad=3,
             history=700, bias=100, mask=True),
        # a full serving batch with every adjustment in use
        dict(name="adjust serving batch", op="adjust", rows=256, vocab=131072, dtype="bfloat16",
             pad=0, history=2048, bias=32, mask=True),
        # a message of a hundred tokens
        dict(name="encode a message", op="encode", rows=100, vocab=32768, dtype="float32", pad=0,
             streams=1, adjust=False),
        # stored replies, coded under the very sampling rules that made them;
        # the history of a token is what came before it in its reply
        dict(name="encode sampled replies", op="encode", rows=777, vocab=50021, dtype="float16",
             pad=5, streams=5, adjust=True),
        # a corpus in 64 pieces
        dict(name="encode a corpus", op="encode", rows=4096, vocab=131072, dtype="bfloat16",
             pad=0, streams=64, adjust=False),
        # one stream, one token: the latency of a decoding step
        dict(name="decode one stream", op="decode", rows=1, vocab=131072, dtype="bfloat16", pad=0,
             adjust=False),
        # a batch under penalties and a grammar, odd vocabulary
        dict(name="decode constrained", op="decode", rows=48, vocab=50021, dtype="float32", pad=3,
             adjust=True),
        # a full decoding batch
        dict(name="decode batch", op="decode", rows=256, vocab=131072, dtype="bfloat16", pad=0,
             adjust=False),
        # a small batch, loss and gradient through autograd
        dict(name="distill small batch", op="distill", rows=96, vocab=32768, dtype="float32",
             pad=0, top=16, tail=True, autograd=True),
        # odd vocabulary, teacher renormalised over its list, some entries absent
        dict(name="distill odd rows", op="distill", rows=1001, vocab=50021, dtype="float16",
             pad=7, top=50, tail=False, autograd=False),
        # a training step's rows, loss and gradient in one call
        dict(name="distill training step", op="distill", rows=4096, vocab=131072,
             dtype="bfloat16", pad=0, top=128, tail=True, autograd=False),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adjust", "encode", "decode", "distill"])
    vocab = _log_between(rng, 1000, 131072)
    c = dict(op=op, vocab=vocab, dtype=rng.choice(sorted(FLOATS)), pad=rng.choice([0, 0, 1, 3, 8]))
    if op == "adjust":
        c["rows"] = _log_between(rng, 1, 256)
        c["history"] = rng.choice([0, _log_between(rng, 1, 4096)])
        c["bias"] = rng.choice([0, _log_between(rng, 1, 300)])
        c["mask"] = rng.random() < 0.5
    elif op == "encode":
        c["adjust"] = rng.random() < 0.5
        c["rows"] = _log_between(rng, 1, 777 if c["adjust"] else 4096)
        c["streams"] = min(c["rows"], _log_between(rng, 1, 64))
    elif op == "decode":
        c["rows"] = _log_between(rng, 1, 256)
        c["adjust"] = rng.random() < 0.5
    else:
        c["rows"] = _log_between(rng, 16, 4096)
        c["top"] = _log_between(rng, 1, 128)
        c["tail"] = rng.random() < 0.5
        c["autograd"] = rng.random() < 0.5
    if c["dtype"] == "float32":  # no more bytes than the largest listed case
        c["rows"] = max(1, c["rows"] // 2)
        if op == "encode":
            c["streams"] = min(c["streams"], c["rows"])
    return c


# ----------------------------------------------------------------- inputs --
def _logits(c, g):
    """Rows as a language model's head gives them: a broad body and a few
    tokens that hold most of the mass, inside a buffer `pad` columns wider."""
    n, v = c["rows"], c["vocab"]
    wide = torch.empty(n, v + c["pad"], device="cuda", dtype=FLOATS[c["dtype"]])
    x = torch.randn(n, v, device="cuda", generator=g).mul_(2.0)
    few = torch.randint(0, v, (n, 8), device="cuda", generator=g)
    x.scatter_add_(1, few, torch.rand(n, 8, device="cuda", generator=g) * 12.0)
    wide[:, v:] = 0
    wide[:, :v] = x
    return wide[:, :v]


def _mask(n, v, g):
    """A grammar's allowed tokens, 32 to a word: about a tenth of them."""
    words = (v + 31) // 32
    m = None
    for _ in range(3):
        r = torch.randint(-2**31, 2**31, (n, words), device="cuda", generator=g)
        m = r if m is None else m & r
    return m.to(torch.int32)


def _ragged(n, most, g):
    """Windows [begin, end) of up to `most` entries, one after another."""
    lens = torch.randint(most // 2, most + 1, (n,), device="cuda", generator=g)
    end = torch.cumsum(lens, 0)
    return end - lens, end, int(lens.sum())


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, v = c["rows"], c["vocab"]
    s = dict(case=c, logits=_logits(c, g), temperature=1.0, repetition=1.0, frequency=0.0,
             presence=0.0, history=None, bias=None, mask=None)
    s["status"] = torch.zeros(32, dtype=torch.int64, device="cuda")
    adjusted = c["op"] == "adjust" or c.get("adjust", False)
    if adjusted:
        s.update(temperature=0.8, repetition=1.1, frequency=0.1, presence=0.3)
        most = c.get("history", 300)
        if most and c["op"] != "encode":
            begin, end, total = _ragged(n, most, g)
            # a text repeats its words: ids crowd towards 0
            r = torch.rand(max(total, 1), device="cuda", generator=g)
            s["history"] = ((r * r * r * v).to(torch.int32).clamp_(0, v - 1), begin, end)
        most = c.get("bias", 24)
        if most:
            begin, end, total = _ragged(n, most, g)
            ids = torch.randint(0, v, (max(total, 1),), device="cuda", generator=g)
            values = torch.randn(max(total, 1), device="cuda", generator=g) * 3.0
            s["bias"] = (ids.to(torch.int32), values, begin, end)
        if c.get("mask", True):
            s["mask"] = _mask(n, v, g)
            if c["op"] != "adjust":
                s["mask"][:, 0] |= 2  # every row allows something
    if c["op"] == "encode":
        _prepare_encode(s, c, g)
    elif c["op"] == "decode":
        # any words are a stream: they decode to tokens of the model's own
        # distribution.  A state and room for two more words per stream.
        lens = torch.randint(3, 6, (n,), device="cuda", generator=g)
        off = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
        off[1:] = torch.cumsum(lens, 0) * 4
        total = int(off[-1]) // 4
        words = torch.randint(-2**31, 2**31, (total,), device="cuda", generator=g)
        s["data"] = words.to(torch.int32).view(torch.uint8)
        s["offsets"] = off
        # states of streams under way (some of them refill in this step), as
        # (state, words taken)
        lo = torch.randint(0, 2**31, (n,), device="cuda", generator=g)
        hi = torch.randint(1, 2**22, (n,), device="cuda", generator=g)
        x = hi * 2**31 + lo
        s["states"] = torch.stack([x, torch.full_like(x, 2)], 1).contiguous()
    elif c["op"] == "distill":
        _prepare_distill(s, c, g)
    return s


def _prepare_encode(s, c, g):
    n, v, k = c["rows"], c["vocab"], c["streams"]
    cuts = torch.randperm(max(n - 1, 1), device="cuda", generator=g)[:k - 1].sort().values + 1
    starts = torch.zeros(k + 1, dtype=torch.int64, device="cuda")
    starts[1:k] = cuts
    starts[k] = n
    s["starts"] = starts
    s["longest"] = int((starts[1:] - starts[:-1]).max())
    # the texts: tokens drawn from the model's rows, among the allowed ones
    u = torch.rand(n, v, device="cuda", generator=g).clamp_(min=1e-30)
    score = u.log_().neg_().log_().neg_()
    score += s["logits"]
    if s["mask"] is not None:
        score.masked_fill_(~_allowed(s["mask"], v), -math.inf)
    tokens = score.argmax(1)
    s["tokens"] = tokens.to(torch.int32)
    if s["case"]["adjust"]:
        at = torch.arange(n, device="cuda")
        mine = torch.searchsorted(starts, at, right=True) - 1
        s["history"] = (s["tokens"], starts[mine].contiguous(), at)
    # room for the longest coding of these texts, and the S + 1 offsets
    s["out"] = torch.zeros(8 * n + 32 * k, dtype=torch.uint8, device="cuda")


def _prepare_distill(s, c, g):
    n, v, k = c["rows"], c["vocab"], min(c["top"], c["vocab"])
    teacher = torch.randn(n, v, device="cuda", generator=g).mul_(0.5).add_(s["logits"])
    top, ids = teacher.topk(k, dim=1)
    lp = top - torch.logsumexp(teacher, 1, keepdim=True)
    if not c["tail"]:  # a ragged teacher: some entries of its lists are absent
        gone = torch.rand(n, k, device="cuda", generator=g) < 0.1
        ids = ids.masked_fill(gone, -1)
        lp = lp.masked_fill(gone, -math.inf)
    s["ids"], s["logprobs"] = ids.to(torch.int32).contiguous(), lp.contiguous()
    # the rows' weights in the loss; half-precision training scales its loss
    # so that small gradients stay above the type's smallest normal number
    scale = 65536.0 if c["dtype"] == "float16" else 1.0
    s["weights"] = torch.rand(n, device="cuda", generator=g).add_(0.5).mul_(scale / n)
    s["distill_temperature"] = 1.5


# ------------------------------------------------------- plain: adjustment --
def _allowed(mask, v):
    at = torch.arange(v, device=mask.device)
    return ((mask[:, at >> 5] >> (at & 31).to(torch.int32)) & 1) != 0


def _pairs(begin, end):
    """(row, position) of every entry of the rows' windows."""
    lens = end - begin
    rows = torch.repeat_interleave(torch.arange(lens.numel(), device=lens.device), lens)
    first = torch.cumsum(lens, 0) - lens
    at = torch.arange(rows.numel(), device=lens.device) - first[rows] + begin[rows]
    return rows, at


def _before_temperature(s):
    """Penalised and biased logits in 32 bits, and the rows' masks."""
    z = s["logits"].float()
    n, v = z.shape
    if s["history"] is not None:
        tokens, begin, end = s["history"]
        rows, at = _pairs(begin, end)
        count = torch.zeros(n * v, device=z.device)
        count.scatter_add_(0, rows * v + tokens[at], torch.ones(at.numel(), device=z.device))
        count = count.view(n, v)
        rho = torch.tensor(s["repetition"], device=z.device)
        less = count * s["frequency"] + s["presence"]
        z = torch.where(count > 0, torch.where(z > 0, z / rho, z * rho) - less, z)
    if s["bias"] is not None:
        ids, values, begin, end = s["bias"]
        rows, at = _pairs(begin, end)
        # the last entry of a row for a token counts
        last = torch.full((n * v,), -1, dtype=torch.int64, device=z.device)
        last.scatter_reduce_(0, rows * v + ids[at], at, "amax")
        last = last.view(n, v)
        z = torch.where(last >= 0, z + values[last.clamp(min=0)], z)
    return z, None if s["mask"] is None else _allowed(s["mask"], v)


def _plain_adjust(s):
    z, allowed = _before_temperature(s)
    z = z * torch.tensor(1.0 / s["temperature"], device=z.device)
    if allowed is not None:
        z = z.masked_fill(~allowed, -math.inf)
    return z.to(s["logits"].dtype)


# ----------------------------------------------------- plain: token coding --
def _weights(s):
    """Integer weights of every token, and which tokens are alive."""
    z, allowed = _before_temperature(s)
    if allowed is not None:
        z = z.masked_fill(~allowed, -math.inf)
    alive = z > -math.inf
    # both factors in 32 bits, as the format has them
    scale = torch.tensor(LOG2E, device=z.device) * torch.tensor(1.0 / s["temperature"],
                                                                device=z.device)
    y = z * scale
    d = (y - y.max(1, keepdim=True).values).clamp(min=LOWEST)
    k = torch.round(d)
    f = d - k
    p = ((f * C3 + C2) * f + C1) * f + 1.0
    power = ((k.to(torch.int32) + (127 + WEIGHT_BITS)) << 23).view(torch.float32)
    return torch.round(p * power).to(torch.int64), alive


def _bounds(w, alive):
    """Start of every token's interval, and the end of the last."""
    c = torch.cumsum(w, 1)
    total, r = c[:, -1:], torch.cumsum(alive.to(torch.int64), 1)
    room = (1 << PRECISION) - r[:, -1:]
    ends = c * room // total + r
    return torch.nn.functional.pad(ends, (1, 0))


def _plain_encode(s):
    bounds = _bounds(*_weights(s))
    at = s["tokens"].to(torch.int64)[:, None]
    start = bounds.gather(1, at)[:, 0]
    freq = bounds.gather(1, at + 1)[:, 0] - start
    first, size = s["starts"][:-1], s["starts"][1:] - s["starts"][:-1]
    k, longest = first.numel(), s["longest"]
    x = torch.full_like(first, STATE_LOW)
    # words from a row's end downwards: a column of slack for what is not kept
    words = torch.zeros(k, longest + 3, dtype=torch.int64, device=x.device)
    used = torch.zeros_like(first)
    for t in range(longest - 1, -1, -1):  # a state follows from the one before
        here = size > t
        i = torch.where(here, first + t, 0)
        f = torch.where(here, freq[i], 1)
        emit = here & (x >> 39 >= f)
        words.scatter_(1, torch.where(emit, longest + 2 - used - 1, longest + 2)[:, None],
                       (x & 0xffffffff)[:, None])
        used += emit
        y = torch.where(emit, x >> 32, x)
        x = torch.where(here, ((y // f) << PRECISION) + y % f + start[i], x)
    words.scatter_(1, (longest + 1 - used)[:, None], (x >> 32)[:, None])
    words.scatter_(1, (longest - used)[:, None], (x & 0xffffffff)[:, None])
    used += 2
    offsets = torch.nn.functional.pad(torch.cumsum(used, 0), (1, 0))
    rows, at = _pairs(offsets[:-1], offsets[1:])
    col = longest + 2 - used[rows] + at - offsets[rows]
    out = torch.zeros_like(s["out"]).view(torch.int32)
    out[:at.numel()] = words[rows, col].to(torch.int32)
    return start.to(torch.int32), freq.to(torch.int32), out.view(torch.uint8), offsets * 4


def _plain_decode(s):
    bounds = _bounds(*_weights(s))
    x, taken = s["states"][:, 0], s["states"][:, 1]
    slot = x & ((1 << PRECISION) - 1)
    token = torch.searchsorted(bounds, slot[:, None], right=True)[:, 0] - 1
    start = bounds.gather(1, token[:, None])[:, 0]
    freq = bounds.gather(1, token[:, None] + 1)[:, 0] - start
    x = freq * (x >> PRECISION) + slot - start
    refill = x < STATE_LOW
    words = s["data"].view(torch.int32).to(torch.int64) & 0xffffffff
    word = words[s["offsets"][:-1] // 4 + taken]
    x = torch.where(refill, (x << 32) | word, x)
    return token.to(torch.int32), torch.stack([x, taken + refill], 1)


# ----------------------------------------------------- plain: distillation --
def _plain_distill(s):
    c = s["case"]
    inv = 1.0 / s["distill_temperature"]
    z = s["logits"].float() * inv
    n, v = z.shape
    here = (s["ids"] >= 0) & (s["logprobs"] > -math.inf)
    ids = torch.where(here, s["ids"].to(torch.int64), v)
    # row sums in 64 bits: the loss is a difference of close numbers
    lp = torch.where(here, s["logprobs"].double(), -math.inf)
    p = lp.exp()
    if c["tail"]:
        tail = (1.0 - p.sum(1)).clamp(min=0.0)
    else:
        lp = lp - torch.logsumexp(lp, 1, keepdim=True)
        p, tail = lp.exp(), torch.zeros(n, dtype=torch.float64, device=z.device)
    mass = p.sum(1) + tail
    m = z.max(1, keepdim=True).values
    e = torch.exp(z - m)
    inside = torch.nn.functional.pad(torch.zeros_like(e), (0, 1)).scatter_(1, ids, 1.0)[:, :v]
    # the listed tokens' own sum in 64 bits, and the others' without them
    listed = e.gather(1, ids.clamp(max=v - 1)).double().masked_fill(~here, 0.0)
    rest = (e * (1.0 - inside)).sum(1, dtype=torch.float64)
    total = rest + listed.sum(1)
    lq = (z.gather(1, ids.clamp(max=v - 1)) - m).double() - total.log()[:, None]
    loss = torch.where(here, p * (lp - lq), 0.0).sum(1)
    share = rest / total
    log_tail = torch.where(tail > 0, tail, 1.0).log()
    loss = loss + torch.where(tail > 0, tail * (log_tail - share.log()), 0.0)
    others = mass - torch.where(tail > 0, tail / share, 0.0)
    q = e / total.float()[:, None]
    grad = q * torch.where(inside > 0, mass.float()[:, None], others.float()[:, None])
    grad = torch.nn.functional.pad(grad, (0, 1)).scatter_add_(1, ids, -p.float())[:, :v]
    grad = grad * (s["weights"] * inv)[:, None]
    return loss.float(), grad.to(s["logits"].dtype)


# -------------------------------------------------------------------- run --
def _own(s):
    import rans_entropy_coding_b200 as rb
    op, c = s["case"]["op"], s["case"]
    adjust = None
    if s["history"] is not None or s["bias"] is not None or s["mask"] is not None or \
            s["temperature"] != 1.0:
        adjust = rb.LogitAdjust(temperature=s["temperature"], repetition=s["repetition"],
                                frequency=s["frequency"], presence=s["presence"],
                                history=s["history"], bias=s["bias"], mask=s["mask"])
    if op == "adjust":
        return rb.adjust_logits(s["logits"], adjust)
    if op == "encode":
        starts, freqs = rb.token_intervals(s["logits"], s["tokens"], adjust, status=s["status"])
        out, offsets, _ = rb.encode_intervals(starts, freqs, rb.Chunking.explicit(s["starts"]),
                                              out=s["out"])
        return starts, freqs, out, offsets
    if op == "decode":
        return rb.decode_tokens(s["logits"], s["data"], s["offsets"], s["states"], adjust,
                                status=s["status"])
    if c["autograd"]:
        x = s["logits"].detach().requires_grad_()
        loss = rb.distill_loss(x, s["ids"], s["logprobs"], temperature=s["distill_temperature"],
                               tail=c["tail"], status=s["status"])
        (grad,) = torch.autograd.grad(loss, x, s["weights"])
        return loss.detach(), grad
    return rb.distill_loss_and_grad(s["logits"], s["ids"], s["logprobs"], s["weights"],
                                    temperature=s["distill_temperature"], tail=c["tail"],
                                    status=s["status"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "adjust":
        return _plain_adjust(state)
    if op == "encode":
        return _plain_encode(state)
    if op == "decode":
        return _plain_decode(state)
    return _plain_distill(state)


def work(case):
    c = case
    n, v, e = c["rows"], c["vocab"], FLOATS[c["dtype"]].itemsize
    logits = n * v * e
    mask = n * ((v + 31) // 32) * 4
    extra = 0
    if c["op"] == "adjust":
        extra = 4 * n * c["history"] * 3 // 4 + 8 * n * c["bias"] * 3 // 4
        extra += mask if c["mask"] else 0
        return {"bytes": 2 * logits + extra, "flops": 2 * n * v}
    if c.get("adjust"):
        extra = mask + 8 * n * 18 + (4 * n * 225 if c["op"] == "decode" else 4 * n)
    if c["op"] == "encode":
        # a token in, an interval out and in again, about two bytes of stream
        return {"bytes": logits + extra + n * (4 + 8 + 8 + 2), "flops": 14 * n * v}
    if c["op"] == "decode":
        return {"bytes": logits + extra + n * (16 + 16 + 4 + 8 + 4), "flops": 14 * n * v}
    # the gradient goes out besides; teacher's ids and log probabilities in
    return {"bytes": 2 * logits + 8 * n * min(c["top"], v) + 8 * n, "flops": 8 * n * v}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """From the definitions in 64 bits.  The token coder's outputs are whole
    numbers that its 32-bit rounding steps define: they have no other value."""
    c = case
    if c["op"] in ("encode", "decode"):
        return None
    s = prepare(case, seed)
    z = s["logits"].double()
    if c["op"] == "adjust":
        out = z.clone()
        if s["history"] is not None:
            tokens, begin, end = s["history"]
            begin, end = begin.tolist(), end.tolist()
            for r in range(c["rows"]):
                seen, n = torch.unique(tokens[begin[r]:end[r]].long(), return_counts=True)
                x = z[r, seen]
                x = torch.minimum(x, x * 0) * s["repetition"] + \
                    torch.maximum(x, x * 0) / s["repetition"]
                out[r, seen] = x - s["presence"] - n.double() * s["frequency"]
        if s["bias"] is not None:
            ids, values, begin, end = (t.tolist() for t in s["bias"])
            for r in range(c["rows"]):
                mine = dict(zip(ids[begin[r]:end[r]], values[begin[r]:end[r]]))
                if mine:
                    at = torch.tensor(list(mine), device="cuda")
                    out[r, at] += torch.tensor(list(mine.values()), dtype=torch.float64,
                                               device="cuda")
        out /= s["temperature"]
        if s["mask"] is not None:
            bits = torch.stack([s["mask"] >> b & 1 for b in range(32)], 2).flatten(1)
            out[bits[:, :c["vocab"]] == 0] = -math.inf
        return out
    t = s["distill_temperature"]
    lq = torch.log_softmax(z / t, 1)
    del z
    keep = (s["ids"] >= 0) & torch.isfinite(s["logprobs"])
    lp = s["logprobs"].double()
    p = torch.where(keep, lp.exp(), 0.0)
    if c["tail"]:
        tail = (1.0 - p.sum(1)).clamp(min=0.0)
    else:
        lp = lp - p.sum(1, keepdim=True).log()
        p = p / p.sum(1, keepdim=True)
        tail = torch.zeros_like(p[:, 0])
    at = s["ids"].long().clamp(min=0)
    loss = torch.where(keep, p * (lp - lq.gather(1, at)), 0.0).sum(1)
    row = torch.arange(c["rows"], device="cuda")[:, None].expand_as(at)[keep]
    out = torch.zeros_like(lq, dtype=torch.bool)
    out[row, at[keep]] = True
    grad = lq.exp()
    rest = grad.masked_fill(out, 0.0).sum(1)
    some = tail > 0
    loss = loss + torch.where(some, tail * (tail.log() - rest.log()), 0.0)
    whole = p.sum(1) + tail
    grad *= torch.where(out, whole[:, None],
                        (whole - torch.where(some, tail / rest, 0.0))[:, None])
    grad[row, at[keep]] -= p[keep]
    grad *= (s["weights"].double() / t)[:, None]
    return loss, grad
