"""Operators before and behind the logits, as cases to measure.

Four families: ``quantise`` (rows to microscaled 4-bit numbers and back),
``head`` (a model's last product on such numbers: hidden rows to logits),
``beam`` (the best continuations of every text over its beams and the
vocabulary) and ``reorder`` (the beams' states following their parents, in
place).  ``run`` computes each in elementary torch operations, or, where
``own`` is set, through the library's calls.
"""
import math

import torch

own = False

FLOATS = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
BLOCK = 32  # elements that share a scale


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one hidden row of a decoding step: launch latency
        dict(name="quantise one row", op="quantise", rows=1, cols=4096, dtype="bfloat16", pad=0),
        # activations inside a wider buffer, the last block of each row partial
        dict(name="quantise odd rows", op="quantise", rows=1001, cols=2053, dtype="float16", pad=3),
        # a model's output head, once when it is loaded
        dict(name="quantise a head", op="quantise", rows=131072, cols=4096, dtype="bfloat16",
             pad=0),
        # one stream, one token: the weights' bytes are all there is
        dict(name="head one token", op="head", rows=1, vocab=32768, cols=4096, dtype="bfloat16",
             pad=0),
        # a small batch, odd vocabulary, a last block of 8
        dict(name="head odd batch", op="head", rows=61, vocab=50021, cols=1000, dtype="float16",
             pad=5),
        # a full decoding batch
        dict(name="head decoding batch", op="head", rows=256, vocab=131072, cols=4096,
             dtype="bfloat16", pad=0),
        # a corpus piece of 4096 positions at once
        dict(name="head corpus", op="head", rows=4096, vocab=131072, cols=4096, dtype="bfloat16",
             pad=0),
        # one request with four beams: latency
        dict(name="beam one text", op="beam", texts=1, beams=4, vocab=32768, dtype="float32",
             pad=0, adjust=False),
        # a few texts under penalties and a grammar, odd vocabulary
        dict(name="beam constrained", op="beam", texts=6, beams=5, vocab=50021, dtype="float16",
             pad=3, adjust=True),
        # a serving batch
        dict(name="beam serving batch", op="beam", texts=32, beams=8, vocab=131072,
             dtype="bfloat16", pad=0, adjust=False),
        # a small model's keys and values, one request
        dict(name="reorder one text", op="reorder", texts=1, beams=4, layers=4, heads=4,
             positions=128, width=64, dtype="float16"),
        # two layers of a serving batch, texts of 512 to 1024 positions
        dict(name="reorder serving batch", op="reorder", texts=32, beams=8, layers=2, heads=8,
             positions=1024, width=128, dtype="bfloat16"),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "head", "beam", "reorder"])
    c = dict(op=op, dtype=rng.choice(sorted(FLOATS)))
    half = 2 if c["dtype"] == "float32" else 1  # no more bytes than the largest listed case
    if op == "quantise":
        c["pad"] = rng.choice([0, 0, 1, 3, 8])
        c["cols"] = _log_between(rng, 32, 4096)
        c["rows"] = _log_between(rng, 1, 131072 // half)
    elif op == "head":
        c["pad"] = rng.choice([0, 0, 1, 3, 8])
        c["vocab"] = _log_between(rng, 1000, 131072)
        c["cols"] = _log_between(rng, 64, 4096)
        c["rows"] = _log_between(rng, 1, 4096 // half)
    elif op == "beam":
        c["pad"] = rng.choice([0, 0, 1, 3, 8])
        c["vocab"] = _log_between(rng, 1000, 131072)
        c["beams"] = rng.randint(1, 16)
        c["texts"] = _log_between(rng, 1, max(1, 256 // half // c["beams"]))
        c["adjust"] = rng.random() < 0.5
        if c["adjust"]:
            c["texts"] = min(c["texts"], 16)
    else:
        c["beams"] = rng.randint(2, 8)
        c["texts"] = _log_between(rng, 1, 32 // half)
        c["layers"] = rng.randint(1, 2)
        c["heads"] = rng.randint(1, 8)
        c["positions"] = _log_between(rng, 16, 1024)
        c["width"] = rng.choice([40, 64, 80, 96, 128])
    return c


# ----------------------------------------------------------------- inputs --
def _wide(n, v, pad, dtype, fill=0.0):
    """Rows of v elements inside a buffer `pad` columns wider."""
    wide = torch.full((n, v + pad), fill, device="cuda", dtype=dtype)
    return wide[:, :v]


def _hidden(n, k, pad, dtype, g):
    """Activations: normal, with a few channels much larger than the others."""
    x = torch.randn(n, k, device="cuda", generator=g)
    loud = torch.rand(k, device="cuda", generator=g) < 0.01
    x *= torch.where(loud, 20.0, 1.0)
    out = _wide(n, k, pad, dtype)
    out.copy_(x)
    return out


def _weight(v, k, g):
    """A head's weights as bfloat16, each row with a size of its own."""
    w = torch.empty(v, k, device="cuda", dtype=torch.bfloat16)
    for at in range(0, v, 16384):
        n = min(16384, v - at)
        x = torch.randn(n, k, device="cuda", generator=g)
        w[at:at + n] = x * (torch.rand(n, 1, device="cuda", generator=g) + 0.5) / math.sqrt(k)
    return w


def _logits(n, v, pad, dtype, g):
    """Rows as a model's head gives them: a broad body and a few tokens that
    hold most of the mass."""
    x = torch.randn(n, v, device="cuda", generator=g).mul_(2.0)
    few = torch.randint(0, v, (n, 8), device="cuda", generator=g)
    x.scatter_add_(1, few, torch.rand(n, 8, device="cuda", generator=g) * 12.0)
    out = _wide(n, v, pad, dtype)
    out.copy_(x)
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = FLOATS[c["dtype"]]
    s = dict(case=c)
    if c["op"] == "quantise":
        s["x"] = _hidden(c["rows"], c["cols"], c["pad"], dtype, g)
    elif c["op"] == "head":
        s["hidden"] = _hidden(c["rows"], c["cols"], c["pad"], dtype, g)
        # the head as a checkpoint holds it: packed codes and a byte of scale
        # per block
        s["codes"], s["scales"] = _pack(_weight(c["vocab"], c["cols"], g))
        # its scales in the order in which a program that loads it lays them out
        s["blocked"] = _blocked(s["scales"])
    elif c["op"] == "beam":
        n, v = c["texts"] * c["beams"], c["vocab"]
        s["logits"] = _logits(n, v, c["pad"], dtype, g)
        s["scores"] = -30.0 * torch.rand(n, device="cuda", generator=g) - 5.0
        s["history"] = s["bias"] = s["mask"] = None
        if c["adjust"]:
            lens = torch.randint(100, 301, (n,), device="cuda", generator=g)
            end = torch.cumsum(lens, 0)
            r = torch.rand(int(lens.sum()), device="cuda", generator=g)
            s["history"] = ((r * r * r * v).to(torch.int32).clamp_(0, v - 1), end - lens, end)
            lens = torch.randint(12, 25, (n,), device="cuda", generator=g)
            end = torch.cumsum(lens, 0)
            ids = torch.randint(0, v, (int(lens.sum()),), device="cuda", generator=g)
            values = torch.randn(ids.numel(), device="cuda", generator=g) * 3.0
            s["bias"] = (ids.to(torch.int32), values, end - lens, end)
            words = (v + 31) // 32
            m = torch.randint(-2**31, 2**31, (2, n, words), device="cuda", generator=g)
            s["mask"] = (m[0] & m[1]).to(torch.int32)
    else:
        n = c["texts"] * c["beams"]
        shape = (n, c["heads"], c["positions"], c["width"])
        s["states"] = [torch.empty(shape, device="cuda", dtype=dtype).normal_(generator=g)
                       for _ in range(2 * c["layers"])]
        # half of the beams end and take over others' states; whoever goes on
        # stays where it is
        order = torch.rand(c["texts"], c["beams"], device="cuda", generator=g).argsort(1)
        stay = c["beams"] - c["beams"] // 2
        pick = torch.randint(0, stay, (c["texts"], c["beams"] // 2), device="cuda", generator=g)
        parents = torch.arange(c["beams"], device="cuda").repeat(c["texts"], 1)
        parents.scatter_(1, order[:, stay:], order.gather(1, pick))
        s["parents"] = parents.to(torch.int32)
        lo = c["positions"] // 2
        s["lengths"] = torch.randint(lo, c["positions"] + 1, (c["texts"],), device="cuda",
                                     generator=g).to(torch.int32)
    return s


# --------------------------------------- plain: microscaled 4-bit numbers --
def _blocks(x):
    """float32 [rows, blocks, 32], the last block padded with zeros."""
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[1] % BLOCK))
    return x.view(x.shape[0], -1, BLOCK)


def _scale_exponents(b):
    """floor(log2(largest magnitude)) - 2 of every block, not below -127."""
    top = b.abs().amax(2)
    e = torch.frexp(top).exponent - 3
    return torch.where(top > 0, e, -127).clamp(min=-127)


def _power(e):
    """2^e in float32 by its bits, for whole e from -127 to 127."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _code(a):
    """Index of the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; of two as near, the
    even index."""
    n = (a > 0.25).to(torch.int32)
    for t, tie in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                   (5.0, False)):
        n += (a >= t) if tie else (a > t)
    return n


def _magnitudes(n):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=n.device)[n]


def _plain_values(x):
    """float32 rows as 4-bit numbers stand for them."""
    b = _blocks(x)
    e = _scale_exponents(b)[:, :, None]
    v = _magnitudes(_code((b * _power(-e)).abs())) * _power(e)
    return torch.where(b < 0, -v, v).flatten(1)[:, :x.shape[1]]


def _pack(w):
    """(codes uint8 [rows, 16 * blocks], low half first; scale bytes uint8
    [rows, blocks]) of a matrix, a part of its rows at a time."""
    codes, scales = [], []
    for at in range(0, w.shape[0], 16384):
        b = _blocks(w[at:at + 16384])
        e = _scale_exponents(b)
        n = _code((b * _power(-e)[:, :, None]).abs()) + 8 * (b < 0)
        n = n.flatten(1).to(torch.uint8)
        codes.append(n[:, 0::2] | n[:, 1::2] << 4)
        scales.append((e + 127).to(torch.uint8))
    return torch.cat(codes), torch.cat(scales)


def _blocked(scales):
    """Scale bytes in tiles of 128 rows by 4 blocks: in a tile of 512 bytes,
    row r's four lie together at 16 (r mod 32) + 4 (r div 32)."""
    rows, blocks = scales.shape
    s = torch.nn.functional.pad(scales, (0, -blocks % 4, 0, -rows % 128))
    s = s.view(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4)
    return s.permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _unpack(codes, scales, cols):
    """float32 [rows, cols]."""
    n = torch.stack([codes & 15, codes >> 4], 2).flatten(1).to(torch.int32)
    v = _magnitudes(n & 7)
    v = torch.where(n >= 8, -v, v).view(n.shape[0], -1, BLOCK)
    e = scales.to(torch.int32) - 127
    return (v * _power(e)[:, :, None]).flatten(1)[:, :cols]


def _plain_head(s):
    h = _plain_values(s["hidden"])
    w = _unpack(s["codes"], s["scales"], h.shape[1])
    return (h @ w.T).to(s["hidden"].dtype)


# ------------------------------------------------------- plain: selection --
REPETITION, FREQUENCY, PRESENCE, TEMPERATURE = 1.1, 0.1, 0.3, 0.8


def _pairs(begin, end):
    """(row, position) of every entry of the rows' windows."""
    lens = end - begin
    rows = torch.repeat_interleave(torch.arange(lens.numel(), device=lens.device), lens)
    first = torch.cumsum(lens, 0) - lens
    at = torch.arange(rows.numel(), device=lens.device) - first[rows] + begin[rows]
    return rows, at


def _adjusted(s):
    """Penalised, biased, scaled and masked logits in 32 bits."""
    z = s["logits"].float()
    if not s["case"]["adjust"]:
        return z
    n, v = z.shape
    tokens, begin, end = s["history"]
    rows, at = _pairs(begin, end)
    count = torch.zeros(n * v, device=z.device)
    count.scatter_add_(0, rows * v + tokens[at], torch.ones(at.numel(), device=z.device))
    count = count.view(n, v)
    rho = torch.tensor(REPETITION, device=z.device)
    less = count * FREQUENCY + PRESENCE
    z = torch.where(count > 0, torch.where(z > 0, z / rho, z * rho) - less, z)
    ids, values, begin, end = s["bias"]
    rows, at = _pairs(begin, end)
    last = torch.full((n * v,), -1, dtype=torch.int64, device=z.device)  # the last entry counts
    last.scatter_reduce_(0, rows * v + ids[at], at, "amax")
    last = last.view(n, v)
    z = torch.where(last >= 0, z + values[last.clamp(min=0)], z)
    z = z * torch.tensor(1.0 / TEMPERATURE, device=z.device)
    bit = torch.arange(v, device=z.device)
    allowed = (s["mask"][:, bit >> 5] >> (bit & 31).to(torch.int32)) & 1
    return z.masked_fill(allowed == 0, -math.inf)


def _plain_beam(s):
    c = s["case"]
    x = _adjusted(s).double()  # candidates of two beams may be next to one another
    m = x.max(1, keepdim=True).values
    total = x - m - torch.exp(x - m).sum(1, keepdim=True).log() + s["scores"].double()[:, None]
    total = total.view(c["texts"], -1)
    best, at = torch.sort(total, dim=1, descending=True, stable=True)
    best, at = best[:, :2 * c["beams"]], at[:, :2 * c["beams"]]
    some = best > -math.inf
    tokens = torch.where(some, at % c["vocab"], -1)
    parents = torch.where(some, at // c["vocab"], -1)
    return best.float(), tokens.to(torch.int32), parents.to(torch.int32)


# ------------------------------------------------------ plain: reordering --
def _plain_reorder(s):
    c = s["case"]
    first = torch.arange(c["texts"], device="cuda")[:, None] * c["beams"]
    source = (s["parents"] + first).flatten()
    length = s["lengths"].repeat_interleave(c["beams"])
    live = torch.arange(c["positions"], device="cuda") < length[:, None]
    for x in s["states"]:
        x.copy_(torch.where(live[:, None, :, None], x[source], x))
    return s["states"]


# -------------------------------------------------------------------- run --
def _own(s):
    import rans_entropy_coding_b200 as rb
    c = s["case"]
    if c["op"] == "quantise":
        return rb.quantize_mxfp4(s["x"]).values(s["x"].dtype)
    if c["op"] == "head":
        return rb.mxfp4_logits(s["hidden"], rb.Mxfp4(s["codes"], s["blocked"], c["cols"]))
    if c["op"] == "beam":
        adjust = None
        if c["adjust"]:
            adjust = rb.LogitAdjust(temperature=TEMPERATURE, repetition=REPETITION,
                                    frequency=FREQUENCY, presence=PRESENCE, history=s["history"],
                                    bias=s["bias"], mask=s["mask"])
        return rb.beam_select(s["logits"], s["scores"], c["beams"], 2 * c["beams"], adjust)
    return rb.reorder_states(s["states"], s["parents"], s["lengths"], axis=2)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "quantise":
        return _plain_values(state["x"]).to(state["x"].dtype)
    if op == "head":
        return _plain_head(state)
    if op == "beam":
        return _plain_beam(state)
    return _plain_reorder(state)


def work(case):
    c = case
    e = FLOATS[c["dtype"]].itemsize
    if c["op"] == "quantise":
        n = c["rows"] * c["cols"]
        # 17 bytes a block, written and read again
        return {"bytes": n * 2 * e + n * 2 * 17 // BLOCK, "flops": 4 * n}
    if c["op"] == "head":
        n, v, k = c["rows"], c["vocab"], c["cols"]
        return {"bytes": v * k * 17 // BLOCK + n * k * e + n * v * e, "flops": 2 * n * v * k}
    if c["op"] == "beam":
        n, v = c["texts"] * c["beams"], c["vocab"]
        extra = n * (4 * ((v + 31) // 32) + 4 * 200 + 8 * 18 + 32) if c["adjust"] else 0
        return {"bytes": n * v * e + extra + 4 * n + 12 * 2 * n, "flops": 12 * n * v}
    moved = c["beams"] // 2
    stay = c["beams"] - moved
    sources = stay * (1.0 - (1.0 - 1.0 / stay) ** moved)  # that at least one beam takes over
    row = c["heads"] * c["positions"] * 3 // 4 * c["width"] * e
    return {"bytes": int(c["texts"] * 2 * c["layers"] * row * (moved + sources)), "flops": 0}


# ------------------------------------------------------------------ exact --
def _to_grid(x):
    """64-bit rows rounded to blocks of 4-bit numbers: steps of a half below 2,
    of one below 4, of two below 6."""
    n, k = x.shape
    out = torch.zeros(n, (k + BLOCK - 1) // BLOCK * BLOCK, dtype=torch.float64, device=x.device)
    out[:, :k] = x
    out = out.view(n, -1, BLOCK)
    _, e = torch.frexp(out.abs().amax(2, keepdim=True))
    unit = torch.pow(2.0, (e - 3).clamp(min=-127).double())
    a = (out / unit).abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    return (torch.sign(out) * a * unit).view(n, -1)[:, :k]


def exact(case, seed):
    """From the definitions in 64 bits."""
    c = case
    s = prepare(case, seed)
    if c["op"] == "quantise":
        return torch.cat([_to_grid(s["x"][at:at + 16384].double())
                          for at in range(0, c["rows"], 16384)])
    if c["op"] == "head":
        table = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        table = torch.tensor(table + [-t for t in table], dtype=torch.float64, device="cuda")
        h = _to_grid(s["hidden"].double())
        out = torch.empty(c["rows"], c["vocab"], dtype=torch.float64, device="cuda")
        for at in range(0, c["vocab"], 16384):
            codes = s["codes"][at:at + 16384].long()
            w = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device="cuda")
            w[:, ::2], w[:, 1::2] = table[codes % 16], table[codes // 16]
            unit = torch.pow(2.0, s["scales"][at:at + 16384].double() - 127)
            w *= unit.repeat_interleave(BLOCK, 1)
            out[:, at:at + 16384] = h @ w[:, :c["cols"]].T
        return out
    if c["op"] == "reorder":
        b = c["beams"]
        source, lengths = s["parents"].tolist(), s["lengths"].tolist()
        for x in s["states"]:
            for t in range(c["texts"]):
                mine = x[t * b:(t + 1) * b, :, :lengths[t]]
                mine.copy_(mine[source[t]].clone())
        return s["states"]
    x = s["logits"].double()
    if c["adjust"]:
        seen, begin, end = (t.tolist() for t in s["history"])
        ids, values, first, stop = (t.tolist() for t in s["bias"])
        for r in range(x.shape[0]):
            at, n = torch.unique(torch.tensor(seen[begin[r]:end[r]], device="cuda"),
                                 return_counts=True)
            y = x[r, at]
            y = y.clamp(max=0) * REPETITION + y.clamp(min=0) / REPETITION
            x[r, at] = y - PRESENCE - n.double() * FREQUENCY
            mine = dict(zip(ids[first[r]:stop[r]], values[first[r]:stop[r]]))
            at = torch.tensor(list(mine), device="cuda")
            x[r, at] += torch.tensor(list(mine.values()), dtype=torch.float64, device="cuda")
        x /= TEMPERATURE
        bits = torch.stack([s["mask"] >> b & 1 for b in range(32)], 2).flatten(1)
        x[bits[:, :c["vocab"]] == 0] = -math.inf
    total = torch.log_softmax(x, 1) + s["scores"].double()[:, None]
    # (the tokens and parents are whole numbers, which follow from the order)
    return total.view(c["texts"], -1).topk(2 * c["beams"], dim=1).values, None, None
