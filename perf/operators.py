"""Cases for the operators over a TQ4_1S key/value cache: rotary positions,
quantising keys and values into the paged cache and reading them back,
attention of drafted token trees (and of single tokens) over the cache, and
moving an accepted branch's records together.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits), or with ``own`` set through the library's entry points.  ``exact``
computes the same from the definitions in 64 bits.

The cache: codes uint8 [pages, 2, kv_heads, page_size, D/2] and scales (fp16
bit patterns) int16 [pages, 2, kv_heads, page_size, D/16], keys in plane 0,
values in plane 1; token ``p`` of sequence ``b`` lies in page
``page_table[b, p // page_size]`` at row ``p % page_size``.  A record holds the
codec's codes of the head's D values in order (element 2i in the low nibble of
byte i) and two scales per 32-element block.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# The codec's tables: the 16-level Lloyd-Max quantiser of N(0, 1).
CENTROIDS = [0.128395036, 0.388048291, 0.656759143, 0.942340434, 1.25623119, 1.6180464, 2.06901717, 2.73258948]
THRESHOLDS = [0.258221656, 0.522403717, 0.799549758, 1.09928584, 1.4371388, 1.84353185, 2.40080333]
SCALE_MAX = 23968.0  # a cache record's scales saturate here


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # rotary: one token for each of 64 sequences far into long contexts; a whole prompt with
        # a partial, interleaved rotation as it leaves a product in fp32
        {"name": "rope decode", "op": "rope", "tokens": 64, "heads": 32, "dim": 128, "rot": 128, "type": "bf16",
         "interleaved": False, "theta": 500000.0, "far": 1000000},
        {"name": "rope prompt f32 partial", "op": "rope", "tokens": 8191, "heads": 32, "dim": 128, "rot": 64,
         "type": "f32", "interleaved": True, "theta": 10000.0, "far": 32768},
        # cache write and read-back: one step of 64 sequences (fp32 out of the products, keys
        # rotated on the way in); a long prompt in bf16; odd head dimension and small pages
        {"name": "cache step", "op": "cache", "tokens": 64, "batch": 64, "kv_heads": 8, "dim": 128, "page": 64,
         "type": "f32", "out": "bf16", "rope": True},
        {"name": "cache prompt", "op": "cache", "tokens": 16384, "batch": 4, "kv_heads": 8, "dim": 128, "page": 64,
         "type": "bf16", "out": "bf16", "rope": True},
        {"name": "cache odd", "op": "cache", "tokens": 1237, "batch": 3, "kv_heads": 3, "dim": 96, "page": 16,
         "type": "f16", "out": "f16", "rope": False},
        # attention: a single stream's token; a serving batch of ragged contexts; a small tree per
        # sequence; odd heads, small pages, chain of 5; the largest tree over a long context
        {"name": "attend token", "op": "attend", "batch": 1, "context": 1000, "ragged": False, "tree": 1,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "type": "bf16", "chain": True},
        {"name": "attend batch", "op": "attend", "batch": 64, "context": 8000, "ragged": True, "tree": 1,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "type": "bf16", "chain": True},
        {"name": "attend odd chain", "op": "attend", "batch": 5, "context": 2777, "ragged": True, "tree": 5,
         "heads": 6, "kv_heads": 2, "dim": 64, "page": 16, "type": "f16", "chain": True},
        {"name": "attend small trees", "op": "attend", "batch": 16, "context": 4000, "ragged": True, "tree": 16,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "type": "bf16", "chain": False},
        {"name": "attend large trees", "op": "attend", "batch": 4, "context": 16384, "ragged": False, "tree": 64,
         "heads": 64, "kv_heads": 8, "dim": 128, "page": 128, "type": "bf16", "chain": False},
        # commit: an accepted branch of one stream, and of a serving batch, over 32 layers
        {"name": "commit stream", "op": "commit", "layers": 32, "batch": 1, "tree": 16, "accepted": 5,
         "kv_heads": 8, "dim": 128, "page": 64},
        {"name": "commit batch", "op": "commit", "layers": 32, "batch": 64, "tree": 64, "accepted": 8,
         "kv_heads": 8, "dim": 128, "page": 64},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "cache", "attend", "attend", "commit"))
    kv = rng.choice((1, 2, 3, 4, 8))
    page = rng.choice((16, 32, 64, 128))
    if op == "rope":
        dim = rng.choice((64, 96, 128, 256))
        return {"op": op, "tokens": _spread(rng, 1, 4000), "heads": rng.randint(1, 64), "dim": dim,
                "rot": rng.choice((dim, dim // 2, dim - 6)), "type": rng.choice(("f32", "bf16", "f16")),
                "interleaved": rng.random() < 0.5, "theta": rng.choice((10000.0, 500000.0)),
                "far": _spread(rng, 100, 1000000)}
    if op == "cache":
        return {"op": op, "tokens": _spread(rng, 1, 12000), "batch": rng.randint(1, 8), "kv_heads": kv,
                "dim": rng.choice((32, 64, 96, 128)), "page": page, "type": rng.choice(("f32", "bf16", "f16")),
                "out": rng.choice(("bf16", "f16")), "rope": rng.random() < 0.5}
    if op == "commit":
        tree = rng.randint(2, 64)
        return {"op": op, "layers": rng.randint(1, 32), "batch": _spread(rng, 1, 48), "tree": tree,
                "accepted": rng.randint(1, min(tree, 10)), "kv_heads": kv, "dim": rng.choice((64, 96, 128)),
                "page": page}
    tree = rng.choice((1, 1, 2, 3, 7, 12, 24, 40, 64))
    return {"op": op, "batch": _spread(rng, 1, 32), "context": _spread(rng, 1, 9000), "ragged": rng.random() < 0.7,
            "tree": tree, "heads": kv * rng.choice((1, 3, 4, 6, 8)), "kv_heads": kv,
            "dim": rng.choice((64, 128)) if tree > 7 else rng.choice((64, 96, 128, 256)), "page": page,
            "type": rng.choice(("bf16", "f16")), "chain": rng.random() < 0.4}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _randint(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def _records(g, shape, dim):
    """Random records as the codec writes them for Gaussian data: (codes, scales)."""
    y = _randn(g, *shape, dim // 16, 16)
    y *= 4.0 + 4.0 * torch.rand(*shape, dim // 16, 1, generator=g, device=DEV)
    d = y.square().mean(-1).sqrt().half()
    t = torch.tensor(THRESHOLDS, device=DEV)
    code = torch.bucketize(y.abs() / d.float()[..., None], t).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
    code = code.view(*shape, dim // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), d.view(torch.int16)


def _filled_cache(g, pages, kv_heads, page, dim):
    codes = torch.empty(pages, 2, kv_heads, page, dim // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(pages, 2, kv_heads, page, dim // 16, dtype=torch.int16, device=DEV)
    step = max(1, (1 << 25) // (2 * kv_heads * page * dim))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        codes[i:i + n], scales[i:i + n] = _records(g, (n, 2, kv_heads, page), dim)
    return codes, scales


def _page_table(g, batch, per_sequence):
    order = torch.randperm(batch * per_sequence, generator=g, device=DEV).to(torch.int32)
    return order.view(batch, per_sequence).contiguous()


def _frequencies(rot, theta):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (theta ** (-2.0 * i / rot)).float().to(DEV)


def _parents(g, batch, tree, chain):
    """A tree for each sequence: a node's parent is an earlier node, or -1 for the context."""
    i = torch.arange(tree, device=DEV)
    if chain:
        return (i - 1).to(torch.int32).expand(batch, tree).contiguous()
    r = torch.rand(batch, tree, generator=g, device=DEV)
    return ((r * (i + 1)).floor().to(torch.int32) - 1).clamp_(max=(i - 1).to(torch.int32)).contiguous()


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    if c["op"] == "rope":
        c["x"] = _randn(g, c["tokens"], c["heads"], c["dim"]).to(DTYPES[c["type"]])
        c["positions"] = _randint(g, 0, c["far"], c["tokens"])
        c["inv_freq"] = _frequencies(c["rot"], c["theta"])
    elif c["op"] == "cache":
        n, B, page = c["tokens"], c["batch"], c["page"]
        per = -(-(-(-n // B)) // page) + 1
        c["page_table"] = _page_table(g, B, per)
        c["codes"] = torch.zeros(B * per, 2, c["kv_heads"], page, c["dim"] // 2, dtype=torch.uint8, device=DEV)
        c["scales"] = torch.zeros(B * per, 2, c["kv_heads"], page, c["dim"] // 16, dtype=torch.int16, device=DEV)
        i = torch.arange(n, device=DEV, dtype=torch.int32)
        c["seqs"] = i % B
        c["places"] = i // B + 3  # behind what the sequence holds already
        shape = (n, c["kv_heads"], c["dim"])
        channel = 1.0 + 7.0 * (torch.rand(c["kv_heads"], c["dim"], generator=g, device=DEV) < 0.02)
        c["k"] = (_randn(g, *shape) * channel).to(DTYPES[c["type"]])  # keys have a few large channels
        c["v"] = _randn(g, *shape).to(DTYPES[c["type"]])
        c["positions"] = c["places"] + _randint(g, 0, 100000, B)[c["seqs"].long()]
        c["inv_freq"] = _frequencies(c["dim"], 500000.0)
    elif c["op"] == "attend":
        B, T, page = c["batch"], c["tree"], c["page"]
        low = max(1, c["context"] // 8) if c["ragged"] else c["context"]
        c["lens"] = _randint(g, low, c["context"] + 1, B)
        per = -(-(c["context"] + T) // page)
        c["page_table"] = _page_table(g, B, per)
        c["codes"], c["scales"] = _filled_cache(g, B * per, c["kv_heads"], page, c["dim"])
        c["parents"] = _parents(g, B, T, c["chain"])
        c["q"] = (2.0 * _randn(g, B, T, c["heads"], c["dim"])).to(DTYPES[c["type"]])
        c["scale"] = c["dim"] ** -0.5
    else:
        B, page, per = c["batch"], c["page"], 2 + -(-c["tree"] // c["page"])
        c["lens"] = _randint(g, 0, page, B)
        c["page_table"] = _page_table(g, B, per)
        codes, scales = _filled_cache(g, c["layers"] * B * per, c["kv_heads"], page, c["dim"])
        c["codes"] = codes.view(c["layers"], B * per, *codes.shape[1:])
        c["scales"] = scales.view(c["layers"], B * per, *scales.shape[1:])
        branch = torch.rand(B, c["tree"], generator=g, device=DEV).argsort(1)[:, :c["accepted"]].sort(1).values
        count = _randint(g, 1, c["accepted"] + 1, B)
        at = torch.arange(c["accepted"], device=DEV)
        c["path"] = torch.where(at < count[:, None], branch, -1).to(torch.int32).contiguous()
    return c


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _signs(dim):
    """The codec's sign of each column: a multiplicative hash with one mixing round, bit 31."""
    h = (torch.arange(dim, device=DEV) * 0x9E3779B9) & 0xFFFFFFFF
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = h ^ (h >> 13)
    return 1.0 - 2.0 * (h >> 31).float()


def _hadamard():
    i = torch.arange(32, device=DEV)
    x = i[:, None] & i
    x = x ^ (x >> 4)
    x = x ^ (x >> 2)
    x = x ^ (x >> 1)
    return 1.0 - 2.0 * (x & 1).float()


def _transform(x, signs_first):
    """H (s . x) per 32-block, or s . (H x)."""
    s = _signs(x.shape[-1]).to(x.dtype)
    y = x * s if signs_first else x
    y = (y.reshape(*x.shape[:-1], -1, 32) @ _hadamard().to(x.dtype)).reshape(x.shape)
    return y if signs_first else y * s


def _encode(x):
    """Codes and scale bit patterns of records x [..., D]."""
    y = _transform(x.float(), True)
    y = y.view(*x.shape[:-1], -1, 16)
    d = y.square().mean(-1).sqrt().clamp(max=SCALE_MAX).half()
    a, df = y.abs(), d.float()[..., None]
    rank = sum((a > t * df).to(torch.uint8) for t in THRESHOLDS)
    code = (rank | ((y < 0).to(torch.uint8) << 3)).view(*x.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), d.view(torch.int16)


def _decode(codes, scales):
    table = torch.tensor(CENTROIDS + [-v for v in CENTROIDS], device=DEV)
    pair = torch.stack((codes & 15, codes >> 4), -1)
    c = table[pair.view(*codes.shape[:-1], -1, 16).int()]
    c = c * scales.view(torch.float16).float()[..., None]
    return _transform(c.flatten(-2), False) * 0.03125


def _rotate(x, positions, inv_freq, interleaved):
    angle = positions.double()[:, None] * inv_freq.double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = 2 * inv_freq.numel()
    head, rest = x[..., :r].float(), x[..., r:].float()
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = head[..., :r // 2], head[..., r // 2:]
        head = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((head, rest), -1)


def _slots(s, seqs, places):
    page = s["page"]
    return s["page_table"][seqs.long(), (places // page).long()].long(), (places % page).long()


def _plain_cache(s):
    k = _rotate(s["k"], s["positions"], s["inv_freq"], False) if s["rope"] else s["k"].float()
    codes, scales = _encode(torch.stack((k, s["v"].float()), 1))
    page, row = _slots(s, s["seqs"], s["places"])
    s["codes"][page, :, :, row] = codes
    s["scales"][page, :, :, row] = scales
    x = _decode(s["codes"][page, :, :, row], s["scales"][page, :, :, row]).to(DTYPES[s["out"]])
    return x[:, 0], x[:, 1]


def _ancestors(parents):
    """[B, T, T]: whether node i sees node j (itself or an ancestor), by squaring the parent relation."""
    T = parents.shape[1]
    i = torch.arange(T, device=DEV)
    reach = ((parents[:, :, None] == i) | (i[:, None] == i)).float()
    hops = 1
    while hops < T:
        reach = ((reach @ reach) > 0).float()
        hops *= 2
    return reach > 0


def _plain_attend(s):
    B, T, H, D = s["q"].shape
    kv = s["kv_heads"]
    n = s["page_table"].shape[1] * s["page"]
    x = _decode(s["codes"][s["page_table"].long()], s["scales"][s["page_table"].long()])
    x = x.permute(2, 0, 3, 1, 4, 5).reshape(2, B, kv, n, D)
    q = s["q"].float().view(B, T, kv, H // kv, D).permute(0, 2, 1, 3, 4).reshape(B, kv, -1, D)
    scores = (q @ x[0].transpose(-1, -2)).mul_(s["scale"]).view(B, kv, T, H // kv, n)
    j = torch.arange(n, device=DEV) - s["lens"][:, None]  # the tree's own numbering
    drafted = torch.gather(_ancestors(s["parents"]), 2, j.clamp(0, T - 1)[:, None].expand(B, T, n))
    seen = (j < 0)[:, None] | ((j < T)[:, None] & drafted)
    scores.masked_fill_(~seen[:, None, :, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True)
    p = scores.exp_()
    o = (p.view(B, kv, -1, n) @ x[1]).view(B, kv, T, H // kv, D) / p.sum(-1, keepdim=True)
    return o.permute(0, 2, 1, 3, 4).reshape(B, T, H, D).to(s["q"].dtype)


def _plain_commit(s):
    B, P = s["path"].shape
    seqs = torch.arange(B, device=DEV).repeat_interleave(P)
    lens = s["lens"].repeat_interleave(P)
    path, at = s["path"].view(-1), torch.arange(P, device=DEV, dtype=torch.int32).repeat(B)
    at = torch.where(path < 0, 0, at)  # past the branch's end: the first record's move again
    path = torch.where(path < 0, s["path"][:, :1].expand(B, P).reshape(-1), path)
    page, row = _slots(s, seqs, lens + path)
    to_page, to_row = _slots(s, seqs, lens + at)
    codes = s["codes"].permute(1, 4, 0, 2, 3, 5)  # [pages, page_size, layers, 2, kv_heads, bytes]
    scales = s["scales"].permute(1, 4, 0, 2, 3, 5)
    codes[to_page, to_row] = codes[page, row]
    scales[to_page, to_row] = scales[page, row]
    return s["codes"], s["scales"]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    s = state
    if own:
        import dequant_gemv_tq4_b200 as tq
        if s["op"] == "rope":
            return tq.rope(s["x"], s["positions"], s["inv_freq"], interleaved=s["interleaved"])
        if s["op"] == "cache":
            rope = (s["positions"], s["inv_freq"]) if s["rope"] else None
            tq.kv_append(s["codes"], s["scales"], s["page_table"], s["seqs"], s["places"], s["k"], s["v"], rope=rope)
            return tq.kv_read(s["codes"], s["scales"], s["page_table"], s["seqs"], s["places"],
                              dtype=DTYPES[s["out"]])
        if s["op"] == "attend":
            return tq.kv_attention(s["codes"], s["scales"], s["page_table"], s["lens"], s["q"],
                                   parents=s["parents"], scale=s["scale"])
        tq.kv_commit(s["codes"], s["scales"], s["page_table"], s["lens"], s["path"])
        return s["codes"], s["scales"]
    if s["op"] == "rope":
        return _rotate(s["x"], s["positions"], s["inv_freq"], s["interleaved"]).to(s["x"].dtype)
    if s["op"] == "cache":
        return _plain_cache(s)
    if s["op"] == "attend":
        return _plain_attend(s)
    return _plain_commit(s)


def _tokens(case):
    """The mean number of context tokens of a sequence."""
    c = case["context"]
    return (max(1, c // 8) + c) / 2 if case["ragged"] else c


def work(case):
    c = case
    record = c["dim"] // 2 + c["dim"] // 8
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": 2 * n * (4 if c["type"] == "f32" else 2), "flops": 3 * c["tokens"] * c["heads"] * c["rot"]}
    if c["op"] == "cache":
        n = 2 * c["tokens"] * c["kv_heads"]
        size = 4 if c["type"] == "f32" else 2
        return {"bytes": n * (c["dim"] * (size + 2) + 2 * record), "flops": n * c["dim"] * 2 * 14}
    if c["op"] == "attend":
        n = _tokens(c) + c["tree"]
        rows = c["batch"] * c["tree"] * c["heads"]
        return {"bytes": c["batch"] * n * c["kv_heads"] * 2 * record + rows * c["dim"] * 4,
                "flops": 4 * rows * n * c["dim"]}
    moved = c["layers"] * c["batch"] * (c["accepted"] + 1) / 2 * 2 * c["kv_heads"]
    return {"bytes": 2 * moved * record, "flops": 0}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_block():
    """[32, 32] fp64: entry (i, j) of Sylvester's Hadamard matrix by doubling."""
    h = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    for _ in range(5):
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)))
    return h


def _exact_signs(dim):
    s = []
    for k in range(dim):
        h = k * 0x9E3779B9 % 2 ** 32
        h = (h ^ h >> 16) * 0x85EBCA6B % 2 ** 32
        s.append(-1.0 if (h ^ h >> 13) >= 2 ** 31 else 1.0)
    return torch.tensor(s, dtype=torch.float64, device=DEV)


def _exact_values(codes, scales, dim):
    """Records [n, D/2], [n, D/16] to their values [n, D]."""
    level = torch.tensor([(1 - 2 * (c >> 3)) * CENTROIDS[c & 7] for c in range(16)], device=DEV).double()
    c = torch.empty(codes.shape[0], dim, dtype=torch.float64, device=DEV)
    c[:, 0::2], c[:, 1::2] = level[(codes % 16).long()], level[(codes // 16).long()]
    c *= scales.view(torch.float16).double().repeat_interleave(16, 1)
    return (c.view(-1, 32) @ _exact_block()).view(-1, dim) * _exact_signs(dim) / 32


def _exact_rotated(x, positions, inv_freq, interleaved):
    out = x.double().clone()
    z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                    torch.outer(positions.double(), inv_freq.double()))[:, None]
    half = inv_freq.numel()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    w = torch.complex(x[..., first].double(), x[..., second].double()) * z
    out[..., first], out[..., second] = w.real, w.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rope":
        return _exact_rotated(s["x"], s["positions"], s["inv_freq"], s["interleaved"])
    D = s["dim"]
    if s["op"] == "cache":
        found = []
        for x in (_exact_rotated(s["k"], s["positions"], s["inv_freq"], False) if s["rope"] else s["k"].double(),
                  s["v"].double()):
            y = ((x * _exact_signs(D)).view(-1, 32) @ _exact_block()).view(-1, 16)
            d = (y * y).mean(1).sqrt().half()
            codes = torch.zeros(y.shape, dtype=torch.uint8, device=DEV)
            for t in THRESHOLDS:
                codes += y.abs() > t * d.double()[:, None]
            codes += 8 * (y < 0)
            codes = codes.view(-1, D)
            codes = codes[:, 0::2] + 16 * codes[:, 1::2]
            found.append(_exact_values(codes, d.view(-1, D // 16), D).view(x.shape))
        return tuple(found)
    if s["op"] == "commit":
        return None
    B, T, H, _ = s["q"].shape
    G = H // s["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    parents = s["parents"].tolist()
    for b in range(B):
        n = int(s["lens"][b]) + T
        sees = torch.ones(T, n, dtype=torch.bool)
        for i in range(T):
            sees[i, n - T:] = False
            j = i
            while j >= 0:
                sees[i, n - T + j] = True
                j = parents[b][j]
        hidden = ~sees.to(DEV)
        pages = s["page_table"][b].long()
        for h in range(s["kv_heads"]):
            k, v = (_exact_values(s["codes"][pages, w, h].reshape(-1, D // 2)[:n],
                                  s["scales"][pages, w, h].reshape(-1, D // 16)[:n], D) for w in (0, 1))
            q = s["q"][b, :, h * G:(h + 1) * G].double()
            z = torch.einsum("tgd,nd->tgn", q, k) * s["scale"]
            p = torch.softmax(z.masked_fill(hidden[:, None], -math.inf), -1)
            out[b, :, h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", p, v)
    return out
