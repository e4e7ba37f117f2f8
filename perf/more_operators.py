"""Cases of the serving-step operators, with their plain forms.

The operators complete a decode step of a served llama-shaped layer whose
weights and caches are block-quantised: keys and values rotated, rounded to
4-bit blocks and stored into a paged cache (qmm_kv4_append, read back by
qmm_kv4_read), attention of a decode batch over that cache (qmm_attn_kv4), a
whole mixture-of-experts layer for a few tokens (qmm_moe), and the choice of
the next token from the output projection's logits (qmm_sample). Sizes are
those of the repository's Llama-7B-shaped layer (32 heads of 128, a vocabulary
of 32000), of its 8-KV-head cache and 8 x 14336 x 4096 expert examples, and
generic ones around them.

run() computes a case in elementary torch operations, in 32 bits (64 where a
border decides: codes, expert choices, cumulative probabilities), or, where
`own` is set, by the library's entry points. exact() is the definition in 64
bits, row by row.

A page of the cache holds `page` tokens of every KV head, head by head, in tiles
of 16 tokens: K codes, V codes [16][dim / 2 bytes], K scales, V scales, both fp16
[dim / 32][16]. Element e of token t's K is nibble e % 8 of dword
(16 (e % 32 / 8) + t) (dim / 32) + e / 32 of the tile's K codes, of its V nibble e
of its row. A value is d (code - 8).
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
Q4_0, Q8_0, Q4_K = 2, 8, 12
QTYPES = {"q4_0": Q4_0, "q8_0": Q8_0, "q4_K": Q4_K}
BLOCK = {"q4_0": (32, 18), "q8_0": (32, 34), "q4_K": (256, 144)}  # weights, bytes


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token of 8 key/value heads as the products leave it, pages of 16 tokens
        {"name": "append decode 1", "op": "append", "tokens": 1, "hkv": 8, "dim": 128, "rot": 128, "pairs": "halves",
         "norm": False, "page": 16, "x": "f32", "far": 30000},
        # an odd batch of normed heads of 64, rotated in part, fp16
        {"name": "append 333 partial", "op": "append", "tokens": 333, "hkv": 12, "dim": 64, "rot": 32,
         "pairs": "neighbours", "norm": True, "page": 32, "x": "f16", "far": 1000000},
        # a whole prompt batch
        {"name": "append 16384", "op": "append", "tokens": 16384, "hkv": 8, "dim": 128, "rot": 128, "pairs": "halves",
         "norm": True, "page": 64, "x": "f32", "far": 130000},
        # one conversation
        {"name": "attn 1 on 700", "op": "attn", "seqs": 1, "keys": 700, "hq": 32, "hkv": 8, "dim": 128, "page": 16,
         "type": "f16"},
        # a serving batch, ragged from an empty cache to 8000 tokens
        {"name": "attn 48 ragged 8000", "op": "attn", "seqs": 48, "keys": 8000, "hq": 32, "hkv": 8, "dim": 128,
         "page": 64, "type": "bf16"},
        # a few long documents, heads of 64, every query head with its own keys
        {"name": "attn 3 on 60000", "op": "attn", "seqs": 3, "keys": 60000, "hq": 16, "hkv": 16, "dim": 64, "page": 32,
         "type": "f16"},
        # the next token of one request
        {"name": "sample 1 of 32000", "op": "sample", "rows": 1, "vocab": 32000, "wide": 2.5, "x": "f32"},
        # a decode batch, every request with settings of its own
        {"name": "sample 64 of 32000", "op": "sample", "rows": 64, "vocab": 32000, "wide": 2.5, "x": "f32"},
        # a large vocabulary of an odd size, flat distributions
        {"name": "sample 37 of 130001", "op": "sample", "rows": 37, "vocab": 130001, "wide": 1.0, "x": "f32"},
        # one token through two of eight large experts
        {"name": "moe 1 of 8x14336", "op": "moe", "tokens": 1, "experts": 8, "used": 2, "ff": 14336, "k": 4096,
         "inner": "q4_0", "outer": "q4_0", "x": "f32"},
        # five tokens on many small experts, the down projection held more precisely
        {"name": "moe 5 of 64x1408", "op": "moe", "tokens": 5, "experts": 64, "used": 6, "ff": 1408, "k": 2048,
         "inner": "q4_0", "outer": "q8_0", "x": "f32"},
        # a decode batch on the large experts, k-quants, fp16 activations
        {"name": "moe 16 of 8x14336", "op": "moe", "tokens": 16, "experts": 8, "used": 2, "ff": 14336, "k": 4096,
         "inner": "q4_K", "outer": "q4_K", "x": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "sample", "moe"])
    if op == "append":
        dim = rng.choice([64, 128])
        return {"op": op, "tokens": _log(rng, 1, 12000), "hkv": rng.choice([1, 4, 8, 11]), "dim": dim,
                "rot": rng.choice([dim, dim // 2]), "pairs": rng.choice(["halves", "neighbours"]),
                "norm": rng.random() < 0.5, "page": rng.choice([16, 32, 64, 128]), "x": rng.choice(["f32", "f16", "bf16"]),
                "far": _log(rng, 1000, 1000000)}
    if op == "attn":
        hkv = rng.choice([1, 2, 8])
        seqs = _log(rng, 1, 64)
        return {"op": op, "seqs": seqs, "keys": _log(rng, 1, min(60000, 300000 // seqs)), "hq": hkv * rng.choice([1, 3, 4, 8]),
                "hkv": hkv, "dim": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128]),
                "type": rng.choice(["f16", "bf16"])}
    if op == "sample":
        return {"op": op, "rows": _log(rng, 1, 64), "vocab": _log(rng, 100, 70000), "wide": round(rng.uniform(0.5, 4.0), 2),
                "x": rng.choice(["f32", "f16", "bf16"])}
    experts = rng.choice([8, 16, 60])
    return {"op": op, "tokens": _log(rng, 1, 16), "experts": experts, "used": rng.randint(1, 6),
            "ff": 256 * rng.randint(2, 16), "k": 256 * rng.randint(2, 16), "inner": rng.choice(["q4_0", "q8_0", "q4_K"]),
            "outer": rng.choice(["q4_0", "q8_0", "q4_K"]), "x": rng.choice(["f32", "f16"])}


# --------------------------------------------------------------- inputs

def _own_lengths(cap, n):
    return [cap] if n == 1 else [cap * i // (n - 1) for i in range(n)]


def _page_bytes(page, hkv, dim):
    return hkv * page * dim * 9 // 8


def _cache(n_pages, c, gen):
    """A cache with keys and values in every place: codes like those of normal values, scales as their blocks have."""
    page, hkv, dim = c["page"], c["hkv"], c["dim"]
    pages = torch.empty(n_pages, hkv * page // 16, 18 * dim, dtype=torch.uint8, device="cuda")

    def codes(*shape):
        return (torch.randn(*shape, generator=gen, device="cuda") * 3.4 + 8.5).clamp_(0, 15).to(torch.uint8)

    for lo in range(0, n_pages, 1024):  # in parts, for the memory of the random numbers
        part = pages[lo:lo + 1024]
        shape = (*part.shape[:2], 16 * dim)
        part[..., :16 * dim] = codes(*shape) | codes(*shape) << 4
        d = 0.27 * (0.6 + 0.8 * torch.rand(*part.shape[:2], dim, generator=gen, device="cuda"))
        sign = torch.where(torch.rand(d.shape, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
        part[..., 16 * dim:] = (d * sign).half().view(torch.uint8)
    return pages.view(n_pages, -1)


def _weights(qtype, experts, rows, k, gen):
    """Random blocks whose weights have a standard deviation of about 1 / sqrt(k)."""
    n, size = BLOCK[qtype]
    w = torch.randint(0, 256, (experts, rows, k // n, size), generator=gen, device="cuda", dtype=torch.uint8)
    spread = 0.5 + torch.rand(experts, rows, k // n, 1, generator=gen, device="cuda")
    if qtype == "q4_0":
        w[..., :2] = (spread / (4.6 * math.sqrt(k))).half().view(torch.uint8)
    elif qtype == "q8_0":
        w[..., :2] = (spread / (74.0 * math.sqrt(k))).half().view(torch.uint8)
    else:
        d = spread / (32.0 * 8.0 * math.sqrt(k))
        w[..., :4] = torch.cat([d, 7.5 * d], -1).half().view(torch.uint8)
    return w.view(experts, rows, -1)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator("cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    s = {"case": c}
    if c["op"] == "append":
        n, dim, hkv, page = c["tokens"], c["dim"], c["hkv"], c["page"]
        s["k"], s["v"] = ((2.0 * normal(n, hkv, dim)).to(TYPES[c["x"]]) for _ in range(2))
        s["w"] = 1.0 + 0.2 * normal(dim) if c["norm"] else None
        s["positions"] = torch.randint(0, c["far"], (n,), generator=gen, device="cuda", dtype=torch.int32)
        # a model keeps this table on the host
        s["freqs"] = torch.tensor([10000.0 ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)], dtype=torch.float64)
        # consecutive tokens fill pages that lie anywhere, the first and the last in part
        n_pages = n // page + 2
        order = torch.randperm(n_pages + 3, generator=host)[:n_pages]
        at = torch.arange(n) + page // 3
        s["slots"] = (order[at // page] * page + at % page).to(torch.int32).cuda()
        s["cache"] = torch.zeros(n_pages + 3, _page_bytes(page, hkv, dim), dtype=torch.uint8, device="cuda")
        s["ko"], s["vo"] = (torch.zeros(n, hkv, dim, dtype=torch.float16, device="cuda") for _ in range(2))
    elif c["op"] == "attn":
        b, page = c["seqs"], c["page"]
        lens = _own_lengths(c["keys"], b)
        s["lens"] = [lens[i] for i in torch.randperm(b, generator=host).tolist()]
        width = -(-c["keys"] // page)
        used = [-(-x // page) for x in s["lens"]]
        order = torch.randperm(sum(used) + 2, generator=host).tolist()
        tables = torch.zeros(b, width, dtype=torch.int32)
        for i, m in enumerate(used):
            tables[i, :m] = torch.tensor(order[:m], dtype=torch.int32)
            order = order[m:]
        s["tables"] = tables.cuda()
        s["lengths"] = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
        s["cache"] = _cache(sum(used) + 2, c, gen)
        s["q"] = normal(b, c["hq"], c["dim"]).to(TYPES[c["type"]])
        s["o"] = torch.zeros_like(s["q"])
    elif c["op"] == "sample":
        n, vocab = c["rows"], c["vocab"]
        z = c["wide"] * normal(n, vocab)
        z += 6.0 * c["wide"] * uniform(n, 1) * (uniform(n, vocab) < 8.0 / vocab)  # a few likely tokens
        s["logits"] = z.to(TYPES[c["x"]])
        s["u"] = uniform(n)
        pick = uniform(4, n)
        s["temperature"] = torch.where(pick[0] < 0.1, 0.0, 0.5 + uniform(n))  # one request in ten is greedy
        s["top_k"] = torch.where(pick[1] < 0.4, 0, torch.randint(1, 200, (n,), generator=gen, device="cuda")).to(torch.int32)
        s["top_p"] = torch.where(pick[2] < 0.3, 1.0, 0.7 + 0.3 * uniform(n))
        s["min_p"] = torch.where(pick[3] < 0.5, 0.0, 0.1 * uniform(n))
        s["tokens"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["probs"] = torch.zeros(n, device="cuda")
    else:
        n, e, k, ff = c["tokens"], c["experts"], c["k"], c["ff"]
        s["x"] = normal(n, k).to(TYPES[c["x"]])
        s["router"] = normal(e, k) / math.sqrt(k)
        s["gate"], s["up"] = (_weights(c["inner"], e, ff, k, gen) for _ in range(2))
        s["down"] = _weights(c["outer"], e, k, ff, gen)
        s["y"] = torch.zeros(n, k, device="cuda")
        s["ids"] = torch.zeros(n, c["used"], dtype=torch.int32, device="cuda")
        s["weights"] = torch.zeros(n, c["used"], device="cuda")
    return s


def work(case):
    c = case
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if c["op"] == "append":
        values = 2 * c["tokens"] * c["hkv"] * c["dim"]  # read once, stored at 4.5 bits, and read back to fp16
        return {"bytes": values * (size[c["x"]] + 9 / 16 + 9 / 16 + 2) + 8 * c["tokens"], "flops": 10 * values}
    if c["op"] == "attn":
        keys = sum(_own_lengths(c["keys"], c["seqs"]))
        return {"bytes": keys * c["hkv"] * c["dim"] * 9 / 8 + 4 * c["seqs"] * c["hq"] * c["dim"],
                "flops": 4 * keys * c["hq"] * c["dim"]}
    if c["op"] == "sample":
        return {"bytes": c["rows"] * (c["vocab"] * size[c["x"]] + 28), "flops": 20 * c["rows"] * c["vocab"]}
    n, e, ff, k, used = c["tokens"], c["experts"], c["ff"], c["k"], c["used"]
    chosen = e * (1.0 - (1.0 - min(used, e) / e) ** n)  # different experts, on average
    per = {q: size / count for q, (count, size) in BLOCK.items()}
    return {"bytes": chosen * ff * k * (2 * per[c["inner"]] + per[c["outer"]]) + 4 * e * k + n * k * (4 + size[c["x"]]),
            "flops": 2 * n * (e * k + 3 * min(used, e) * ff * k)}


# ------------------------------------------------- the operators, plain

def _plain_heads(x, weight, positions, rot, pairs, eps=1e-6):
    """Norm and rotation, in 64 bits: a code is decided at a border."""
    x = x.double()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()
    freq = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=x.device) / rot)
    angle = positions.double()[:, None] * freq
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    head, rest = x[..., :rot], x[..., rot:]
    if pairs == "halves":
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1).float()
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1).float()


def _plain_codes(x):
    """The values that 4-bit blocks of x stand for."""
    blocks = x.float().unflatten(-1, (-1, 32))
    most = torch.gather(blocks, -1, blocks.abs().argmax(-1, keepdim=True))
    d = (most / -8.0).half().double()
    codes = torch.floor(torch.where(d == 0, 0.0, blocks.double() / d) + 8.5).clamp(0.0, 15.0)
    return (d * (codes - 8.0)).flatten(-2)


def _plain_append(s):
    c = s["case"]
    s["ko"].copy_(_plain_codes(_plain_heads(s["k"], s["w"], s["positions"], c["rot"], c["pairs"])))
    s["vo"].copy_(_plain_codes(s["v"]))
    return {"k": s["ko"], "v": s["vo"]}


def _plain_pages(pages, page, hkv, dim):
    """Keys and values of pages [..., bytes], each [..., page, hkv, dim] in 32 bits."""
    tiles = pages.unflatten(-1, (hkv, page // 16, 18 * dim))
    codes, scales = tiles[..., : 16 * dim], tiles[..., 16 * dim:].contiguous().view(torch.float16).float()
    codes = (torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8.0).unflatten(-1, (2, 16 * dim))
    k = codes.select(-2, 0).unflatten(-1, (4, 16, dim // 32, 8)).movedim(-4, -2)  # [..., token, block, 4, 8]
    v = codes.select(-2, 1).unflatten(-1, (16, dim // 32, 4, 8))
    scales = scales.unflatten(-1, (2, dim // 32, 16)).transpose(-1, -2)[..., None, None]  # [..., 2, token, block, 1, 1]
    # [..., hkv, tile, token, dim] to [..., page, hkv, dim]
    return tuple((x * scales.select(-5, i)).flatten(-3).flatten(-3, -2).transpose(-2, -3) for i, x in enumerate((k, v)))


def _plain_attn(s):
    c = s["case"]
    b, hkv, dim, g = c["seqs"], c["hkv"], c["dim"], c["hq"] // c["hkv"]
    k, v = (t.flatten(1, 2).transpose(1, 2) for t in _plain_pages(s["cache"][s["tables"].long()], c["page"], hkv, dim))
    q = s["q"].float().view(b, hkv, g, dim)
    w = torch.matmul(q, k.transpose(-1, -2).contiguous()) / math.sqrt(dim)
    hidden = torch.arange(w.shape[-1], device=q.device)[None, :] >= s["lengths"][:, None]
    w = w.masked_fill(hidden[:, None, None], float("-inf"))
    w = (w - w.amax(-1, keepdim=True).clamp_min(-3e38)).exp()
    o = torch.matmul(w, v.contiguous()) / w.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.view(b, c["hq"], dim).to(s["q"].dtype)


def _plain_sample(s):
    """In 64 bits: a token is decided at the border of two cumulative probabilities."""
    z, order = s["logits"].double().sort(dim=-1, descending=True, stable=True)
    place = torch.arange(z.shape[1], device=z.device)[None]
    t = s["temperature"].double()[:, None]
    w = torch.where(t > 0, ((z - z[:, :1]) / torch.where(t > 0, t, 1.0)).exp(), (place == 0).double())
    limit = torch.where(s["top_k"] > 0, s["top_k"], z.shape[1])[:, None]
    kept = torch.where(place < limit, w, 0.0)
    before = kept.cumsum(-1) - kept
    stay = (place < limit) & (before < s["top_p"].double()[:, None] * kept.sum(-1, keepdim=True))
    stay = stay & (w >= s["min_p"].double()[:, None])
    kept = torch.where(stay, w, 0.0)
    total = kept.sum(-1, keepdim=True)
    pick = (kept.cumsum(-1) <= s["u"].double()[:, None] * total).sum(-1, keepdim=True)
    pick = torch.minimum(pick, stay.sum(-1, keepdim=True) - 1)
    s["tokens"].copy_(order.gather(1, pick)[:, 0])
    s["probs"].copy_((w.gather(1, pick) / total)[:, 0])
    return {"tokens": s["tokens"], "probs": s["probs"]}


def _plain_weights(w, qtype):
    """Blocks [experts][rows][bytes] as 32-bit weights [experts][rows][k]."""
    blocks = w.unflatten(-1, (-1, BLOCK[qtype][1]))
    if qtype == "q8_0":
        return (blocks[..., :2].contiguous().view(torch.float16).float() * blocks[..., 2:].view(torch.int8).float()).flatten(-2)
    if qtype == "q4_0":
        d, q = blocks[..., :2].contiguous().view(torch.float16).float(), blocks[..., 2:]
        return (d * (torch.cat([q & 15, q >> 4], -1).float() - 8.0)).flatten(-2)
    d = blocks[..., :4].contiguous().view(torch.float16).float()
    low, mid, high = blocks[..., 4:8], blocks[..., 8:12], blocks[..., 12:16]
    scale = torch.cat([low & 63, (high & 15) | (low >> 6) << 4], -1).float() * d[..., :1]
    least = torch.cat([mid & 63, (high >> 4) | (mid >> 6) << 4], -1).float() * d[..., 1:]
    q = blocks[..., 16:].unflatten(-1, (4, 32))
    q = torch.stack([q & 15, q >> 4], -2).flatten(-3, -2).float()
    return (q * scale[..., None] - least[..., None]).flatten(-3)


def _plain_moe(s):
    """Every token through every expert, then its own experts' results."""
    c = s["case"]
    e, k, ff = c["experts"], c["k"], c["ff"]
    x = s["x"].float()
    logits = s["x"].double() @ s["router"].double().t().contiguous()
    share = (logits - logits.amax(-1, keepdim=True)).exp()
    share, ids = share.sort(dim=-1, descending=True, stable=True)
    share, ids = share[:, : c["used"]], ids[:, : c["used"]]
    share = (share / share.sum(-1, keepdim=True)).float()
    gate = (x @ _plain_weights(s["gate"], c["inner"]).view(e * ff, k).t()).view(-1, e, ff)
    up = (x @ _plain_weights(s["up"], c["inner"]).view(e * ff, k).t()).view(-1, e, ff)
    h = gate / (1.0 + (-gate).exp()) * up
    mine = torch.zeros(x.shape[0], e, device=x.device).scatter_(1, ids, share)
    h = (h * mine[..., None]).transpose(0, 1).contiguous()
    y = torch.matmul(h, _plain_weights(s["down"], c["outer"]).transpose(1, 2)).sum(0)
    return {"y": y, "ids": ids.to(torch.int32), "weights": share}


# ------------------------------------------- the operators, the library's

def _own(s):
    import block_quantized_matmul_amd as qmm
    c = s["case"]
    if c["op"] == "append":
        qmm.qmm_kv4_append(s["k"], s["v"], s["cache"], c["page"], s["slots"], positions=s["positions"], freqs=s["freqs"],
                           pairs=c["pairs"], norm=c["norm"], weight=s["w"], eps=1e-6)
        qmm.qmm_kv4_read(s["cache"], c["page"], s["slots"], K=s["ko"], V=s["vo"])
        return {"k": s["ko"], "v": s["vo"]}
    if c["op"] == "attn":
        return qmm.qmm_attn_kv4(s["q"], s["cache"], c["page"], c["hkv"], s["tables"], s["lengths"], O=s["o"])
    if c["op"] == "sample":
        qmm.qmm_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                       min_p=s["min_p"], tokens=s["tokens"], probs=s["probs"])
        return {"tokens": s["tokens"], "probs": s["probs"]}
    qmm.qmm_moe(s["x"], s["router"], s["gate"], s["up"], QTYPES[c["inner"]], s["down"], QTYPES[c["outer"]], c["used"],
                Y=s["y"], ids=s["ids"], weights=s["weights"])
    return {"y": s["y"], "ids": s["ids"], "weights": s["weights"]}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attn": _plain_attn, "sample": _plain_sample,
            "moe": _plain_moe}[state["case"]["op"]](state)


# ------------------------------------------------ the definitions, 64 bits

def _exact_codes(x):
    """Block by block: the scale that takes the largest element to code 0, the nearest code of every element."""
    x = x.float().double()
    out = torch.empty_like(x)
    for lo in range(0, x.shape[-1], 32):
        block = x[..., lo:lo + 32]
        high, low = block.amax(-1, keepdim=True), block.amin(-1, keepdim=True)
        # the first of the two where they are equally far from zero
        first = (block == high).double().argmax(-1, keepdim=True) < (block == low).double().argmax(-1, keepdim=True)
        most = torch.where((high > -low) | ((high == -low) & first), high, low)
        d = (most * -0.125).float().half().double()
        q = torch.floor(block / torch.where(d == 0, 1.0, d) + 0.5).clamp(-8, 7)
        out[..., lo:lo + 32] = torch.where(d == 0, 0.0, q * d)
    return out


def _exact_page_value(head, which, dim):
    """Keys (0) or values (1) of one head's tiles [pages][tiles][bytes], [pages][page][dim]."""
    codes = head[..., 8 * dim * which: 8 * dim * (which + 1)]
    d = head[..., dim * (16 + which): dim * (17 + which)].contiguous().view(torch.float16).double()
    out = torch.empty(*head.shape[:2], 16, dim, dtype=torch.float64, device=head.device)
    for t in range(16):
        for e in range(dim):
            if which == 0:
                nibble = ((e % 32 // 8 * 16 + t) * (dim // 32) + e // 32) * 8 + e % 8
            else:
                nibble = t * dim + e
            out[..., t, e] = ((codes[..., nibble // 2] >> 4 * (nibble % 2) & 15).double() - 8.0) * d[..., e // 32 * 16 + t]
    return out.flatten(1, 2)


def _exact_weights(w, qtype):
    """One expert's blocks [rows][bytes] in 64 bits."""
    count, size = BLOCK[qtype]
    b = w.view(w.shape[0], -1, size)
    out = torch.empty(*b.shape[:2], count, dtype=torch.float64, device=w.device)
    half = [b[..., i:i + 2].contiguous().view(torch.float16).double() for i in (0, 2)]
    if qtype == "q8_0":
        out[:] = half[0] * b[..., 2:].view(torch.int8)
    elif qtype == "q4_0":
        for j in range(16):
            out[..., j] = half[0][..., 0] * ((b[..., 2 + j] & 15).double() - 8)
            out[..., j + 16] = half[0][..., 0] * ((b[..., 2 + j] >> 4).double() - 8)
    else:
        for j in range(8):
            if j < 4:
                scale, least = b[..., 4 + j] & 63, b[..., 8 + j] & 63
            else:
                scale = (b[..., 8 + j] & 15) + 16 * (b[..., j] >> 6)
                least = (b[..., 8 + j] >> 4) + 16 * (b[..., 4 + j] >> 6)
            q = b[..., 16 + 32 * (j // 2): 48 + 32 * (j // 2)] >> 4 * (j % 2) & 15
            out[..., 32 * j:32 * j + 32] = half[0] * scale[..., None] * q - half[1] * least[..., None]
    return out.view(w.shape[0], -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "append":
        rot, k = c["rot"], s["k"].double()
        if c["norm"]:
            k = k / (k.pow(2).sum(-1, keepdim=True) / c["dim"] + 1e-6).sqrt() * s["w"].double()
        y = k.clone()
        for i in range(rot // 2):
            j, m = (i, i + rot // 2) if c["pairs"] == "halves" else (2 * i, 2 * i + 1)
            turn = (s["positions"].double() * 10000.0 ** (-2.0 * i / rot))[:, None]
            y[..., j] = k[..., j] * turn.cos() - k[..., m] * turn.sin()
            y[..., m] = k[..., m] * turn.cos() + k[..., j] * turn.sin()
        return {"k": _exact_codes(y), "v": _exact_codes(s["v"])}
    if c["op"] == "attn":
        g, dim, page = c["hq"] // c["hkv"], c["dim"], c["page"]
        heads = s["cache"].view(-1, c["hkv"], page // 16, 18 * dim)
        o = torch.zeros(c["seqs"], c["hq"], dim, dtype=torch.float64, device="cuda")
        for h in range(c["hkv"]):
            k, v = (_exact_page_value(heads[:, h], i, dim) for i in (0, 1))
            for i, n in enumerate(s["lens"]):
                mine = s["tables"][i, : -(-n // page)].long()
                if n:
                    w = s["q"][i, h * g:h * g + g].double() @ k[mine].view(-1, dim)[:n].t().contiguous()
                    o[i, h * g:h * g + g] = torch.softmax(w / math.sqrt(dim), -1) @ v[mine].view(-1, dim)[:n]
        return o
    if c["op"] == "sample":
        tokens, probs = [], []
        for i in range(c["rows"]):
            z = s["logits"][i].double()
            t, u, keep = float(s["temperature"][i]), float(s["u"][i]), int(s["top_k"][i])
            if t == 0:
                tokens.append(int((z == z.max()).nonzero()[0, 0]))
                probs.append(1.0)
                continue
            order = torch.argsort(-z, stable=True)
            p = torch.softmax(z[order] / t, 0)
            p = p[:keep] if keep > 0 else p
            p = p / p.sum()
            enough = (p.cumsum(0) >= float(s["top_p"][i])).nonzero()
            n = min(int(enough[0, 0]) + 1 if len(enough) else len(p), int((p >= float(s["min_p"][i]) * p[0]).sum()))
            p = p[:n] / p[:n].sum()
            at = (p.cumsum(0) > u).nonzero()
            at = int(at[0, 0]) if len(at) else n - 1
            tokens.append(int(order[at]))
            probs.append(float(p[at]))
        return {"tokens": torch.tensor(tokens, dtype=torch.int32, device="cuda"),
                "probs": torch.tensor(probs, dtype=torch.float64, device="cuda")}
    p = torch.softmax(s["x"].double() @ s["router"].double().t().contiguous(), -1)
    ids = torch.argsort(-p, dim=-1, stable=True)[:, : c["used"]]
    weights = p.gather(1, ids)
    weights = weights / weights.sum(-1, keepdim=True)
    y = torch.zeros(c["tokens"], c["k"], dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        row, slot = (ids == e).nonzero(as_tuple=True)
        if len(row):
            x = s["x"][row].double()
            gate, up = (x @ _exact_weights(s[name][e], c["inner"]).t().contiguous() for name in ("gate", "up"))
            h = gate * torch.sigmoid(gate) * up
            y[row] += weights[row, slot, None] * (h @ _exact_weights(s["down"][e], c["outer"]).t().contiguous())
    return {"y": y, "ids": ids.to(torch.int32), "weights": weights}
