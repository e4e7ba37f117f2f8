"""Cases of the attention-block operators, with their plain forms.

The operators surround the MUL_MATs of a served llama-shaped layer: low-rank
adapters beside a projection (qmm_lora), norms and rotation of the heads on
their way into the cache (qmm_norm_rope), causal attention over packed prompts
(qmm_attn_prompt) and attention of a decode batch over a shared prefix and
each sequence's own cache (qmm_attn_shared). Sizes are those of the
repository's Llama-7B-shaped layer (4096 wide, 32 heads of 128, feed-forward
11008), of its 8-KV-head cache example, and generic ones around them.

run() computes a case in elementary torch operations in 32 bits, or, where
`own` is set, by the library's entry points. exact() is the definition in 64
bits, sequence by sequence.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of one request with a rank-16 adapter on a square projection
        {"name": "lora decode 1", "op": "lora", "tokens": 1, "requests": 1, "adapters": 8, "rank": 16, "k": 4096,
         "rows": 4096, "x": "f32"},
        # a decode batch: one token each of 64 requests on 32 adapters, some without, beside the gate or up product
        {"name": "lora decode 64", "op": "lora", "tokens": 64, "requests": 64, "adapters": 32, "rank": 16, "k": 4096,
         "rows": 11008, "x": "f32"},
        # the prompts of 9 requests in one batch, fp16 activations, rank 64, beside the down product
        {"name": "lora prompt 2048", "op": "lora", "tokens": 2048, "requests": 9, "adapters": 8, "rank": 64, "k": 11008,
         "rows": 4096, "x": "f16"},
        # one decoded token: 32 query heads and 8 key/value heads of 128 into a cache
        {"name": "norm_rope decode 1", "op": "norm_rope", "tokens": 1, "hq": 32, "hkv": 8, "dim": 128, "rot": 128,
         "pairs": "halves", "x": "f32", "out": "f16", "far": 30000},
        # an odd batch, fp16 heads of 64 rotated in part, neighbouring pairs, 12 heads each, bf16 results
        {"name": "norm_rope 333 partial", "op": "norm_rope", "tokens": 333, "hq": 12, "hkv": 12, "dim": 64, "rot": 32,
         "pairs": "neighbours", "x": "f16", "out": "bf16", "far": 1000000},
        # a whole prompt batch at fp32 as the products leave it
        {"name": "norm_rope 16384", "op": "norm_rope", "tokens": 16384, "hq": 32, "hkv": 8, "dim": 128, "rot": 128,
         "pairs": "halves", "x": "f32", "out": "f16", "far": 130000},
        # a few short prompts, one empty and one of one token
        {"name": "prompt 8 short", "op": "prompt", "tokens": 301, "seqs": 8, "behind": 19, "hq": 32, "hkv": 8, "dim": 128,
         "type": "f16"},
        # ragged prompts packed into one batch
        {"name": "prompt 16 ragged", "op": "prompt", "tokens": 8109, "seqs": 16, "behind": 83, "hq": 32, "hkv": 8,
         "dim": 128, "type": "f16"},
        # one long prompt, bf16
        {"name": "prompt 8192", "op": "prompt", "tokens": 8192, "seqs": 1, "behind": 0, "hq": 32, "hkv": 8, "dim": 128,
         "type": "bf16"},
        # heads of 64, every query head with its own keys
        {"name": "prompt 3 heads of 64", "op": "prompt", "tokens": 4001, "seqs": 3, "behind": 0, "hq": 16, "hkv": 16,
         "dim": 64, "type": "f16"},
        # a small batch on a short system prompt
        {"name": "shared 4 on 500", "op": "shared", "seqs": 4, "prefix": 500, "own": 130, "hq": 32, "hkv": 8, "dim": 128,
         "type": "f16"},
        # a serving batch on a long document, ragged own caches
        {"name": "shared 48 on 32000", "op": "shared", "seqs": 48, "prefix": 32000, "own": 2047, "hq": 32, "hkv": 8,
         "dim": 128, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "norm_rope", "prompt", "shared"])
    if op == "lora":
        tokens = _log(rng, 1, 2048)
        return {"op": op, "tokens": tokens, "requests": min(tokens, _log(rng, 1, 64)), "adapters": rng.randint(1, 16),
                "rank": rng.choice([4, 8, 16, 24, 32, 64]), "k": 32 * _log(rng, 8, 256), "rows": _log(rng, 100, 11008),
                "x": rng.choice(["f32", "f16"])}
    if op == "norm_rope":
        dim = rng.choice([64, 80, 128])
        hkv = rng.choice([1, 4, 8])
        return {"op": op, "tokens": _log(rng, 1, 8192), "hq": hkv * rng.randint(1, 5), "hkv": hkv, "dim": dim,
                "rot": rng.choice([dim, dim // 2]), "pairs": rng.choice(["halves", "neighbours"]),
                "x": rng.choice(["f32", "f16", "bf16"]), "out": rng.choice(["f16", "bf16", "f32"]),
                "far": _log(rng, 1000, 1000000)}
    hkv = rng.choice([1, 2, 8])
    hq = hkv * rng.choice([1, 3, 4])
    if op == "prompt":
        tokens = _log(rng, 40, 8000)
        return {"op": op, "tokens": tokens, "seqs": min(tokens, _log(rng, 1, 40)), "behind": rng.randint(0, 50), "hq": hq,
                "hkv": hkv, "dim": rng.choice([64, 128]), "type": rng.choice(["f16", "bf16"])}
    return {"op": op, "seqs": _log(rng, 1, 48), "prefix": _log(rng, 17, 32000), "own": _log(rng, 1, 2000), "hq": hq,
            "hkv": hkv, "dim": rng.choice([64, 128]), "type": rng.choice(["f16", "bf16"])}


# --------------------------------------------------------------- inputs

def _lengths(total, n):
    """n lengths of a packed batch that sum to total: growing shares, the first of several empty, the second one
    token."""
    if n == 1:
        return [total]
    share = [0 if i == 0 and n > 3 else i + 1 for i in range(n)]
    out = [total * s // sum(share) for s in share]
    if n > 3:
        out[1] = min(1, total)
    out[-1] += total - sum(out)
    return out


def _own_lengths(cap, n):
    return [cap] if n == 1 else [cap * i // (n - 1) for i in range(n)]


def _shuffled(values, gen):
    order = torch.randperm(len(values), generator=gen).tolist()
    return [values[i] for i in order]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator("cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    s = {"case": c}
    if c["op"] == "lora":
        n, k, r, rows, ad = c["tokens"], c["k"], c["rank"], c["rows"], c["adapters"]
        s["x"] = normal(n, k).to(TYPES[c["x"]])
        s["a"] = (normal(ad, r, k) / math.sqrt(k)).half()
        s["b"] = (normal(ad, rows, r) / math.sqrt(r)).half()
        s["scales"] = 0.5 + torch.rand(ad, generator=gen, device="cuda")
        s["base"] = normal(n, rows)
        # the tokens of a request stand together; about one request in ten has no adapter
        of = torch.randint(0, ad, (c["requests"],), generator=host)
        of[torch.rand(c["requests"], generator=host) < 0.1] = -1
        lens = _shuffled(_lengths(n, c["requests"]) if n > c["requests"] else [1] * n, host)
        s["ids"] = torch.repeat_interleave(of, torch.tensor(lens)).to(torch.int32).cuda()
        s["y"] = torch.zeros(n, rows, device="cuda")
    elif c["op"] == "norm_rope":
        n, dim, hq, hkv = c["tokens"], c["dim"], c["hq"], c["hkv"]
        slots = 2 * n + 3  # the cache is larger than the batch; the new rows lie anywhere in it
        out = TYPES[c["out"]]
        for name, h in (("q", hq), ("k", hkv), ("v", hkv)):
            s[name] = (2.0 * normal(n, h, dim)).to(TYPES[c["x"]])
        s["wq"], s["wk"] = 1.0 + 0.2 * normal(dim), 1.0 + 0.2 * normal(dim)
        s["positions"] = torch.randint(0, c["far"], (n,), generator=gen, device="cuda", dtype=torch.int32)
        # a model keeps this table on the host
        s["freqs"] = torch.tensor([10000.0 ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)], dtype=torch.float64)
        s["slots"] = torch.randperm(slots, generator=host)[:n].to(torch.int32).cuda()
        s["qo"] = torch.zeros(n, hq, dim, dtype=out, device="cuda")
        s["kc"] = torch.zeros(slots, hkv, dim, dtype=out, device="cuda")
        s["vc"] = torch.zeros(slots, hkv, dim, dtype=out, device="cuda")
    elif c["op"] == "prompt":
        n, dim, t = c["tokens"] + c["behind"], c["dim"], TYPES[c["type"]]
        s["q"] = normal(n, c["hq"], dim).to(t)
        kv = normal(n, 2, c["hkv"], dim).to(t)  # keys and values interleaved by token, as one product writes them
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        lens = _shuffled(_lengths(c["tokens"], c["seqs"]), host)
        s["lens"] = lens
        starts = [0]
        for x in lens:
            starts.append(starts[-1] + x)
        s["starts"] = ints(starts)
        s["o"] = torch.zeros(n, c["hq"], dim, dtype=t, device="cuda")
    else:
        b, dim, t = c["seqs"], c["dim"], TYPES[c["type"]]
        cap = (c["own"] + 63) // 64 * 64
        s["q"] = normal(b, c["hq"], dim).to(t)
        s["kp"], s["vp"] = normal(c["prefix"], c["hkv"], dim).to(t), normal(c["prefix"], c["hkv"], dim).to(t)
        s["k"], s["v"] = normal(b, cap, c["hkv"], dim).to(t), normal(b, cap, c["hkv"], dim).to(t)
        s["lens"] = _shuffled(_own_lengths(c["own"], b), host)
        s["lengths"] = ints(s["lens"])
        s["o"] = torch.zeros(b, c["hq"], dim, dtype=t, device="cuda")
    return s


def work(case):
    c = case
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if c["op"] == "lora":
        n, k, r, rows = c["tokens"], c["k"], c["rank"], c["rows"]
        used = min(c["adapters"], c["requests"])
        return {"bytes": n * k * size[c["x"]] + used * r * (k + rows) * 2 + 8 * n * rows + 4 * n,
                "flops": 2 * n * r * (k + rows)}
    if c["op"] == "norm_rope":
        heads = c["tokens"] * (c["hq"] + 2 * c["hkv"]) * c["dim"]
        return {"bytes": heads * (size[c["x"]] + size[c["out"]]) + 8 * c["tokens"], "flops": 8 * heads}
    if c["op"] == "prompt":
        pairs = sum(x * (x + 1) // 2 for x in _lengths(c["tokens"], c["seqs"]))
        return {"bytes": 4 * c["tokens"] * c["dim"] * (c["hq"] + c["hkv"]), "flops": 4 * pairs * c["hq"] * c["dim"]}
    own_tokens = sum(_own_lengths(c["own"], c["seqs"]))
    keys = c["prefix"] * c["seqs"] + own_tokens
    return {"bytes": 4 * c["dim"] * (c["seqs"] * c["hq"] + (c["prefix"] + own_tokens) * c["hkv"]),
            "flops": 4 * keys * c["hq"] * c["dim"]}


# ------------------------------------------------- the operators, plain

def _plain_lora(s):
    x, a, b = s["x"].float(), s["a"].float(), s["b"].float()
    ad, r, k = a.shape
    ids = s["ids"].long()
    # every token through every adapter, then its own kept
    v = (x @ a.reshape(ad * r, k).t()).view(-1, ad, r)
    keep = (ids[:, None] == torch.arange(ad, device=x.device)).float() * s["scales"]
    v = (v * keep[:, :, None]).reshape(-1, ad * r)
    return s["base"] + v @ b.permute(0, 2, 1).reshape(ad * r, -1)


def _plain_heads(x, weight, positions, rot, pairs, eps=1e-6):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight
    if positions is None:
        return x
    freq = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=x.device) / rot)
    angle = positions.double()[:, None] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    head, rest = x[..., :rot], x[..., rot:]
    if pairs == "halves":
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _plain_norm_rope(s):
    c, at = s["case"], s["slots"].long()
    s["qo"].copy_(_plain_heads(s["q"], s["wq"], s["positions"], c["rot"], c["pairs"]))
    s["kc"][at] = _plain_heads(s["k"], s["wk"], s["positions"], c["rot"], c["pairs"]).to(s["kc"].dtype)
    s["vc"][at] = s["v"].to(s["vc"].dtype)
    return {"q": s["qo"], "k": s["kc"], "v": s["vc"]}


def _plain_prompt(s):
    c, n = s["case"], s["case"]["tokens"]
    g, dim = c["hq"] // c["hkv"], c["dim"]
    q = s["q"][:n].float().permute(1, 0, 2).reshape(c["hkv"], g, n, dim)
    k = s["k"][:n].float().permute(1, 2, 0).contiguous()
    v = s["v"][:n].float().permute(1, 0, 2).contiguous()
    at = torch.arange(n, device=q.device)
    seq = torch.searchsorted(s["starts"].long(), at, right=True)
    hidden = (seq[:, None] != seq[None, :]) | (at[None, :] > at[:, None])
    p = torch.matmul(q.reshape(c["hkv"], g * n, dim), k).view(c["hkv"], g, n, n).mul_(1.0 / math.sqrt(dim))
    p.masked_fill_(hidden, float("-inf"))
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(c["hkv"], g * n, n), v).view(c["hkv"], g, n, dim) / total
    out = torch.zeros_like(s["o"])
    out[:n] = o.reshape(c["hq"], n, dim).permute(1, 0, 2).to(out.dtype)
    return out


def _plain_shared(s):
    c = s["case"]
    b, g, dim, hkv, cap = c["seqs"], c["hq"] // c["hkv"], c["dim"], c["hkv"], s["k"].shape[1]
    q = s["q"].float().view(b, hkv, g, dim)
    far = torch.matmul(q.permute(1, 0, 2, 3).reshape(hkv, b * g, dim), s["kp"].float().permute(1, 2, 0).contiguous())
    near = torch.matmul(q, s["k"].float().permute(0, 2, 3, 1).contiguous())
    far = far.view(hkv, b, g, -1).permute(1, 0, 2, 3) / math.sqrt(dim)
    near = near / math.sqrt(dim)
    hidden = torch.arange(cap, device=q.device)[None, :] >= s["lengths"][:, None]
    near = near.masked_fill(hidden[:, None, None], float("-inf"))
    top = torch.maximum(far.amax(-1, keepdim=True), near.amax(-1, keepdim=True))
    far, near = (far - top).exp(), (near - top).exp()
    total = far.sum(-1, keepdim=True) + near.sum(-1, keepdim=True)
    far = far.permute(1, 0, 2, 3).reshape(hkv, b * g, -1)
    o = torch.matmul(far, s["vp"].float().permute(1, 0, 2).contiguous()).view(hkv, b, g, dim).permute(1, 0, 2, 3)
    o = o + torch.matmul(near, s["v"].float().permute(0, 2, 1, 3).contiguous())
    return (o / total).reshape(b, c["hq"], dim).to(s["q"].dtype)


# ------------------------------------------- the operators, the library's

def _own(s):
    import block_quantized_matmul_amd as qmm
    c = s["case"]
    if c["op"] == "lora":
        return qmm.qmm_lora(s["x"], s["a"], s["b"], s["ids"], scales=s["scales"], base=s["base"], Y=s["y"])
    if c["op"] == "norm_rope":
        qmm.qmm_norm_rope(
            [qmm.qmm_head_part(s["q"], s["qo"], norm=True, weight=s["wq"], rotate=True),
             qmm.qmm_head_part(s["k"], s["kc"], norm=True, weight=s["wk"], rotate=True, slotted=True),
             qmm.qmm_head_part(s["v"], s["vc"], slotted=True)],
            positions=s["positions"], freqs=s["freqs"], pairs=c["pairs"], eps=1e-6, slots=s["slots"])
        return {"q": s["qo"], "k": s["kc"], "v": s["vc"]}
    if c["op"] == "prompt":
        return qmm.qmm_attn_prompt(s["q"], s["k"], s["v"], s["starts"], O=s["o"])
    return qmm.qmm_attn_shared(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["lengths"], O=s["o"])


def run(state):
    if own:
        return _own(state)
    return {"lora": _plain_lora, "norm_rope": _plain_norm_rope, "prompt": _plain_prompt,
            "shared": _plain_shared}[state["case"]["op"]](state)


# ------------------------------------------------ the definitions, 64 bits

def _attend(q, k, v, causal):
    """softmax(q k^T / sqrt(d)) v of one head in 64 bits."""
    w = q @ k.t().contiguous() / math.sqrt(q.shape[-1])
    if causal:
        w = w.masked_fill(torch.ones_like(w, dtype=torch.bool).triu(1), -math.inf)
    return torch.softmax(w, -1) @ v


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "lora":
        y = s["base"].double()
        for a in range(c["adapters"]):
            rows = (s["ids"] == a).nonzero()[:, 0]
            low = s["x"][rows].double() @ s["a"][a].double().t().contiguous()
            y[rows] += s["scales"][a].double() * (low @ s["b"][a].double().t().contiguous())
        return y
    if c["op"] == "norm_rope":
        rot = c["rot"]

        def heads(x, weight):
            x = x.double()
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + 1e-6).sqrt() * weight.double()
            y = x.clone()
            for i in range(rot // 2):
                j, m = (i, i + rot // 2) if c["pairs"] == "halves" else (2 * i, 2 * i + 1)
                turn = (s["positions"].double() * 10000.0 ** (-2.0 * i / rot))[:, None]
                y[..., j] = x[..., j] * turn.cos() - x[..., m] * turn.sin()
                y[..., m] = x[..., m] * turn.cos() + x[..., j] * turn.sin()
            return y

        kc, vc = s["kc"].double(), s["vc"].double()
        kc[s["slots"].long()] = heads(s["k"], s["wk"])
        vc[s["slots"].long()] = s["v"].double()
        return {"q": heads(s["q"], s["wq"]), "k": kc, "v": vc}
    g = c["hq"] // c["hkv"]
    o = s["o"].double()
    if c["op"] == "prompt":
        first = 0
        for n in s["lens"]:
            rows = slice(first, first + n)
            for h in range(c["hq"] if n else 0):
                o[rows, h] = _attend(s["q"][rows, h].double(), s["k"][rows, h // g].double(),
                                     s["v"][rows, h // g].double(), True)
            first += n
        return o
    for i, n in enumerate(s["lens"]):
        for h in range(c["hkv"]):
            k = torch.cat([s["kp"][:, h], s["k"][i, :n, h]]).double()
            v = torch.cat([s["vp"][:, h], s["v"][i, :n, h]]).double()
            heads = slice(h * g, h * g + g)
            o[i, heads] = _attend(s["q"][i, heads].double(), k, v, False)
    return o
