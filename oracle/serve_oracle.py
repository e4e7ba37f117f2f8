"""Plain 64-bit definitions of the operators of include/qmm_serve.h (test
infrastructure only), with bounds on the rounding that the library's stated
numerics allow (E32, half a step of fp32, and HALF_STEP as in attn_oracle).

Every function takes and returns numpy arrays and loops over rows; it shares
no code with the HIP path.
"""
import numpy as np

from oracle.attn_oracle import E32, HALF_STEP, SUBNORMAL


def half(x):
    """fp32 to binary16 and back to 64 bits."""
    with np.errstate(over="ignore", invalid="ignore"):
        return np.asarray(x, np.float32).astype(np.float16)


# ------------------------------------------------------- the 4-bit cache

def page_bytes(page, heads, dim):
    return heads * (page // 16) * 18 * dim


def place(slot, page, heads, head, dim):
    """(page index, byte of the tile in the page, token of the tile) of a slot's head."""
    return slot // page, (head * (page // 16) + slot % page // 16) * 18 * dim, slot % 16


def key_nibble(t, e, dim):
    return ((e % 32 // 8 * 16 + t) * (dim // 32) + e // 32) * 8 + e % 8


def quantise(x):
    """(scale bits as uint16, codes) of 32 float64 values, rounded to fp32 first."""
    with np.errstate(over="ignore", invalid="ignore"):
        x = np.asarray(x, np.float64).astype(np.float32)
        if not np.isfinite(x).all():
            return 0x7E00, np.full(32, 8)
        m = x[int(np.argmax(np.abs(x)))]  # the first of several
        d = half(np.float64(m) / -8)
    if not np.isfinite(d):
        return 0x7E00, np.full(32, 8)
    if d == 0:
        return 0, np.full(32, 8)
    # 80 bits hold x / d + 8.5 to far below the distance of any quotient that is not at a border
    q = np.floor(x.astype(np.longdouble) / np.longdouble(d) + np.longdouble(8.5))
    return int(d.view(np.uint16)), np.clip(q, 0, 15).astype(np.int64)


def rotated(x, weight, norm, eps, positions, freqs, pairs):
    """Keys [n][heads][dim] normed and rotated, in 80 bits."""
    y = np.asarray(x, np.longdouble)
    if norm:
        y = y / np.sqrt(np.mean(y * y, -1, keepdims=True) + np.longdouble(eps))
        if weight is not None:
            y = y * np.asarray(weight, np.longdouble)
    z = y.copy()
    for i, f in enumerate(freqs if freqs is not None else []):
        j, m = (i, i + len(freqs)) if pairs == "halves" else (2 * i, 2 * i + 1)
        angle = (positions.astype(np.longdouble) * np.longdouble(f))[:, None]
        c, s = np.cos(angle), np.sin(angle)
        z[..., j] = y[..., j] * c - y[..., m] * s
        z[..., m] = y[..., m] * c + y[..., j] * s
    return z


def append(k, v, cache, page, slots, weight=None, norm=False, eps=1e-6, positions=None, freqs=None, pairs="halves"):
    """The cache (uint8 [pages][page bytes]) with the tokens stored, in order."""
    out = cache.copy()
    n, heads, dim = k.shape
    with np.errstate(invalid="ignore"):
        k = rotated(k, weight, norm, eps, positions, freqs, pairs)
    for t in range(n):
        slot = int(slots[t])
        if not 0 <= slot < cache.shape[0] * page:
            continue
        for h in range(heads):
            p, at, row = place(slot, page, heads, h, dim)
            tile = out[p, at:at + 18 * dim]
            for b in range(dim // 32):
                for which, x in ((0, k), (1, v)):
                    d, codes = quantise(x[t, h, 32 * b:32 * b + 32])
                    s = (16 + which) * dim + 2 * (16 * b + row)
                    tile[s], tile[s + 1] = d & 255, d >> 8
                    for i in range(32):
                        e = 32 * b + i
                        nibble = key_nibble(row, e, dim) if which == 0 else 16 * dim + row * dim + e
                        byte = tile[nibble // 2]
                        tile[nibble // 2] = (byte & 0xF0 | codes[i]) if nibble % 2 == 0 else (byte & 0x0F | codes[i] << 4)
    return out


def read(cache, page, slots, heads, dim):
    """(K, V, scales of K, scales of V), the first two [n][heads][dim], the last [n][heads][dim / 32]; NaN outside."""
    n = len(slots)
    kv = np.full((2, n, heads, dim), np.nan)
    sc = np.full((2, n, heads, dim // 32), np.nan)
    for i, slot in enumerate(int(s) for s in slots):
        if not 0 <= slot < cache.shape[0] * page:
            continue
        for h in range(heads):
            p, at, row = place(slot, page, heads, h, dim)
            tile = cache[p, at:at + 18 * dim]
            nib = np.stack([tile[:16 * dim] & 15, tile[:16 * dim] >> 4], -1).reshape(-1).astype(np.float64) - 8
            d = np.ascontiguousarray(tile[16 * dim:]).view(np.float16).astype(np.float64).reshape(2, dim // 32, 16)[:, :, row]
            sc[:, i, h] = d
            e = np.arange(dim)
            with np.errstate(invalid="ignore"):
                kv[0, i, h] = nib[key_nibble(row, e, dim)] * d[0, e // 32]
                kv[1, i, h] = nib[16 * dim + row * dim + e] * d[1, e // 32]
    return kv[0], kv[1], sc[0], sc[1]


def attend(q, k, v, dk, dv, scale, kind):
    """One query row over its keys (values, and their blocks' scales): output and bound.

    A score is a sum of code times q with the zero point apart: its terms are at
    most (15 + 8) |d| |q|, summed in fp32, and q below 2^-33 of its largest element
    is lost. That error, the exponent's own (a few steps of the scores' size) and
    the exponential's 2^-22 change the output by at most 2 d max |v|. A weight times
    a scale is two binary16 numbers, 2^-22, or absolutely half a step of binary16's
    smallest, where the largest product is 2^7 at least: with codes of 16 times the
    size, and 8 of them, 2^-25 2^4 2^3 2^-7 of it. The outputs' sums have terms of
    23 w |d|."""
    n, dim = k.shape
    if n == 0:
        return np.zeros(dim), np.zeros(dim)
    s = (k @ q) * scale
    blocks = np.repeat(np.abs(dk), 32, -1)
    s_abs = 23 * (blocks @ np.abs(q)) * scale
    lost = 2.0 ** -33 * np.abs(q).max() * 23 * blocks.sum(-1).max() * scale
    w = np.exp(s - s.max())
    w = w / w.sum()
    o = w @ v
    size = w @ np.repeat(np.abs(dv), 32, -1)
    most = np.repeat((w[:, None] * np.abs(dv)).max(0), 32, -1)
    u = HALF_STEP[kind]
    d = (dim + 16) * E32 * s_abs.max() + lost + 16 * E32 * (np.abs(s).max() + 16) + 2.0 ** -22
    err = 2.0 ** -22 * (w @ np.abs(v)) + (n + 64) * E32 * 23 * size + n * 2.0 ** -25 * most \
        + 2 * d * np.abs(v).max(0)
    return o, err + u * (np.abs(o) + err) + SUBNORMAL[kind]


def attn_kv4(q, cache, page, heads, tables, lengths, scale, kind):
    n, hq, dim = q.shape
    o, err = np.zeros(q.shape), np.zeros(q.shape)
    g = hq // heads
    for i in range(n):
        length = int(lengths[i])
        if not 0 <= length <= tables.shape[1] * page:
            o[i] = np.nan
            continue
        pages = tables[i, :-(-length // page)].astype(np.int64)
        if ((pages < 0) | (pages >= cache.shape[0])).any():
            o[i] = np.nan
            continue
        u = np.arange(length)
        k, v, dk, dv = read(cache, page, pages[u // page] * page + u % page, heads, dim)
        for h in range(hq):
            x = h // g
            with np.errstate(invalid="ignore", over="ignore"):
                o[i, h], err[i, h] = attend(q[i, h], k[:, x], v[:, x], dk[:, x], dv[:, x], scale, kind)
    return o, err


# ------------------------------------------------------ the expert layer

def choice(x, router, n_used, renormalise=True):
    """ids and weights [n][n_used]: logits in 80 bits (64 suffice, but for ties), the first of equal ones first."""
    logits = np.asarray(x, np.longdouble) @ np.asarray(router, np.longdouble).T
    with np.errstate(invalid="ignore", over="ignore"):
        key = np.where(np.isnan(logits), -np.inf, logits)
        ids = np.lexsort((np.isnan(logits), -key), axis=-1)[:, :n_used]  # (a NaN behind -infinity)
        top = np.take_along_axis(key, ids[:, :1], -1)
        w = np.exp(np.take_along_axis(logits, ids, -1) - top)
        total = w.sum(-1, keepdims=True) if renormalise else np.exp(logits - top).sum(-1, keepdims=True)
        return ids, np.asarray(w / total, np.float64)


def moe(x, router, gate, up, down, n_used, renormalise=True):
    """Y, its bound, ids and weights. gate, up, down: float64 [experts][rows][k].

    A product's sums: 32 terms in a block and then block by block, k / 32 + 40
    roundings of sums whose terms are at most 16 times the block's largest weight
    (4-bit codes are taken with an offset of 16, whose sum is taken off again).
    Activations, h among them, are off by 2^-22 and 2^-32. A routing weight's
    difference of logits is rounded to fp32 after 64-bit sums, its exponential and
    quotient are a few steps."""
    n, k = x.shape
    ids, w = choice(x, router, n_used, renormalise)
    y, err = np.zeros((n, k)), np.zeros((n, k))
    ff = gate.shape[1]

    def product(m, v, v_err, terms):
        size = np.repeat(np.abs(m).reshape(m.shape[0], -1, 32).max(-1), 32, -1)
        return m @ v, np.abs(m) @ v_err + (terms / 32 + 40) * E32 * (16 * size @ (np.abs(v) + v_err))

    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(n):
            for i in range(n_used):
                e, r = int(ids[t, i]), w[t, i]
                x_err = 2.0 ** -22 * np.abs(x[t]) + 2.0 ** -32
                g, eg = product(gate[e], x[t], x_err, k)
                u, eu = product(up[e], x[t], x_err, k)
                s = g / (1 + np.exp(-g))
                h = s * u
                eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu
                eh = (r * (eh + (8 + 12) * E32 * np.abs(h))) * (1 + 2.0 ** -20)
                h = r * h
                eh = eh + 2.0 ** -22 * np.abs(h) + 2.0 ** -32
                d, ed = product(down[e], h, eh, ff * n_used * n)
                y[t] += d
                err[t] += ed
    return y, err, ids, w


# ------------------------------------------------------------- the choice of a token

def sample(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probability, distance): one row, in 80 bits. The distance is how far, as a share of the kept mass, any
    of the decisions on the way was from its border: a result of other arithmetic may differ where that is tiny."""
    z = np.asarray(z, np.longdouble).copy()
    z[np.isnan(z)] = -np.inf
    if z.max() == -np.inf:
        return -1, np.nan, 1.0
    order = np.argsort(-z, kind="stable")
    z = z[order]
    if not temperature > 0:
        return int(order[0]), 1.0, 1.0
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        d = np.where(z == z[0], 0, z[0] - z)
        w = np.where(np.isinf(d), 0, np.exp(-np.where(np.isinf(d), 0, d) / np.longdouble(temperature)))
    near = 1.0
    n = min(top_k, len(w)) if top_k > 0 else len(w)
    if top_p < 1:  # (a NaN is none)
        before = np.concatenate([[0], np.cumsum(w[:n])[:-1]])
        goal = np.longdouble(max(top_p, 0)) * w[:n].sum()
        m = max(1, int((before < goal).sum()))
        near = min(near, float(np.abs(before[1:] - goal).min() / w[:n].sum()) if n > 1 else 1.0)
    else:
        m = n
    if min_p > 0:
        keep = w >= np.longdouble(min_p)
        near = min(near, float(np.abs(w[1:] - min_p).min()) if len(w) > 1 and min_p < 1 else 1.0)
        m = min(m, max(1, int(keep.sum())) if min_p < 1 else int((w == 1).sum()))
    w = w[:m]
    u = min(max(float(u), 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    after = np.cumsum(w)
    goal = np.longdouble(u) * after[-1]
    i = min(int((after <= goal).sum()), m - 1)
    if m > 1 and u > 0:
        near = min(near, float(np.abs(after[:-1] - goal).min() / after[-1]))
    return int(order[i]), float(w[i] / after[-1]), near
