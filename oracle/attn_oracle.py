"""Plain 64-bit definitions of the operators of include/qmm_attn.h (test
infrastructure only), with bounds on the rounding of a computation in 32 bits.

Every function takes and returns numpy float64 arrays (integers for ids,
positions and lengths) and loops over rows; it shares no code with the HIP
path. Each also returns the largest error that the library's stated numerics
allow, from these parts:

  u        half a step of the stored type, finfo(t).eps / 2, relative to the
           value (plus half of the smallest subnormal)
  e        half a step of fp32, 2^-24: a sum of n terms in any order is off
           by at most (n + 1) e times the sum of their magnitudes
"""
import numpy as np

E32 = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUBNORMAL = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def lora(x, a, b, ids, scales=None, base=None):
    """Y and its bound: V sums k terms, Y sums rank terms of V's rounded values."""
    n, (ad, rank, k), rows = x.shape[0], a.shape, b.shape[1]
    y = np.zeros((n, rows)) if base is None else base.astype(np.float64).copy()
    err = 2 * E32 * np.abs(y)
    for t in range(n):
        i = int(ids[t])
        if i == -1:
            continue
        if not 0 <= i < ad:
            y[t] = np.nan
            continue
        s = 1.0 if scales is None else float(scales[i])
        v = a[i] @ x[t]
        v_err = (k + 64) * E32 * (np.abs(a[i]) @ np.abs(x[t]))
        d = s * (b[i] @ v)
        d_err = abs(s) * (np.abs(b[i]) @ (v_err + (rank + 8) * E32 * (np.abs(v) + v_err)))
        err[t] += d_err + 2 * E32 * (np.abs(y[t]) + np.abs(d) + d_err)
        y[t] += d
    return y, err


def norm_rope(x, weight=None, norm=False, eps=1e-6, positions=None, freqs=None, pairs="halves", out="f32"):
    """One part: [n_tokens][heads][dim] and its bound. The norm's sum has dim
    terms and its square root, quotient and two products a step each; sine and
    cosine are off by at most 2^-22 in all (polynomial and angle)."""
    y = x.astype(np.float64).copy()
    dim = x.shape[-1]
    rel = 0.0
    if norm:
        y = y / np.sqrt(np.mean(y * y, -1, keepdims=True) + eps)
        if weight is not None:
            y = y * weight
        rel = (dim / 2 + 16) * E32  # half the sum's relative error, by the square root
    err = rel * np.abs(y)
    if positions is not None:
        z, z_err = y.copy(), err.copy()
        for i, f in enumerate(freqs):
            j, m = (i, i + len(freqs)) if pairs == "halves" else (2 * i, 2 * i + 1)
            # the product and the sines in 80 bits: 2^31 positions times a frequency leave 64 bits no fraction to spare
            angle = (positions.astype(np.longdouble) * np.longdouble(f))[:, None]
            c, s = np.cos(angle).astype(np.float64), np.sin(angle).astype(np.float64)
            z[..., j] = y[..., j] * c - y[..., m] * s
            z[..., m] = y[..., m] * c + y[..., j] * s
            z_err[..., j] = z_err[..., m] = (rel + 2.0 ** -22 + 4 * E32) * (np.abs(y[..., j]) + np.abs(y[..., m]))
        y, err = z, z_err
    return y, err + HALF_STEP[out] * (np.abs(y) + err) + SUBNORMAL[out]


def attend(q, k, v, scale, kind):
    """One query row over its keys: output and bound.

    A score's error d (its dot product of D terms, the scaling and the
    difference to the maximum, and the exponential's 2^-22) changes a weight
    by the factor e^d, hence the output by at most 2 d max |v| (twice: weight
    and sum); a weight is rounded to `kind` for the product (u, or absolutely
    below the type's normal range, relative to the largest weight), the output
    once more; sums of n terms with a rescaling per block of keys, and a join
    of pieces, cost at most (3 n + 64) e."""
    n, dim = k.shape
    if n == 0:
        return np.zeros(v.shape[1] if v.ndim == 2 else dim), np.zeros(dim)
    s = (k @ q) * scale
    s_abs = (np.abs(k) @ np.abs(q)) * scale
    w = np.exp(s - s.max())
    total = w.sum()
    w = w / total
    o = w @ v
    mag = w @ np.abs(v)
    u = HALF_STEP[kind]
    d = (dim + 8) * E32 * s_abs.max() + 4 * E32 * (np.abs(s).max() + 1) + 2.0 ** -22
    err = (u + (3 * n + 64) * E32) * mag + SUBNORMAL[kind] * np.abs(v).sum(0) / total + 2 * d * np.abs(v).max(0)
    return o, err + u * (np.abs(o) + err) + SUBNORMAL[kind]


def attn_prompt(q, k, v, starts, scale, kind):
    """[n][hq][dim] output (NaN where no sequence holds the token) and bound."""
    o = np.full(q.shape, np.nan)
    err = np.zeros(q.shape)
    g = q.shape[1] // k.shape[1]
    for b, e in zip(starts[:-1], starts[1:]):
        if not 0 <= b <= e <= q.shape[0]:
            continue
        for t in range(b, e):
            for h in range(q.shape[1]):
                o[t, h], err[t, h] = attend(q[t, h], k[b:t + 1, h // g], v[b:t + 1, h // g], scale, kind)
    return o, err


def attn_shared(q, pk, pv, k, v, lengths, scale, kind):
    o, err = np.zeros(q.shape), np.zeros(q.shape)
    hkv = pk.shape[1] if pk is not None else k.shape[2]
    g = q.shape[1] // hkv
    for b in range(q.shape[0]):
        n = 0 if k is None else int(lengths[b])
        if n < 0 or (k is not None and n > k.shape[1]):
            o[b] = np.nan
            continue
        for h in range(q.shape[1]):
            keys = [pk[:, h // g]] if pk is not None else []
            values = [pv[:, h // g]] if pv is not None else []
            if k is not None:
                keys.append(k[b, :n, h // g])
                values.append(v[b, :n, h // g])
            o[b, h], err[b, h] = attend(q[b, h], np.concatenate(keys), np.concatenate(values), scale, kind)
    return o, err
