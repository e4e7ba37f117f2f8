"""qmm_attn_kv4 where keys that hardly count have by far the largest values: a weight
times its value's scale is rounded relative to the largest such product of the row, so
that those keys cost the others no precision."""
import numpy as np
import pytest
import torch

import oracle.serve_oracle as S
from attn_util import assert_within, f64, rng, say
from test_gpu_attn_kv4 import run, scales_at, setup

pytestmark = pytest.mark.gpu


def expected(q, cache, page, tables, lens, scale, kind):
    """As serve_oracle.attend's bound (one KV head), but for the products' smallest steps: 2^-25 of a code of 16
    times the size, relative to 2^7 of the row's largest product, instead of its largest scale."""
    want, err = np.zeros(q.shape), np.zeros(q.shape)
    for i, n in enumerate(lens):
        u = np.arange(n)
        k, v, dk, dv = (x[:, 0] for x in S.read(cache, page, tables[i, u // page].astype(np.int64) * page + u % page, 1, q.shape[2]))
        for h in range(q.shape[1]):
            o, _ = S.attend(q[i, h], k, v, dk, dv, scale, kind)
            s = (k @ q[i, h]) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            d = np.repeat(np.abs(dv), 32, -1)
            s_abs = 23 * (np.repeat(np.abs(dk), 32, -1) @ np.abs(q[i, h])) * scale
            off = (q.shape[2] + 16) * S.E32 * s_abs.max() + 16 * S.E32 * (np.abs(s).max() + 16) + 2.0 ** -22
            e = (2.0 ** -11 + (n + 64) * S.E32 * 23 + 2 * off) * 8 * (w @ d) + n * 2.0 ** -22 * (w[:, None] * d).max(0)
            want[i, h], err[i, h] = o, e + S.HALF_STEP[kind] * (np.abs(o) + e) + S.SUBNORMAL[kind]
    return want, err


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kind,large,small", [("bf16", 60000.0, 1e-4), ("bf16", 60000.0, 1e-6), ("f16", 60000.0, 2e-3)])
@pytest.mark.parametrize("lens,width", [([150, 700], None), ([700, 3000], 100)])
def test_large_values_without_a_weight(dim, kind, large, small, lens, width):
    g = rng(130, dim, len(kind))
    say(f"attn_kv4 outliers {dim} {kind} {small} {lens}")
    q, cache, tables = setup(g, lens, 64, 1, 1, dim, kind, width=width)
    scale = 1.0
    for i, n in enumerate(lens):
        u = np.arange(n)
        k = S.read(cache, 64, tables[i, u // 64].astype(np.int64) * 64 + u % 64, 1, dim)[0][:, 0]
        s = (k @ f64(q)[i, 0]) * scale
        out = s < s.max() - 30  # below 2^-43 of the largest weight
        assert 5 < out.sum() < n - 5
        for x in u:
            scales_at(cache, 64, 1, dim, int(tables[i, x // 64]) * 64 + x % 64, 0, 1)[:] *= np.float16(large if out[x] else small)
    want, err = expected(f64(q), cache, 64, tables, lens, scale, kind)
    assert (err < 0.06 * np.abs(want).max(-1, keepdims=True)).all()
    assert_within(run(q, cache, 64, 1, tables, lens, scale=scale), want, err, "outliers")


@pytest.mark.parametrize("dim", [64, 128])
def test_zero_values_first_and_tiny_weights_behind_zeros(dim):
    """The key that holds nearly all the weight has zeros as values: the outputs are the others', however small."""
    g = rng(131, dim)
    lens = [300]
    for gap in (5, 30, 60):
        q, cache, tables = setup(g, lens, 64, 1, 1, dim, "bf16")
        u = np.arange(300)
        k = S.read(cache, 64, tables[0, u // 64].astype(np.int64) * 64 + u % 64, 1, dim)[0][:, 0]
        s = k @ f64(q)[0, 0]
        top = int(np.argmax(s))
        scale = gap / (s[top] - np.sort(s)[-2])
        for x in u:
            v = scales_at(cache, 64, 1, dim, int(tables[0, x // 64]) * 64 + x % 64, 0, 1)
            v[:] = 0 if x == top or x < 64 else v
        want, err = expected(f64(q), cache, 64, tables, lens, scale, "bf16")
        say(f"attn_kv4 zeros first {dim} {gap}")
        assert_within(run(q, cache, 64, 1, tables, lens, scale=scale), want, err, "zeros first")
