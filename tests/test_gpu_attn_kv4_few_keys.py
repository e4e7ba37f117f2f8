"""qmm_attn_kv4 over so few keys that every rounding shows where their values cancel:
weights are as exact as fp32's, not rounded to the operands' 11 bits."""
import numpy as np
import pytest

import oracle.serve_oracle as S
from attn_util import assert_within, f64, rng, say
from test_gpu_attn_kv4 import run, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim,hq,heads", [(64, 4, 2), (128, 4, 2), (64, 12, 1), (128, 8, 1)])
def test_few_keys(dim, hq, heads, kind):
    """A weight, its two halves and the products are off by 2^-22 each; a score's and its exponential's error as in
    serve_oracle.attend; sums of at most 17 keys, the zero point, four wavefronts and the quotient: 32 roundings."""
    g = rng(140, dim, hq)
    lens = [2, 3, 5, 17] * 8
    scale = 1e-3
    say(f"attn_kv4 few keys {dim} {hq} {kind}")
    q, cache, tables = setup(g, lens, 32, hq, heads, dim, kind)
    v64 = f64(q)
    want, err = np.zeros(q.shape), np.zeros(q.shape)
    for i, n in enumerate(lens):
        k, v, dk, dv = S.read(cache, 32, int(tables[i, 0]) * 32 + np.arange(n), heads, dim)
        for h in range(hq):
            x = h // (hq // heads)
            s = (k[:, x] @ v64[i, h]) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            d = np.repeat(np.abs(dv[:, x]), 32, -1)
            off = (dim + 16) * S.E32 * 23 * scale * (np.repeat(np.abs(dk[:, x]), 32, -1) @ np.abs(v64[i, h])).max() + 2.0 ** -20
            want[i, h] = w @ v[:, x]
            e = (2 * off + 3 * 2.0 ** -22) * (w @ np.abs(v[:, x])) + 32 * S.E32 * 23 * (w @ d)
            err[i, h] = e + S.HALF_STEP[kind] * (np.abs(want[i, h]) + e) + S.SUBNORMAL[kind]
    assert_within(run(q, cache, 32, heads, tables, lens, scale=scale), want, err, "few keys")
