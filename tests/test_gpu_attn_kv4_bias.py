"""qmm_attn_kv4 over many keys: the errors of its sums have no sign in common."""
import numpy as np
import pytest

import oracle.serve_oracle as S
from attn_util import f64, rng, say
from test_gpu_attn_kv4 import run, setup

pytestmark = pytest.mark.gpu


def read(cache, page, slots, heads, dim):
    """Keys and values as serve_oracle.read gives them, of many places at once."""
    t = cache.reshape(cache.shape[0], heads, page // 16, 18 * dim)[slots // page, :, slots % page // 16]
    i, row = np.arange(len(slots)), slots % 16
    nib = np.stack([t[..., :16 * dim] & 15, t[..., :16 * dim] >> 4], -1).reshape(len(slots), heads, 32 * dim).astype(np.float64) - 8
    e = np.arange(dim)
    at = np.stack([[S.key_nibble(r, x, dim) for x in e] for r in range(16)])[row], 16 * dim + row[:, None] * dim + e
    d = np.ascontiguousarray(t[..., 16 * dim:]).view(np.float16).astype(np.float64).reshape(len(slots), heads, 2, dim // 32, 16)
    return [np.take_along_axis(nib, np.repeat(at[w][:, None], heads, 1), -1) *
            np.repeat(d[i, :, w, :, row], 32, -1) for w in range(2)]


@pytest.mark.parametrize("dim", [64, 128])
def test_mean_error(dim):
    """The mean of N outputs' errors: their roundings', each uniform within half a step and independent, six standard
    deviations, and a step of fp32 of the values' size for all that the sums may have in common."""
    g = rng(150, dim)
    hq, n, scale = 12, 16000, 0.02
    say(f"attn_kv4 mean error {dim}")
    q, cache, tables = setup(g, [n, n], 256, hq, hq, dim, "f16")
    o, q64 = f64(run(q, cache, 256, hq, tables, [n, n], scale=scale)), f64(q)
    off, steps, values = np.zeros(o.shape), np.zeros(o.shape), []
    for i in range(2):
        total, size, want = np.zeros(hq), np.zeros((hq, dim)), np.zeros((hq, dim))
        for at in range(0, n, 1000):
            u = np.arange(at, at + 1000)
            k, v = read(cache, 256, tables[i, u // 256].astype(np.int64) * 256 + u % 256, hq, dim)
            w = np.exp(scale * np.einsum("uhe,he->uh", k, q64[i]))
            total += w.sum(0)
            want += np.einsum("uh,uhe->he", w, v)
            size += np.einsum("uh,uhe->he", w, np.abs(v))
        want /= total[:, None]
        off[i] = o[i] - want
        steps[i] = np.spacing(np.abs(want).astype(np.float16)).astype(np.float64)
        values.append(size / total[:, None])
    bound = 6 * np.sqrt((steps ** 2).mean() / 12 / off.size) + 2.0 ** -23 * np.mean(values)
    say(f"mean {off.mean():.3g} within {bound:.3g}")
    assert abs(off.mean()) <= bound


def test_read():
    g = rng(151)
    _, cache, tables = setup(g, [100], 64, 2, 2, 64, "f16")
    slots = tables[0, np.arange(100) // 64].astype(np.int64) * 64 + np.arange(100) % 64
    for got, want in zip(read(cache, 64, slots, 2, 64), S.read(cache, 64, slots, 2, 64)):
        assert np.array_equal(got, want)
