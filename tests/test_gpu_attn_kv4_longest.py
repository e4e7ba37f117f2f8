"""qmm_attn_kv4 at the longest lengths that it takes, just below 2^31 keys: a table
that lists a few pages again and again, so that the definition needs their keys once."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.serve_oracle as S
from attn_util import assert_within, f64, rng, say
from test_gpu_attn_kv4 import make_cache

pytestmark = pytest.mark.gpu


def test_longest_lengths():
    """Sums of 2^19 keys by each wavefront: 2^14 additions of products and 2^13 of weights, and some 2^11 to join them."""
    g = rng(120)
    page, dim, pages = 32, 64, 3
    width = 2 ** 26 - 1
    lens = [width * page, width * page - 5, 2 ** 31 - 64, 2 ** 31 - 63, 100]
    cache = make_cache(g, pages, page, 1, dim)
    q = torch.from_numpy(g.standard_normal((len(lens), 2, dim))).to(torch.float16)
    table = (torch.arange(width, dtype=torch.int32, device="cuda") % pages).expand(len(lens), -1)
    say("attn_kv4 lengths near 2^31")
    o = qmm.qmm_attn_kv4(q.cuda(), torch.from_numpy(cache).cuda(), page, 1, table,
                         torch.tensor(lens, dtype=torch.int32).cuda(), scale=0.3)
    torch.cuda.synchronize()
    k, v, _, dv = S.read(cache, page, np.arange(pages * page), 1, dim)
    want, err = np.zeros(q.shape), np.zeros(q.shape)
    for i, n in enumerate(lens):
        times = np.full(pages, n // page // pages, np.float64)
        times[:n // page % pages] += 1
        times = np.repeat(times, page)
        last = n // page % pages * page
        times[last:last + n % page] += 1
        assert times.sum() == n
        for h in range(2):
            s = 0.3 * (k[:, 0] @ f64(q)[i, h])
            w = times * np.exp(s - s.max())
            w /= w.sum()
            want[i, h] = w @ v[:, 0]
            size = np.repeat(w @ np.abs(dv[:, 0]), 32, -1)
            # weights to 2^-11; products' terms of at most 23 |d|, and the weights' sum, with 2^15 roundings each
            err[i, h] = 2.0 ** -11 * (w @ np.abs(v[:, 0])) + 2.0 ** -9 * (23 * size + np.abs(want[i, h])) + 2.0 ** -11
    assert_within(o, want, err, "longest")
