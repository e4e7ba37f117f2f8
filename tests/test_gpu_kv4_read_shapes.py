"""qmm_kv4_read with few and odd numbers of heads, of keys, values or both: how
rows are laid on wavefronts depends on them."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.serve_oracle as S
from attn_util import rng, say
from test_gpu_attn_kv4 import make_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [1, 2, 3, 4, 5, 8, 17])
def test_shapes(dim, heads):
    g = rng(95, dim, heads)
    page, pages = 32, 5
    cache = make_cache(g, pages, page, heads, dim)
    dev = torch.from_numpy(cache).cuda()
    for n in (1, 2, 7, 37, 129):
        slots = g.integers(-3, pages * page + 3, n).astype(np.int32)
        want = S.read(cache, page, slots, heads, dim)[:2]
        s = torch.from_numpy(slots).cuda()
        for use in ((True, False), (False, True), (True, True)):
            say(f"kv4 read {dim} {heads} {n} {use}")
            out = [torch.full((n + 1, heads, dim), -3.0, device="cuda") if u else None for u in use]
            qmm.qmm_kv4_read(dev, page, s, K=None if out[0] is None else out[0][:n],
                             V=None if out[1] is None else out[1][:n])
            torch.cuda.synchronize()
            for o, w in zip(out, want):
                if o is not None:
                    assert np.array_equal(o[:n].double().cpu().numpy(), w, equal_nan=True)
                    assert (o[n] == -3.0).all()
