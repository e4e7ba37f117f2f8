"""qmm_norm_rope against the 64-bit definition on the GPU."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.attn_oracle as O
from attn_util import TORCH, assert_within, f64, rng, rounded, say

pytestmark = pytest.mark.gpu

KEPT = 7.0


def _freqs(n):
    return [10000.0 ** (-i / max(n, 1)) for i in range(n)]


def _ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


@pytest.mark.parametrize("xt,yt", [("f32", "f16"), ("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f16", "bf16"),
                                   ("bf16", "f32")])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("dim,n_freqs", [(128, 64), (128, 32), (64, 32), (80, 40), (80, 20), (2, 1), (6, 2), (10, 5),
                                         (66, 33), (256, 128), (512, 256), (512, 6), (258, 129)])
def test_norm_and_rotation(xt, yt, pairs, dim, n_freqs):
    n, hq, hkv = 5, 3, 2
    r = rng(3, dim, n_freqs)
    x = [rounded(2 * r.standard_normal((n, h, dim)), xt) for h in (hq, hkv, hkv)]
    w = [torch.from_numpy((1 + 0.3 * r.standard_normal(dim)).astype(np.float32)) for _ in range(2)]
    pos = r.integers(0, 100000, n)
    f = _freqs(n_freqs)
    y = [torch.full(t.shape, KEPT, dtype=TORCH[yt], device="cuda") for t in x]
    what = f"norm_rope {xt}->{yt} {pairs} dim={dim} freqs={n_freqs}"
    say(what)
    qmm.qmm_norm_rope([qmm.qmm_head_part(x[0].cuda(), y[0], norm=True, weight=w[0].cuda(), rotate=True),
                       qmm.qmm_head_part(x[1].cuda(), y[1], norm=True, weight=w[1].cuda(), rotate=True),
                       qmm.qmm_head_part(x[2].cuda(), y[2])], _ints(pos), f, pairs=pairs)
    torch.cuda.synchronize()
    for i in range(3):
        want, err = O.norm_rope(f64(x[i]), None if i == 2 else f64(w[i]), i < 2, 1e-6, pos if i < 2 else None,
                                f, pairs, yt)
        assert_within(y[i], want, err, f"{what} part {i}")


@pytest.mark.parametrize("n", [1, 4, 63, 1000])
@pytest.mark.parametrize("heads", [(32, 8), (1, 1), (5, 0)])
def test_token_and_head_counts(n, heads):
    """One pass per wavefront, a whole token per wavefront, and counts between."""
    hq, hkv = heads
    r = rng(4, n, hq)
    x = [rounded(r.standard_normal((n, h, 128)), "f32") for h in (hq, hkv)]
    pos = r.integers(0, 5000, n)
    y = [torch.full(t.shape, KEPT, dtype=torch.float16, device="cuda") for t in x]
    say(f"norm_rope n={n} heads={heads}")
    qmm.qmm_norm_rope([qmm.qmm_head_part(a.cuda(), b, norm=True, rotate=True) for a, b in zip(x, y)], _ints(pos),
                      _freqs(64))
    torch.cuda.synchronize()
    for a, b in zip(x, y):
        want, err = O.norm_rope(f64(a), None, True, 1e-6, pos, _freqs(64), "halves", "f16")
        assert_within(b, want, err, f"n={n} heads={heads}")


def test_many_tokens():
    n = 20011
    r = rng(5)
    x = rounded(r.standard_normal((n, 2, 64)), "f16")
    pos = r.integers(0, 1 << 20, n)
    y = torch.empty(x.shape, dtype=torch.float16, device="cuda")
    say("norm_rope 20011 tokens")
    qmm.qmm_norm_rope([qmm.qmm_head_part(x.cuda(), y, norm=True, rotate=True)], _ints(pos), _freqs(32))
    torch.cuda.synchronize()
    want, err = O.norm_rope(f64(x), None, True, 1e-6, pos, _freqs(32), "halves", "f16")
    assert_within(y, want, err, "20011 tokens")


def test_far_and_negative_positions():
    """Angles of far positions keep fp32's full accuracy (an angle formed in fp32 would be off by whole radians)."""
    pos = np.array([0, 1, -1, 1 << 20, 16777217, 2 ** 31 - 1, -2 ** 31, 123456789])
    r = rng(6)
    x = rounded(r.standard_normal((len(pos), 2, 64)), "f32")
    for f in (_freqs(32), [3.7 ** (-i) * 40 for i in range(32)], [0.0] * 31 + [-1.5]):
        for pairs in ("halves", "neighbours"):
            y = torch.empty(x.shape, dtype=torch.float32, device="cuda")
            say(f"norm_rope far positions {pairs} first frequency {f[0]}")
            qmm.qmm_norm_rope([qmm.qmm_head_part(x.cuda(), y, rotate=True)], _ints(pos), f, pairs=pairs)
            torch.cuda.synchronize()
            want, err = O.norm_rope(f64(x), None, False, 0.0, pos, f, pairs, "f32")
            assert_within(y, want, err, f"far positions {pairs}")


@pytest.mark.parametrize("dim", [64, 66])
def test_slots(dim):
    """Rows go to their slots; tokens with a slot outside the cache and the cache's other rows are left alone."""
    n, n_slots = 7, 12
    r = rng(7, dim)
    k, v = (rounded(r.standard_normal((n, 2, dim)), "f32") for _ in range(2))
    q = rounded(r.standard_normal((n, 4, dim)), "f32")
    slots = [11, -1, 0, 12, 5, 2 ** 31 - 1, 3]
    pos = np.arange(n)
    kc, vc = (torch.full((n_slots, 2, dim), KEPT, dtype=torch.float16, device="cuda") for _ in range(2))
    qo = torch.empty((n, 4, dim), dtype=torch.float16, device="cuda")
    say(f"norm_rope slots dim={dim}")
    qmm.qmm_norm_rope([qmm.qmm_head_part(q.cuda(), qo, rotate=True),
                       qmm.qmm_head_part(k.cuda(), kc, rotate=True, slotted=True),
                       qmm.qmm_head_part(v.cuda(), vc, slotted=True)], _ints(pos), _freqs(dim // 2), slots=_ints(slots))
    torch.cuda.synchronize()
    want, err = O.norm_rope(f64(q), None, False, 0, pos, _freqs(dim // 2), "halves", "f16")
    assert_within(qo, want, err, "queries")
    for x, c, p in ((k, kc, pos), (v, vc, None)):
        want, err = O.norm_rope(f64(x), None, False, 0, p, _freqs(dim // 2), "halves", "f16")
        full, ferr = np.full((n_slots, 2, dim), KEPT), np.zeros((n_slots, 2, dim))
        for t, s in enumerate(slots):
            if 0 <= s < n_slots:
                full[s], ferr[s] = want[t], err[t]
        assert_within(c, full, ferr, "cache")
    # no slots at all: nothing is stored, nothing read
    empty = torch.empty((0, 2, dim), dtype=torch.float16, device="cuda")
    qmm.qmm_norm_rope([qmm.qmm_head_part(k.cuda(), empty, slotted=True)], slots=_ints(slots))
    torch.cuda.synchronize()


def test_strides_alignment_and_in_place():
    n, h, dim = 6, 3, 64
    r = rng(8)
    base = rounded(r.standard_normal((n, h, dim)), "f32")
    pos = np.arange(n) * 977
    want, err = O.norm_rope(f64(base), None, True, 1e-6, pos, _freqs(32), "halves", "f32")
    for off, gap, major in ((0, 0, False), (1, 3, False), (4, 8, True), (3, 1, True)):
        shape = (h, n, dim + gap) if major else (n, h, dim + gap)
        xb = torch.full((int(np.prod(shape)) + off,), 5.0, device="cuda")
        yb = torch.full_like(xb, KEPT)
        x, y = (t[off:].view(shape)[..., :dim] for t in (xb, yb))
        x, y = (x.transpose(0, 1), y.transpose(0, 1)) if major else (x, y)
        x.copy_(base)
        say(f"norm_rope offset {off} gap {gap} head-major {major}")
        qmm.qmm_norm_rope([qmm.qmm_head_part(x, y, norm=True, rotate=True)], _ints(pos), _freqs(32))
        torch.cuda.synchronize()
        assert_within(y, want, err, f"offset {off} gap {gap}")
        assert bool((yb[:off] == KEPT).all())
        if gap:
            assert bool((yb[off:].view(shape)[..., dim:] == KEPT).all())
        qmm.qmm_norm_rope([qmm.qmm_head_part(x, x, norm=True, rotate=True)], _ints(pos), _freqs(32))
        torch.cuda.synchronize()
        assert torch.equal(x, y)
    # one key head for all tokens of a batch (stride 0 in, own rows out)
    one = rounded(r.standard_normal((1, h, dim)), "f32")
    y = torch.empty((n, h, dim), device="cuda")
    say("norm_rope broadcast input")
    qmm.qmm_norm_rope([qmm.qmm_head_part(one.cuda().expand(n, h, dim), y, rotate=True)], _ints(pos), _freqs(32))
    torch.cuda.synchronize()
    want, err = O.norm_rope(np.repeat(f64(one), n, 0), None, False, 0, pos, _freqs(32), "halves", "f32")
    assert_within(y, want, err, "broadcast")


def test_zeros_eps_and_nonfinite_heads():
    """A head of zeros stays zero; a head with a NaN or an infinity does not touch its neighbours."""
    n, h, dim = 3, 4, 128
    r = rng(9)
    x = rounded(r.standard_normal((n, h, dim)), "f16")
    x[0, 0] = 0
    x[1, 2, 7] = float("nan")
    x[2, 1, 9] = float("inf")
    y = torch.empty(x.shape, dtype=torch.float16, device="cuda")
    say("norm_rope zeros and non-finite heads")
    qmm.qmm_norm_rope([qmm.qmm_head_part(x.cuda(), y, norm=True, rotate=True)], _ints([4, 5, 6]), _freqs(64), eps=1e-5)
    torch.cuda.synchronize()
    want, err = O.norm_rope(f64(x), None, True, 1e-5, np.array([4, 5, 6]), _freqs(64), "halves", "f16")
    got = f64(y)
    assert (got[0, 0] == 0).all() and np.isnan(got[1, 2]).all() and np.isnan(got[2, 1, 9])
    ok = np.ones((n, h), bool)
    ok[1, 2] = ok[2, 1] = False
    assert (np.abs(got - want)[ok] <= err[ok]).all()


def test_replayed_with_new_positions():
    n = 40
    r = rng(10)
    x = rounded(r.standard_normal((n, 8, 128)), "f32").cuda()
    pos, slots = _ints(np.arange(n)), _ints(r.permutation(64)[:n])
    cache = torch.zeros((64, 8, 128), dtype=torch.bfloat16, device="cuda")
    parts = [qmm.qmm_head_part(x, cache, norm=True, rotate=True, slotted=True)]
    say("norm_rope graph")
    qmm.qmm_norm_rope(parts, pos, _freqs(64), slots=slots)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.qmm_norm_rope(parts, pos, _freqs(64), slots=slots)
    for i in range(3):
        pos.add_(n)
        slots.copy_((slots + 1) % 64)
        cache.zero_()
        qmm.qmm_norm_rope(parts, pos, _freqs(64), slots=slots)
        want = cache.clone()
        cache.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(cache, want), i
