"""qmm_attn_shared against the 64-bit definition on the GPU."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.attn_oracle as O
from attn_util import TORCH, assert_within, f64, rng, rounded, say

pytestmark = pytest.mark.gpu


def _inputs(seed, b, prefix, cap, hq, hkv, dim, kind):
    r = rng(2, seed, b, prefix, cap, hq, hkv, dim)
    q = rounded(r.standard_normal((b, hq, dim)), kind)
    pk, pv = (rounded(r.standard_normal((prefix, hkv, dim)), kind) for _ in range(2))
    k, v = (rounded(r.standard_normal((b, cap, hkv, dim)), kind) for _ in range(2))
    return q, pk, pv, k, v


def _dev(x):
    return None if x is None else x.cuda()


def _run(q, pk, pv, k, v, lengths, **kw):
    lens = None if k is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    o = qmm.qmm_attn_shared(*(_dev(x) for x in (q, pk, pv, k, v)), lens, **kw)
    torch.cuda.synchronize()
    return o


def _check(q, pk, pv, k, v, lengths, kind, what, o=None):
    say(what)
    o = _run(q, pk, pv, k, v, lengths) if o is None else o
    want, err = O.attn_shared(f64(q), *(None if x is None else f64(x) for x in (pk, pv, k, v)), lengths,
                              q.shape[2] ** -0.5, kind)
    assert_within(o, want, err, what)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("b,prefix,cap,lengths,hq,hkv", [
    (1, 1, 1, [0], 1, 1), (1, 0, 5, [5], 4, 1), (3, 0, 40, [0, 1, 40], 2, 2), (2, 63, 33, [32, 33], 8, 2),
    (5, 64, 31, [0, 1, 7, 30, 31], 4, 4), (4, 65, 300, [300, 0, 129, 257], 7, 1), (33, 130, 8, None, 4, 1),
    (2, 700, 700, [699, 13], 6, 2), (3, 257, 64, [64, 3, 0], 40, 1), (40, 300, 3, None, 8, 8),
    # more keys than are taken without pieces
    (1, 1025, 0, [0], 4, 2), (3, 1087, 1, [1, 0, 1], 40, 1), (33, 1030, 5, None, 4, 1), (2, 1, 1100, [1100, 0], 6, 2),
    (5, 64, 1000, [0, 1000, 33, 256, 257], 4, 4), (3, 0, 1500, [1500, 0, 700], 7, 1), (17, 1024, 40, None, 8, 2),
    (70, 0, 40, None, 8, 8),
])
def test_against_the_definition(kind, dim, b, prefix, cap, lengths, hq, hkv):
    lengths = [i % (cap + 1) for i in range(b)] if lengths is None else lengths
    x = _inputs(0, b, prefix, cap, hq, hkv, dim, kind)
    _check(*x, lengths, kind, f"shared {kind} dim={dim} b={b} prefix={prefix} cap={cap} heads={hq}/{hkv}")


@pytest.mark.parametrize("dim", [64, 128])
def test_prefix_only_and_caches_only(dim):
    q, pk, pv, k, v = _inputs(1, 6, 200, 50, 4, 2, dim, "f16")
    lengths = [0, 1, 2, 31, 32, 50]
    _check(q, pk, pv, None, None, lengths, "f16", "shared prefix only")
    _check(q, None, None, k, v, lengths, "f16", "shared caches only (a row of zeros first)")


def test_long_ranges_in_many_pieces():
    """Enough keys that both ranges are cut into several pieces, with ends inside a block."""
    b, prefix, cap, hq, hkv, dim = 3, 5003, 1500, 8, 2, 128
    x = _inputs(2, b, prefix, cap, hq, hkv, dim, "bf16")
    _check(*x, [1499, 0, 777], "bf16", "shared long")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("prefix", [90, 1090])
def test_nothing_past_a_length_counts(bad, prefix):
    """What the cache holds past a sequence's length, and what other sequences hold, does not reach it."""
    b, cap, hq, hkv, dim = 4, 70, 4, 2, 64
    q, pk, pv, k, v = _inputs(3, b, prefix, cap, hq, hkv, dim, "f16")
    lengths = [0, 33, 69, 70]
    for i, n in enumerate(lengths):
        k[i, n:], v[i, n:] = bad, bad
    want, err = O.attn_shared(f64(q), f64(pk), f64(pv), f64(k), f64(v), lengths, 0.125, "f16")
    say(f"shared {bad} past the lengths")
    assert_within(_run(q, pk, pv, k, v, lengths), want, err, "past the lengths")
    v[2, 10, 1, 3] = bad  # one value that sequence 2 does attend to
    say(f"shared {bad} in one value")
    o = f64(_run(q, pk, pv, k, v, lengths))
    assert not np.isfinite(o[2, 2:, 3]).any()
    ok = np.ones(o.shape, bool)
    ok[2, 2:, 3] = False
    assert (np.abs(o - want)[ok] <= err[ok]).all()


@pytest.mark.parametrize("prefix,cap", [(90, 70), (1090, 70), (200, 1000)])
def test_scores_of_minus_infinity(prefix, cap):
    """A key whose score is -infinity has no weight; a row with keys, but without any weight, is 0 / 0."""
    b, hq, hkv, dim = 4, 4, 2, 64
    q, pk, pv, k, v = _inputs(7, b, prefix, cap, hq, hkv, dim, "f16")
    q[:, :, 0] = 1.0
    pk[:, :, 0] = -float("inf")
    lengths = [0, 1, 33, 70]
    want, err = O.attn_shared(f64(q), None, None, f64(k), f64(v), lengths, 0.125, "f16")
    want[0] = np.nan
    say(f"shared scores of -inf, prefix {prefix}")
    assert_within(_run(q, pk, pv, k, v, lengths), want, err, "no weight in the prefix")
    k[2, :, :, 0] = -float("inf")
    want[2] = np.nan
    assert_within(_run(q, pk, pv, k, v, lengths), want, err, "no weight at all")


def test_lengths_outside_the_cache_give_nan_rows():
    for prefix in (40, 1040):
        q, pk, pv, k, v = _inputs(4, 5, prefix, 16, 2, 1, 64, "f16")
        _check(q, pk, pv, k, v, [3, -1, 17, 16, 2 ** 31 - 1], "f16", f"shared bad lengths, prefix {prefix}")


@pytest.mark.parametrize("prefix", [100, 1100])
def test_strides_and_a_given_workspace(prefix):
    b, cap, hq, hkv, dim = 3, 50, 4, 2, 64
    q, pk, pv, k, v = _inputs(5, b, prefix, cap, hq, hkv, dim, "f16")
    lengths = [50, 0, 21]
    say("shared strides")
    kvp = torch.zeros(hkv, prefix, 2, dim, dtype=torch.float16, device="cuda")
    pkd, pvd = kvp[:, :, 0].transpose(0, 1), kvp[:, :, 1].transpose(0, 1)
    kv = torch.full((b, hkv, cap + 6, 2, dim), float("nan"), dtype=torch.float16, device="cuda")
    kd, vd = kv[:, :, :cap, 0].transpose(1, 2), kv[:, :, :cap, 1].transpose(1, 2)
    od = torch.full((hq, b, dim + 8), 7.0, dtype=torch.float16, device="cuda")
    for d, s in ((pkd, pk), (pvd, pv), (kd, k), (vd, v)):
        d.copy_(s)
    need = qmm.qmm_attn_shared_workspace_bytes(b, prefix, cap, hq, hkv, dim)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    o = qmm.qmm_attn_shared(q.cuda(), pkd, pvd, kd, vd, torch.tensor(lengths, dtype=torch.int32).cuda(),
                            O=od[..., :dim].transpose(0, 1), workspace=ws[:need])
    torch.cuda.synchronize()
    _check(q, pk, pv, k, v, lengths, "f16", "shared strides", o=o)
    assert bool((od[..., dim:] == 7.0).all()) and bool((ws[need:] == 0xFF).all())


def test_repeats_bit_for_bit_on_another_stream_and_replayed():
    b, prefix, cap = 9, 1000, 400
    q, pk, pv, k, v = (x.cuda() for x in _inputs(6, b, prefix, cap, 8, 2, 128, "bf16"))
    lengths = torch.tensor([i * 50 for i in range(b)], dtype=torch.int32).cuda()
    say("shared streams and graph")
    first = qmm.qmm_attn_shared(q, pk, pv, k, v, lengths)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = qmm.qmm_attn_shared(q, pk, pv, k, v, lengths, stream=s)
    s.synchronize()
    assert torch.equal(first, other)
    o = torch.zeros_like(q)
    ws = torch.zeros(qmm.qmm_attn_shared_workspace_bytes(b, prefix, cap, 8, 2, 128), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.qmm_attn_shared(q, pk, pv, k, v, lengths, O=o, workspace=ws)
    for i in range(3):  # the next step of a decode loop: longer caches, another query
        o.zero_()
        lengths.copy_((lengths + 37) % (cap + 1))
        q.copy_(q.roll(1, 0))
        want = qmm.qmm_attn_shared(q, pk, pv, k, v, lengths)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want), i


def test_offsets_past_32_bits():
    """A cache whose later sequences lie past 2^32 elements, and a prefix whose tokens do."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB")
    b, prefix, cap, dim = 5, 130, 40, 64
    q, pk, pv, k, v = _inputs(7, b, prefix, cap, 2, 1, dim, "f16")
    say("shared wide strides")
    big = torch.empty((b << 30) + (prefix << 25) // 8, dtype=torch.float16, device="cuda")
    kd = big.as_strided((b, cap, 1, dim), (1 << 30, 128, 128, 1))
    vd = big.as_strided((b, cap, 1, dim), (1 << 30, 128, 128, 1), 64)
    pkd = big.as_strided((prefix, 1, dim), (1 << 25, 128, 1), 1 << 20)
    pvd = big.as_strided((prefix, 1, dim), (1 << 25, 128, 1), (1 << 20) + 64)
    for d, s in ((kd, k), (vd, v), (pkd, pk), (pvd, pv)):
        d.copy_(s)
    lengths = [40, 3, 0, 17, 39]
    o = qmm.qmm_attn_shared(q.cuda(), pkd, pvd, kd, vd, torch.tensor(lengths, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    _check(q, pk, pv, k, v, lengths, "f16", "shared wide strides", o=o)
