"""qmm_lora above 512 tokens, where a tile of 64 consecutive tokens may hold several
adapters: what one token or adapter holds stays with the tokens that use it, Y may
be base, and rows and stacks may be aligned to their elements only."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.attn_oracle as O
from attn_util import assert_within, f64, rng, rounded, say

pytestmark = pytest.mark.gpu


def _inputs(seed, n, k, rows, ad, rank, kind):
    r = rng(60, seed, n, k, rows, ad, rank)
    x = rounded(r.standard_normal((n, k)), kind)
    a = rounded(r.standard_normal((ad, rank, k)) / np.sqrt(k), "f16")
    b = rounded(r.standard_normal((ad, rows, rank)) / np.sqrt(rank), "f16")
    scales = torch.from_numpy(r.uniform(-2, 2, ad).astype(np.float32))
    base = torch.from_numpy(r.standard_normal((n, rows)).astype(np.float32))
    return x, a, b, scales, base


def _ids(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def _layout(pattern, n, ad):
    """Adapters that alternate, in runs that end inside tiles, or one per tile but for a few tokens."""
    t = np.arange(n)
    return {"alternating": t % (ad + 1) - 1, "runs": t // 23 % (ad + 1) - 1,
            "one but a few": np.where(t % 50 == 7, t // 50 % ad, t // 64 % ad)}[pattern]


def _lora(x, a, b, ids, scales, base, **kw):
    y = qmm.qmm_lora(x.cuda(), a.cuda(), b.cuda(), _ids(ids), scales.cuda(), base=base.cuda(), **kw)
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("rank", [8, 7, 64, 100])
@pytest.mark.parametrize("pattern", ["alternating", "runs", "one but a few"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_values_stay_with_their_tokens(kind, rank, pattern, bad):
    n, k, rows, ad = 580, 288, 40, 4
    x, a, b, scales, base = _inputs(1, n, k, rows, ad, rank, kind)
    ids = _layout(pattern, n, ad)
    clean, err = O.lora(f64(x), f64(a), f64(b), ids, f64(scales), f64(base))
    token = int(np.flatnonzero(ids == 0)[5])
    x[token, 3] = bad
    a[1, 2, 9] = bad
    b[2, 4, 1] = bad
    none = np.flatnonzero(ids == -1)
    if none.size:  # a token without an adapter: its X is used nowhere
        x[none[0]] = bad
    say(f"lora {kind} rank={rank}, {pattern}, {bad} among {n} tokens")
    y = f64(_lora(x, a, b, ids, scales, base))
    assert not np.isfinite(y[token]).any()
    cols = np.ones((n, rows), bool)
    cols[token], cols[ids == 1] = False, False
    cols[ids == 2, 4] = False
    assert not np.isfinite(y[ids == 2, 4]).any()
    assert (np.abs(y - clean)[cols] <= err[cols]).all()


@pytest.mark.parametrize("rank", [12, 7])
@pytest.mark.parametrize("rows", [64, 33])
@pytest.mark.parametrize("pattern", ["alternating", "runs"])
def test_in_place_on_base_and_unaligned_rows(rank, rows, pattern):
    n, k, ad = 660, 96, 5
    x, a, b, scales, base = _inputs(2, n, k, rows, ad, rank, "f32")
    ids = _layout(pattern, n, ad)
    want, err = O.lora(f64(x), f64(a), f64(b), ids, f64(scales), f64(base))
    say(f"lora in place rank={rank} rows={rows}, {pattern}")
    y = base.cuda()
    args = x.cuda(), a.cuda(), b.cuda(), _ids(ids), scales.cuda()
    qmm.qmm_lora(*args, base=y, Y=y)
    torch.cuda.synchronize()
    assert_within(y, want, err, "in place")
    buf = torch.full((n * rows + 5,), 7.0, device="cuda")
    off = buf[1:1 + n * rows].view(n, rows)  # Y only 4-byte aligned
    qmm.qmm_lora(*args, base=base.cuda(), Y=off)
    boff = torch.zeros(b.numel() + 1, dtype=torch.float16, device="cuda")[1:].view(b.shape)  # B 2-byte aligned
    boff.copy_(b)
    other = qmm.qmm_lora(args[0], args[1], boff, *args[3:], base=base.cuda())
    base_off = torch.zeros(n * rows + 3, device="cuda")[3:].view(n, rows)  # base only 4-byte aligned
    base_off.copy_(base)
    third = qmm.qmm_lora(*args, base=base_off)
    torch.cuda.synchronize()
    assert torch.equal(off, y) and torch.equal(other, y) and torch.equal(third, y)
    assert bool((buf[0] == 7).all()) and bool((buf[1 + n * rows:] == 7).all())


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("rank", [5, 33, 128, 200, 256])
def test_ranks_and_adapters_per_tile(kind, rank):
    """Every tile with as many adapters as the stack has, one token of each."""
    n, k, rows, ad = 513, 160, 36, 64
    x, a, b, scales, base = _inputs(3, n, k, rows, ad, rank, kind)
    ids = rng(61, rank).permutation(np.arange(n) % ad)
    say(f"lora {kind} rank={rank}, 64 adapters among 513 tokens")
    want, err = O.lora(f64(x), f64(a), f64(b), ids, f64(scales), f64(base))
    assert_within(_lora(x, a, b, ids, scales, base), want, err, "64 adapters")


def test_repeats_bit_for_bit_and_replayed():
    n, k, rows, ad, rank = 700, 512, 200, 6, 16
    x, a, b, scales, base = (t.cuda() for t in _inputs(4, n, k, rows, ad, rank, "f16"))
    ids = _ids(_layout("runs", n, ad))
    say("lora 700 tokens, graph")
    first = qmm.qmm_lora(x, a, b, ids, scales, base)
    y = torch.zeros_like(base)
    ws = torch.full((qmm.qmm_lora_workspace_bytes(n, k, rank),), 0xFF, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.qmm_lora(x, a, b, ids, scales, base, Y=y, workspace=ws)
    for i in range(4):
        y.zero_()
        want = qmm.qmm_lora(x, a, b, ids, scales, base)
        torch.cuda.synchronize()
        assert i > 0 or torch.equal(want, first)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
        ids.copy_((ids + 2) % 7 - 1)
        x.copy_(x.roll(1, 0))
