"""qmm_lora against the 64-bit definition on the GPU."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.attn_oracle as O
from attn_util import TORCH, assert_within, f64, rng, rounded, say

pytestmark = pytest.mark.gpu


def _inputs(seed, n, k, rows, ad, rank, kind):
    r = rng(5, seed, n, k, rows, ad, rank)
    x = rounded(r.standard_normal((n, k)), kind)
    a = rounded(r.standard_normal((ad, rank, k)) / np.sqrt(k), "f16")
    b = rounded(r.standard_normal((ad, rows, rank)) / np.sqrt(rank), "f16")
    scales = torch.from_numpy(r.uniform(-2, 2, ad).astype(np.float32))
    base = torch.from_numpy(r.standard_normal((n, rows)).astype(np.float32))
    ids = r.integers(-1, ad, n)
    return x, a, b, scales, base, ids


def _ids(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def _check(x, a, b, scales, base, ids, what, **kw):
    say(what)
    y = qmm.qmm_lora(x.cuda(), a.cuda(), b.cuda(), _ids(ids), scales=None if scales is None else scales.cuda(),
                     base=None if base is None else base.cuda(), **kw)
    torch.cuda.synchronize()
    want, err = O.lora(f64(x), f64(a), f64(b), ids, None if scales is None else f64(scales),
                       None if base is None else f64(base))
    assert_within(y, want, err, what)
    return y


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 67])
@pytest.mark.parametrize("k,rows,rank", [(32, 1, 1), (64, 5, 3), (96, 64, 4), (256, 100, 16), (288, 67, 20),
                                         (1056, 260, 32), (512, 130, 64), (320, 36, 100), (64, 16, 256), (128, 77, 7)])
def test_against_the_definition(kind, n, k, rows, rank):
    x, a, b, scales, base, ids = _inputs(0, n, k, rows, 5, rank, kind)
    _check(x, a, b, scales, base, ids, f"lora {kind} n={n} k={k} rows={rows} rank={rank}")


@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_many_tiles_take_long_ranges(kind):
    """Enough tokens for the long ranges of k and several row steps per workgroup; one request per run of tokens."""
    n, k, rows = 4500, 1056, 260
    x, a, b, scales, base, _ = _inputs(1, n, k, rows, 6, 16, kind)
    ids = np.repeat([0, 3, -1, 5, 2], 900)
    _check(x, a, b, scales, base, ids, f"lora {kind} 4500 tokens")


def test_wide_k_split_over_rounds():
    x, a, b, scales, base, ids = _inputs(2, 3000, 4128, 64, 3, 40, "f16")
    _check(x, a, b, scales, base, ids, "lora 3000 tokens of 4128")


@pytest.mark.parametrize("n,pattern", [(512, "one"), (511, "mixed"), (513, "mixed"), (200, "runs"), (130, "late")])
def test_tiles_by_adapter(n, pattern):
    """Batches around the largest one whose tiles are gathered by adapter: all tokens on one adapter, adapters
    interleaved, in runs that cross the scan's steps of 64 tokens, or first met late in the batch."""
    ad = 7
    x, a, b, scales, base, ids = _inputs(8, n, 96, 40, ad, 12, "f16")
    ids = {"one": np.full(n, 3), "mixed": ids, "runs": np.arange(n) // 45 % ad,
           "late": np.where(np.arange(n) < n - 5, -1, np.arange(n) % ad)}[pattern]
    _check(x, a, b, scales, base, ids, f"lora {n} tokens, {pattern}")


def test_long_k_of_few_tokens():
    """More k than 256 ranges of the smallest size hold."""
    x, a, b, scales, base, ids = _inputs(9, 3, 256 * 256 + 4128, 16, 2, 3, "f32")
    _check(x, a, b, scales, base, ids, "lora k=69664")


def test_without_base_scales_or_adapters():
    x, a, b, scales, base, ids = _inputs(3, 20, 128, 48, 4, 8, "f32")
    _check(x, a, b, None, base, ids, "lora without scales")
    _check(x, a, b, scales, None, ids, "lora without base")
    y = _check(x, a, b, scales, base, [-1] * 20, "lora without adapters")
    assert torch.equal(y.cpu(), base)
    y = _check(x, a[:0], b[:0], scales[:0], base, [-1] * 20, "lora with an empty stack")
    assert torch.equal(y.cpu(), base)


def test_bad_ids_give_nan_rows():
    x, a, b, scales, base, ids = _inputs(4, 40, 64, 20, 4, 8, "f16")
    ids[[0, 7, 16, 39]] = [4, -2, 2 ** 31 - 1, -2 ** 31]
    _check(x, a, b, scales, base, ids, "lora bad ids")


def test_in_place_on_base_and_unaligned_rows():
    for rows in (64, 33):
        x, a, b, scales, base, ids = _inputs(5, 19, 96, rows, 3, 12, "f32")
        y = base.cuda()
        want, err = O.lora(f64(x), f64(a), f64(b), ids, f64(scales), f64(base))
        say(f"lora in place rows={rows}")
        qmm.qmm_lora(x.cuda(), a.cuda(), b.cuda(), _ids(ids), scales.cuda(), base=y, Y=y)
        torch.cuda.synchronize()
        assert_within(y, want, err, "in place")
        off = torch.zeros(19 * rows + 1, device="cuda")[1:].view(19, rows)  # Y only 4-byte aligned
        qmm.qmm_lora(x.cuda(), a.cuda(), b.cuda(), _ids(ids), scales.cuda(), base=base.cuda(), Y=off)
        boff = torch.zeros(b.numel() + 1, dtype=torch.float16, device="cuda")[1:].view(b.shape)  # B 2-byte aligned
        boff.copy_(b)
        other = qmm.qmm_lora(x.cuda(), a.cuda(), boff, _ids(ids), scales.cuda(), base=base.cuda())
        torch.cuda.synchronize()
        assert torch.equal(off, y) and torch.equal(other, y)


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("rank", [7, 16, 64, 100])
def test_tiles_of_several_adapters(kind, rank):
    """Prompts whose tiles of 64 tokens hold none, one, two, three and many adapters, with tokens without an adapter
    or with an id outside the stack among them, and a last tile that is not full."""
    n, k, rows, ad = 700, 288, 68, 7
    x, a, b, scales, base, ids = _inputs(9, n, k, rows, ad, rank, kind)
    t = np.arange(n)
    ids = np.where(t < 300, t // 45 % ad, np.where(t < 500, t // 20 % ad, ids))
    ids[:64], ids[64:130] = -1, 3
    ids[[5, 70, 199, 320]] = [ad, ad + 9, -7, 2 ** 31 - 1]
    ids[[64, 310, 640]] = -1
    _check(x, a, b, scales, base, ids, f"lora {kind} rank={rank}, tiles of several adapters")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_values_stay_with_their_tokens(bad):
    """A token's own non-finite activation, or an adapter's, reaches the rows that use it and no other."""
    x, a, b, scales, base, _ = _inputs(6, 33, 64, 40, 3, 8, "f32")
    ids = np.arange(33) % 4 - 1
    clean, err = O.lora(f64(x), f64(a), f64(b), ids, f64(scales), f64(base))
    x[5, 3] = bad          # token 5 has adapter 0
    a[1, 2, 9] = bad
    b[2, 4, 1] = bad
    say(f"lora {bad}")
    y = f64(qmm.qmm_lora(x.cuda(), a.cuda(), b.cuda(), _ids(ids), scales.cuda(), base=base.cuda()))
    assert not np.isfinite(y[5]).any()
    for t in range(33):
        if t == 5 or ids[t] == 1:
            continue
        cols = np.ones(40, bool)
        if ids[t] == 2:
            cols[4] = False
            assert not np.isfinite(y[t, 4])
        assert (np.abs(y[t] - clean[t])[cols] <= err[t][cols]).all(), t


def test_repeats_bit_for_bit_on_another_stream_and_replayed():
    x, a, b, scales, base, ids = _inputs(7, 50, 512, 200, 6, 16, "f16")
    x, a, b, scales, base, ids = x.cuda(), a.cuda(), b.cuda(), scales.cuda(), base.cuda(), _ids(ids)
    say("lora streams and graph")
    first = qmm.qmm_lora(x, a, b, ids, scales, base)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = qmm.qmm_lora(x, a, b, ids, scales, base, stream=s)
    s.synchronize()
    assert torch.equal(first, other)
    y = torch.zeros_like(base)
    ws = torch.full((qmm.qmm_lora_workspace_bytes(50, 512, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.qmm_lora(x, a, b, ids, scales, base, Y=y, workspace=ws)
    for i in range(3):
        ids.copy_((ids + 2) % 7 - 1)
        x.copy_(x.roll(1, 0))
        y.zero_()
        want = qmm.qmm_lora(x, a, b, ids, scales, base)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
