"""qmm_attn_prompt against the 64-bit definition on the GPU."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.attn_oracle as O
from attn_util import TORCH, assert_within, f64, rng, rounded, say

pytestmark = pytest.mark.gpu

KEPT = 7.0  # what rows that a call must leave alone hold


def _inputs(seed, n, hq, hkv, dim, kind, spread=1.0):
    r = rng(1, seed, n, hq, hkv, dim)
    q = rounded(spread * r.standard_normal((n, hq, dim)), kind)
    k = rounded(spread * r.standard_normal((n, hkv, dim)), kind)
    v = rounded(r.standard_normal((n, hkv, dim)), kind)
    return q, k, v


def _run(q, k, v, starts, scale=None):
    o = torch.full(q.shape, KEPT, dtype=q.dtype, device="cuda")
    qmm.qmm_attn_prompt(q.cuda(), k.cuda(), v.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), scale=scale, O=o)
    torch.cuda.synchronize()
    return o


def _check(q, k, v, starts, kind, what, scale=None, o=None):
    say(what)
    o = _run(q, k, v, starts, scale) if o is None else o
    want, err = O.attn_prompt(f64(q), f64(k), f64(v), starts, scale or q.shape[2] ** -0.5, kind)
    outside = np.isnan(want).all((1, 2))
    want[outside], err[outside] = KEPT, 0.0
    assert_within(o, want, err, what)


def _starts(lens, first=0):
    return [int(x) for x in first + np.concatenate([[0], np.cumsum(lens)])]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,hkv,lens", [
    (1, 1, [1]), (4, 1, [1, 1, 1]), (2, 2, [64]), (2, 2, [65]), (3, 1, [63, 2]), (8, 2, [31, 33, 32]),
    (4, 4, [129]), (7, 1, [40, 0, 1, 90]), (8, 8, [5, 0, 0, 17]), (6, 2, [200]), (33, 1, [9, 3]),
])
def test_against_the_definition(kind, dim, hq, hkv, lens):
    n = sum(lens)
    q, k, v = _inputs(0, n + 3, hq, hkv, dim, kind)
    _check(q, k, v, _starts(lens), kind, f"prompt {kind} dim={dim} heads={hq}/{hkv} lens={lens}")


@pytest.mark.parametrize("dim", [64, 128])
def test_many_sequences_and_an_offset_start(dim):
    """More sequences than one scan step holds, empty ones among them, the first behind other tokens."""
    lens = [(i * 5) % 4 for i in range(150)]
    n = sum(lens) + 9
    q, k, v = _inputs(2, n, 4, 2, dim, "f16")
    _check(q, k, v, _starts(lens, 5), "f16", f"prompt 150 sequences dim={dim}")


@pytest.mark.parametrize("n,hq,hkv,dim,kind", [(2300, 8, 2, 128, "f16"), (2300, 8, 2, 64, "bf16"),
                                               (4700, 32, 8, 128, "bf16"), (5003, 32, 8, 64, "f16")])
def test_long_sequence_sampled_rows(n, hq, hkv, dim, kind):
    """Rows in every block of a long sequence, compared one by one: few tiles, and more than run at once."""
    q, k, v = _inputs(3, n, hq, hkv, dim, kind)
    say(f"prompt one sequence of {n}, heads {hq}/{hkv} of {dim}")
    o = f64(_run(q, k, v, [0, n]))
    qn, kn, vn = f64(q), f64(k), f64(v)
    for t in list(range(0, n, n // 37)) + [n - 1]:
        for h in (0, 3, 4, hq - 1):
            g = h * hkv // hq
            want, err = O.attend(qn[t, h], kn[:t + 1, g], vn[:t + 1, g], dim ** -0.5, kind)
            assert (np.abs(o[t, h] - want) <= err).all(), (t, h)


@pytest.mark.parametrize("dim", [64, 128])
def test_many_short_sequences(dim):
    """More tiles than run at once, each with one block."""
    lens = [1 + i % 3 for i in range(700)]
    n = sum(lens)
    q, k, v = _inputs(12, n + 2, 4, 2, dim, "f16")
    _check(q, k, v, _starts(lens), "f16", f"prompt 700 short sequences dim={dim}")


@pytest.mark.parametrize("dim", [64, 128])
def test_many_tiles_with_masked_ends(dim):
    """The same with ragged lengths around block and tile borders."""
    lens = [63, 64, 65, 127, 128, 129, 1, 200] * 6
    n = sum(lens)
    q, k, v = _inputs(13, n, 64, 16, dim, "bf16")
    say(f"prompt 48 ragged sequences dim={dim}")
    o = f64(_run(q, k, v, _starts(lens)))
    qn, kn, vn = f64(q), f64(k), f64(v)
    for i, (b, e) in enumerate(zip(_starts(lens)[:-1], _starts(lens)[1:])):
        for t in {b, (b + e) // 2, e - 1}:
            for h in (0, 5 + i % 50, 63):
                want, err = O.attend(qn[t, h], kn[b:t + 1, h // 4], vn[b:t + 1, h // 4], dim ** -0.5, "bf16")
                assert (np.abs(o[t, h] - want) <= err).all(), (t, h)


@pytest.mark.parametrize("layout", ["interleaved", "head-major", "wide rows"])
def test_strides(layout):
    n, hq, hkv, dim, kind = 130, 4, 2, 64, "f16"
    q, k, v = _inputs(4, n, hq, hkv, dim, kind)
    starts = torch.tensor([0, 70, 130], dtype=torch.int32).cuda()
    if layout == "interleaved":
        buf = torch.zeros(n, hq + 2 * hkv, dim, dtype=TORCH[kind], device="cuda")
        qd, kd, vd = buf[:, :hq], buf[:, hq:hq + hkv], buf[:, hq + hkv:]
        o = torch.full((n, hq, dim), KEPT, dtype=TORCH[kind], device="cuda")
    elif layout == "head-major":
        qd, kd, vd = (torch.zeros(h, n, dim, dtype=TORCH[kind], device="cuda").transpose(0, 1) for h in (hq, hkv, hkv))
        o = torch.full((hq, n, dim), KEPT, dtype=TORCH[kind], device="cuda").transpose(0, 1)
    else:
        qd, kd, vd = (torch.full((n, h, dim + 24), 9.0, dtype=TORCH[kind], device="cuda")[..., 8:8 + dim]
                      for h in (hq, hkv, hkv))
        o = torch.full((n, hq, dim + 8), KEPT, dtype=TORCH[kind], device="cuda")[..., :dim]
    for d, s in ((qd, q), (kd, k), (vd, v)):
        d.copy_(s)
    say(f"prompt strides {layout}")
    qmm.qmm_attn_prompt(qd, kd, vd, starts, O=o)
    torch.cuda.synchronize()
    _check(q, k, v, [0, 70, 130], kind, f"prompt strides {layout}", o=o)
    if layout == "wide rows":
        assert bool((o.as_strided((n, hq, 8), (hq * (dim + 8), dim + 8, 1), dim) == KEPT).all())


@pytest.mark.parametrize("scale,spread", [(0.02, 1.0), (1.0, 1.0), (0.125, 6.0)])
def test_flat_and_peaked_weights(scale, spread):
    q, k, v = _inputs(5, 150, 2, 1, 64, "f16", spread)
    _check(q, k, v, [0, 150], "f16", f"prompt scale={scale} spread={spread}", scale=scale)


def test_scores_that_grow_and_fall_along_the_keys():
    """The running maximum moves in every block, or never after the first."""
    n, dim = 330, 64
    for sign in (1.0, -1.0):
        q = rounded(np.full((n, 1, dim), 0.5), "f16")
        k = rounded(sign * np.linspace(-2, 2, n)[:, None, None] * np.ones((n, 1, dim)), "f16")
        _, _, v = _inputs(6, n, 1, 1, dim, "f16")
        _check(q, k, v, [0, n], "f16", f"prompt monotone scores {sign}")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("more", [0, 600])
def test_nonfinite_values_of_later_tokens_stay_there(kind, bad, more):
    """A non-finite key or value reaches the rows from its token on, of its KV
    head, and no other; the tokens behind the last sequence reach none."""
    n, hq, hkv, dim = 140, 4, 2, 128
    q, k, v = _inputs(7, n + 20 + more, hq, hkv, dim, kind)
    starts = [0, 50, n] + list(range(n + 21, n + 21 + more))  # further sequences of one token
    clean, err = O.attn_prompt(f64(q), f64(k), f64(v), starts, dim ** -0.5, kind)
    for which, t in ((v, 77), (v, 130), (k, 90), (v, 20)):
        keep = which[t, 1].clone()
        which[t, 1, 5] = bad
        for x in (q, k, v):
            x[n:n + 20] = bad
        say(f"prompt {kind} {bad} at token {t}, {more} more sequences")
        o = f64(_run(q, k, v, starts))
        end = 50 if t < 50 else n
        free = np.ones((n, hq), bool)
        free[t:end, 2:] = False
        assert (np.abs(o[:n] - clean[:n])[free] <= err[:n][free]).all(), (t, bad)
        if which is v:  # the column itself is non-finite, the others are as they were
            assert not np.isfinite(o[t:end, 2:, 5]).any()
            cols = [c for c in range(dim) if c != 5]
            assert (np.abs(o[t:end, 2:] - clean[t:end, 2:])[..., cols] <= err[t:end, 2:][..., cols]).all()
        which[t, 1] = keep


@pytest.mark.parametrize("hq,hkv,dim", [(4, 1, 64), (2, 2, 128)])
def test_sequences_of_many_and_few_tiles(hq, hkv, dim):
    """Tiles are taken in order of their length across 64 sequences at a time: every one exactly once."""
    lens = [300, 0, 1, 611, 64, 40, 259] + [3] * 60 + [290, 0, 128] + [1, 33] * 5
    q, k, v = _inputs(11, sum(lens) + 5, hq, hkv, dim, "f16")
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    say(f"prompt many and few tiles {hq}/{hkv} dim={dim}")
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    qmm.qmm_attn_prompt(q.cuda(), k.cuda(), v.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), O=o)
    torch.cuda.synchronize()
    want, err = O.attn_prompt(f64(q), f64(k), f64(v), starts, dim ** -0.5, "f16")
    assert bool((o[starts[-1]:] == 7.0).all())
    assert_within(o[:starts[-1]], want[:starts[-1]], err[:starts[-1]], "many and few tiles")


def test_rows_outside_and_bad_starts():
    """A sequence whose ends are out of order or outside the tokens is left out; its rows stay."""
    n = 60
    q, k, v = _inputs(8, n, 2, 2, 64, "f16")
    for starts in ([0, 20, 20, 10, 40], [5, 30], [0, 30, 61], [-3, 10, 30], [0, 0, 0], [60, 60]):
        say(f"prompt starts {starts}")
        o = f64(_run(q, k, v, starts))
        want, err = O.attn_prompt(f64(q), f64(k), f64(v), starts, 0.125, "f16")
        out = np.isnan(want).all((1, 2))
        if starts == [0, 20, 20, 10, 40]:  # two sequences overlap on tokens 10..19: either's rows
            out[10:20] = True
            assert (np.abs(o - want)[~out] <= err[~out]).all()
            continue
        assert (o[out] == KEPT).all() and (np.abs(o - want)[~out] <= err[~out]).all()


def test_repeats_bit_for_bit_on_another_stream_and_replayed():
    n, lens = 700, [300, 1, 399]
    q, k, v = (x.cuda() for x in _inputs(9, n, 8, 2, 128, "bf16"))
    starts = torch.tensor(_starts(lens), dtype=torch.int32).cuda()
    say("prompt streams and graph")
    first = qmm.qmm_attn_prompt(q, k, v, starts)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = qmm.qmm_attn_prompt(q, k, v, starts, stream=s)
    s.synchronize()
    assert torch.equal(first, other)
    o = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.qmm_attn_prompt(q, k, v, starts, O=o)
    for i in range(3):
        o.zero_()
        q.copy_(q.roll(1, 0))
        want = qmm.qmm_attn_prompt(q, k, v, starts)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want), i


def test_offsets_past_32_bits():
    """Keys and values whose token stride puts the later ones past 2^31 elements."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    n, dim, stride = 300, 64, 1 << 23
    q, k, v = _inputs(10, n, 2, 1, dim, "f16")
    say("prompt wide token stride")
    buf = torch.empty(n * stride + 128, dtype=torch.float16, device="cuda")
    kd, vd = buf.as_strided((n, 1, dim), (stride, dim, 1)), buf.as_strided((n, 1, dim), (stride, dim, 1), 64)
    kd.copy_(k), vd.copy_(v)
    o = qmm.qmm_attn_prompt(q.cuda(), kd, vd, torch.tensor([0, n], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    _check(q, k, v, [0, n], "f16", "prompt wide token stride", o=o)
