"""qmm_kv4_append and qmm_kv4_read on the GPU against the 64-bit definition:
codes and scales are compared bit for bit, over the whole cache, so that
places which no token takes are seen to stay as they were."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.serve_oracle as S
from attn_util import TORCH, assert_within, f64, rng, rounded, say

pytestmark = pytest.mark.gpu


def freqs_of(n, base=10000.0):
    return [base ** (-i / max(n, 1)) for i in range(n)]


def run_append(k, v, cache, page, slots, positions=None, weight=None, **kw):
    c = torch.from_numpy(cache).cuda()
    if positions is not None:
        kw["positions"] = torch.from_numpy(positions).cuda()
    if weight is not None:
        kw["weight"] = weight.cuda()
    qmm.qmm_kv4_append(k.cuda(), v.cuda(), c, page, torch.from_numpy(slots).cuda(), **kw)
    torch.cuda.synchronize()
    return c.cpu().numpy()


def check_append(k, v, cache, page, slots, **kw):
    got = run_append(k, v, cache, page, slots, **kw)
    w = kw.pop("weight", None)
    want = S.append(f64(k), f64(v), cache, page, slots, weight=None if w is None else f64(w), **kw)
    diff = np.argwhere(got != want)
    assert len(diff) == 0, f"{len(diff)} bytes differ, first at {diff[:4].tolist()}"


def old_cache(g, pages, page, heads, dim):
    return g.integers(0, 256, (pages, S.page_bytes(page, heads, dim)), dtype=np.uint8)


CASES = [
    # tokens, heads, dim, page, type, rotated pairs, pairs, norm
    (1, 8, 128, 16, "f32", 64, "halves", False),
    (7, 3, 64, 32, "f16", 32, "neighbours", True),
    (33, 5, 128, 64, "bf16", 16, "halves", True),
    (20, 1, 64, 16, "f32", 5, "halves", True),
    (9, 9, 64, 128, "f16", 7, "neighbours", False),
    (40, 2, 128, 256, "f32", 0, "halves", False),
    (300, 2, 64, 16, "bf16", 32, "halves", False),
    (5, 4, 128, 16, "f16", 64, "neighbours", True),
]


@pytest.mark.parametrize("n,heads,dim,page,kind,rot,pairs,norm", CASES)
def test_append_bytes(n, heads, dim, page, kind, rot, pairs, norm):
    g = rng(n, heads, dim, page, rot)
    say(f"append {n} {heads} {dim} {page} {kind} {rot} {pairs} {norm}")
    pages = n // page + 3
    k, v = (rounded(2 * g.standard_normal((n, heads, dim)), kind) for _ in range(2))
    slots = g.permutation(pages * page - 1)[:n].astype(np.int32)
    slots[-1] = pages * page - 1
    if n > 5:
        slots[1], slots[2], slots[3] = -1, pages * page, 2 ** 31 - 1  # left out
    kw = {}
    if rot:
        kw = dict(positions=g.integers(-2 ** 31, 2 ** 31, n).astype(np.int32), freqs=freqs_of(rot), pairs=pairs)
    if norm:
        kw.update(norm=True, weight=rounded(1 + 0.3 * g.standard_normal(dim), "f32"))
    check_append(k, v, old_cache(g, pages, page, heads, dim), page, slots, **kw)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_append_strides(kind, dim):
    """Keys and values out of one product's rows, heads at odd distances, and one key row for all tokens."""
    g = rng(4, dim)
    n, heads, page = 12, 3, 16
    slots = g.permutation(2 * page)[:n].astype(np.int32)
    for row, off in ((2 * heads * dim, 0), (2 * heads * dim + 3, 1)):
        say(f"append strides {kind} {dim} {row} {off}")
        buf = rounded(g.standard_normal(n * row + off), kind)
        rows = buf[off:].view(n, row)
        k = rows[:, :heads * dim].view(n, heads, dim)
        v = rows[:, heads * dim:2 * heads * dim].view(n, heads, dim)
        cache = old_cache(g, 2, page, heads, dim)
        pos = g.integers(0, 5000, n).astype(np.int32)
        dev = buf.cuda()
        r = dev[off:].view(n, row)
        c = torch.from_numpy(cache).cuda()
        qmm.qmm_kv4_append(r[:, :heads * dim].view(n, heads, dim), r[:, heads * dim:2 * heads * dim].view(n, heads, dim),
                           c, page, torch.from_numpy(slots).cuda(), positions=torch.from_numpy(pos).cuda(),
                           freqs=freqs_of(dim // 2))
        want = S.append(f64(k), f64(v), cache, page, slots, positions=pos, freqs=freqs_of(dim // 2))
        assert np.array_equal(c.cpu().numpy(), want)
    one = rounded(g.standard_normal((1, heads, dim)), kind)
    got = run_append(one.expand(n, heads, dim), one.expand(n, heads, dim), cache, page, slots)
    many = one.expand(n, heads, dim).contiguous()
    assert np.array_equal(got, S.append(f64(many), f64(many), cache, page, slots))


def test_append_special_blocks():
    """Zeros, ties of magnitude, exact borders, infinities, NaNs, values at and past the scale's range, subnormals."""
    say("append special blocks")
    rows = []
    for fill in (0.0, -0.0, 3.0, -3.0, 1e-8, 3e-7, 5e-7, 524032.0, 524100.0, 1e30, 3.4e38, 1e-45, -1e-40):
        rows.append(np.full(32, fill))
    tie = np.linspace(-1, 1, 32)
    rows += [tie, -tie, np.roll(tie, 5)]
    for d in (1.0, -0.25, 0.333251953125):  # every border exactly, and its neighbours
        b = np.array([d * (c - 0.5) for c in range(-7, 8)])
        r = np.concatenate([b, np.nextafter(b.astype(np.float32), np.float32(np.inf)).astype(np.float64), [-8 * d, 0.0]])
        rows.append(r)
        rows.append(np.concatenate([np.nextafter(b.astype(np.float32), np.float32(-np.inf)).astype(np.float64), b, [-8 * d, 0.1]]))
    for bad in (np.nan, np.inf, -np.inf):
        r = np.arange(32.0)
        r[17] = bad
        rows.append(r)
    while len(rows) % 2:
        rows.append(np.ones(32))
    x = np.array(rows).reshape(-1, 1, 64).astype(np.float32)
    n = len(x)
    k = torch.from_numpy(x)
    cache = old_cache(rng(9), 4, 16, 1, 64)
    check_append(k, k.clone(), cache, 16, np.arange(n, dtype=np.int32))
    # a bad element reaches the blocks it is rotated into, and the whole head where it is normed
    pos = np.arange(n, dtype=np.int32)
    got = run_append(k, k, cache, 16, np.arange(n, dtype=np.int32), positions=pos, freqs=freqs_of(32), norm=True)
    kk = torch.full((n, 1, 64), 7.0)
    kv, _ = qmm.qmm_kv4_read(torch.from_numpy(got).cuda(), 16, torch.arange(n, dtype=torch.int32).cuda(), K=kk.cuda())
    assert np.array_equal(np.isnan(f64(kv)).all(-1)[:, 0], ~np.isfinite(x).all((1, 2)))


def test_append_extreme_angles():
    say("append extreme angles")
    g = rng(10)
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789], np.int32)
    n = len(pos)
    k = rounded(g.standard_normal((n, 2, 64)), "f32")
    fr = [64.0, -64.0, 0.0, 3.141592653589793, 1e-9, 5e-324, 1.0] + [0.1 * i for i in range(25)]
    check_append(k, k.clone(), old_cache(g, 1, 16, 2, 64), 16, np.arange(n, dtype=np.int32), positions=pos, freqs=fr)


def test_append_same_slot_twice_leaves_others():
    say("append one slot twice")
    g = rng(11)
    k = rounded(g.standard_normal((64, 2, 64)), "f32")
    cache = old_cache(g, 2, 16, 2, 64)
    slots = np.full(64, 5, np.int32)
    got = run_append(k, k, cache, 16, slots)
    free = np.array([s for s in range(32) if s != 5], np.int32)
    a, b = S.read(got, 16, free, 2, 64), S.read(cache, 16, free, 2, 64)
    assert all(np.array_equal(x, y, equal_nan=True) for x, y in zip(a, b))


def test_append_empty_and_large_offset():
    say("append no tokens")
    c = torch.zeros(2, qmm.qmm_kv4_page_bytes(16, 1, 64), dtype=torch.uint8, device="cuda")
    e = torch.zeros(0, 1, 64, device="cuda")
    i = torch.zeros(0, dtype=torch.int32, device="cuda")
    qmm.qmm_kv4_append(e, e, c, 16, i)
    k, v = qmm.qmm_kv4_read(c, 16, i, 1, 64)
    assert k.shape == (0, 1, 64) and v.shape == (0, 1, 64)
    say("append into a cache of more than 2^32 bytes")
    heads, dim, page = 8, 128, 256
    size = qmm.qmm_kv4_page_bytes(page, heads, dim)
    pages = 2 ** 33 // size + 2
    c = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
    g = rng(12)
    k = rounded(g.standard_normal((3, heads, dim)), "f16")
    slots = np.array([pages * page - 1, pages * page // 2 + 7, 3], np.int32)
    qmm.qmm_kv4_append(k.cuda(), (2 * k).cuda(), c, page, torch.from_numpy(slots).cuda())
    kr, vr = qmm.qmm_kv4_read(c, page, torch.from_numpy(slots).cuda(), heads, dim)
    small = S.append(f64(k), 2 * f64(k), np.zeros((1, size), np.uint8), page, np.arange(3, dtype=np.int32))
    wk, wv, _, _ = S.read(small, page, np.arange(3), heads, dim)
    assert np.array_equal(f64(kr), wk) and np.array_equal(f64(vr), wv)
    q = rounded(g.standard_normal((2, 16, dim)), "f16")
    table = torch.tensor([[pages - 1], [pages // 2]], dtype=torch.int32, device="cuda")
    o = qmm.qmm_attn_kv4(q.cuda(), c, page, heads, table, torch.tensor([256, 9], dtype=torch.int32, device="cuda"))
    host = torch.stack([c[pages - 1], c[pages // 2]]).cpu().numpy()
    want, err = S.attn_kv4(f64(q), host, page, heads, np.array([[0], [1]]), [256, 9], dim ** -0.5, "f16")
    assert_within(o, want, err, "attention at large offsets")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
def test_read_values(kind, dim, page):
    g = rng(20, dim)
    heads, pages = 3, 3
    cache = old_cache(g, pages, page, heads, dim)  # any bytes: scales of all kinds, infinities and NaNs among them
    slots = np.concatenate([g.permutation(pages * page)[:17], [-1, pages * page, -2 ** 31]]).astype(np.int32)
    say(f"read {kind} {dim} {page}")
    c, s = torch.from_numpy(cache).cuda(), torch.from_numpy(slots).cuda()
    wk, wv, _, _ = S.read(cache, page, slots, heads, dim)
    k, v = qmm.qmm_kv4_read(c, page, s, heads, dim, TORCH[kind])
    for got, want in ((k, wk), (v, wv)):
        ref = torch.from_numpy(want).to(torch.float32).to(TORCH[kind])
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got.cpu().float(), 0.0), torch.nan_to_num(ref.float(), 0.0))
    # strided outputs, one of the two alone, and what lies between the heads stays
    buf = torch.full((len(slots), heads, dim + 5), 7.0, dtype=TORCH[kind], device="cuda")
    out = buf[:, :, 1:dim + 1]
    qmm.qmm_kv4_read(c, page, s, V=out)
    assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(v))
    assert bool((buf[:, :, 0] == 7).all()) and bool((buf[:, :, dim + 1:] == 7).all())


def test_append_other_stream_and_graph():
    """On a stream of its own, and captured: replays take the slots and positions of the moment."""
    say("append stream and graph")
    g = rng(30)
    n, heads, dim, page = 6, 2, 128, 32
    k, v = (rounded(g.standard_normal((n, heads, dim)), "f16").cuda() for _ in range(2))
    cache = old_cache(g, 2, page, heads, dim)
    c = torch.from_numpy(cache).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    qmm.qmm_kv4_append(k, v, c, page, slots, positions=pos, freqs=freqs_of(64), stream=side)
    torch.cuda.synchronize()
    want = S.append(f64(k), f64(v), cache, page, np.arange(n), positions=np.arange(n), freqs=freqs_of(64))
    assert np.array_equal(c.cpu().numpy(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.qmm_kv4_append(k, v, c, page, slots, positions=pos, freqs=freqs_of(64))
    for step in range(3):
        slots.add_(n)
        pos.add_(100)
        graph.replay()
        torch.cuda.synchronize()
        want = S.append(f64(k), f64(v), want, page, slots.cpu().numpy(), positions=pos.cpu().numpy(), freqs=freqs_of(64))
        assert np.array_equal(c.cpu().numpy(), want), step
