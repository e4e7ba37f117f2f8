"""qmm_attn_kv4 on the GPU against the 64-bit definition, every output within
the bound that the stated numerics give."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.serve_oracle as S
from attn_util import assert_within, f64, rng, rounded, say

pytestmark = pytest.mark.gpu


def make_cache(g, pages, page, heads, dim, spread=0.3):
    """Codes like those of normal values, scales of both signs."""
    tiles = np.zeros((pages, heads * page // 16, 18 * dim), np.uint8)
    codes = np.clip(np.rint(8.5 + 3.3 * g.standard_normal((*tiles.shape[:2], 32 * dim))), 0, 15).astype(np.uint8)
    tiles[..., :16 * dim] = codes[..., ::2] | codes[..., 1::2] << 4
    d = spread * (0.5 + g.random((*tiles.shape[:2], dim))) * g.choice([-1.0, 1.0], (*tiles.shape[:2], dim))
    tiles[..., 16 * dim:] = d.astype(np.float16).view(np.uint8)
    return tiles.reshape(pages, -1)


def scales_at(cache, page, heads, dim, slot, head, which):
    """A writable view of the scales [dim / 32] of a slot's head (0: keys, 1: values)."""
    p, at, t = S.place(slot, page, heads, head, dim)
    tile = cache[p, at:at + 18 * dim]
    return tile[(16 + which) * dim:(17 + which) * dim].view(np.float16).reshape(dim // 32, 16)[:, t]


def setup(g, lens, page, hq, heads, dim, kind, width=None):
    width = width or max(1, -(-max(lens) // page))
    used = [-(-x // page) for x in lens]
    cache = make_cache(g, sum(used) + 2, page, heads, dim)
    order = g.permutation(sum(used) + 2)
    tables = g.integers(-5, 10 ** 6, (len(lens), width)).astype(np.int32)  # entries past a length are not used
    at = 0
    for i, m in enumerate(used):
        tables[i, :m] = order[at:at + m]
        at += m
    return rounded(g.standard_normal((len(lens), hq, dim)), kind), cache, tables


def run(q, cache, page, heads, tables, lens, **kw):
    o = qmm.qmm_attn_kv4(q if q.is_cuda else q.cuda(), torch.from_numpy(cache).cuda(), page, heads,
                         torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), **kw)
    torch.cuda.synchronize()
    return o


def check(q, cache, page, heads, tables, lens, kind, what, scale=None, **kw):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    o = run(q, cache, page, heads, tables, lens, scale=scale, **kw)
    want, err = S.attn_kv4(f64(q), cache, page, heads, tables, lens, scale, kind)
    assert_within(o, want, err, what)
    return o


EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 255, 256, 257]


@pytest.mark.parametrize("dim,kind,page", [(64, "f16", 16), (64, "bf16", 64), (128, "f16", 32), (128, "bf16", 256)])
def test_lengths(dim, kind, page):
    g = rng(1, dim, page)
    say(f"attn_kv4 lengths {dim} {kind} {page}")
    q, cache, tables = setup(g, EDGES, page, 4, 2, dim, kind)
    check(q, cache, page, 2, tables, EDGES, kind, "lengths")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 8, 9, 12, 17])
def test_groups(dim, group):
    """Groups that fill a column tile in part, one, two, and several workgroups' tiles."""
    g = rng(2, dim, group)
    lens = [70, 3, 130]
    say(f"attn_kv4 group {group} {dim}")
    q, cache, tables = setup(g, lens, 16, 2 * group, 2, dim, "f16")
    check(q, cache, 16, 2, tables, lens, "f16", "group")


@pytest.mark.parametrize("dim,lens", [(128, [3000]), (64, [2500, 0, 700, 1]), (128, [1025, 1279, 511, 512, 513])])
def test_split_rows(dim, lens):
    """Few rows: their keys are split over workgroups; short ones over fewer."""
    g = rng(3, dim, len(lens))
    say(f"attn_kv4 split {dim} {lens}")
    q, cache, tables = setup(g, lens, 64, 8, 2, dim, "f16", width=64)
    assert qmm.qmm_attn_kv4_workspace_bytes(len(lens), 8, 2, dim, 64, 64) > 0
    check(q, cache, 64, 2, tables, lens, "f16", "split")


def test_many_rows_one_workgroup_each():
    g = rng(4)
    lens = [int(x) for x in g.integers(0, 90, 300)]
    say("attn_kv4 300 rows")
    q, cache, tables = setup(g, lens, 16, 8, 4, 64, "bf16")
    assert qmm.qmm_attn_kv4_workspace_bytes(300, 8, 4, 64, tables.shape[1], 16) == 0
    check(q, cache, 16, 4, tables, lens, "bf16", "many rows")


def test_strides_and_in_place():
    g = rng(5)
    lens, hq, heads, dim, page = [100, 33, 500], 6, 2, 128, 32
    q, cache, tables = setup(g, lens, page, hq, heads, dim, "f16", width=40)
    want = run(q, cache, page, heads, tables, lens)
    say("attn_kv4 strides")
    buf = torch.full((3, 10, 136), 7.0, dtype=torch.float16, device="cuda")
    view = buf[:, 2:8, :dim]
    view.copy_(q)
    out = torch.full((hq, 3, dim + 8), 7.0, dtype=torch.float16, device="cuda")
    o = out[:, :, 8:].transpose(0, 1)
    run(view, cache, page, heads, tables, lens, O=o)
    assert torch.equal(o, want) and bool((out[:, :, :8] == 7).all())
    say("attn_kv4 in place")
    run(view, cache, page, heads, tables, lens, O=view)
    assert torch.equal(view, want)
    rest = buf.clone()
    rest[:, 2:8, :dim] = 7.0
    assert bool((rest == 7).all())


def test_one_table_for_several_tokens():
    """Drafted tokens of one sequence: one table for all rows, lengths one apart."""
    g = rng(6)
    n = 5
    q, cache, tables = setup(g, [400], 16, 8, 2, 64, "f16")
    q = rounded(g.standard_normal((n, 8, 64)), "f16")
    lens = [396 + i for i in range(n)]
    say("attn_kv4 one table")
    t = torch.from_numpy(tables).cuda().expand(n, -1)
    assert t.stride(0) == 0 or n == 1
    o = qmm.qmm_attn_kv4(q.cuda(), torch.from_numpy(cache).cuda(), 16, 2, t, torch.tensor(lens, dtype=torch.int32).cuda())
    want, err = S.attn_kv4(f64(q), cache, 16, 2, np.repeat(tables, n, 0), lens, 0.125, "f16")
    assert_within(o, want, err, "one table")


def test_bad_lengths_and_pages():
    g = rng(7)
    lens = [100, 100, 100, 100, 100, 0, 100]
    for width in (7, 200):  # without and with split rows
        q, cache, tables = setup(g, lens, 16, 4, 1, 64, "f16", width=width)
        lens2 = list(lens)
        lens2[1], lens2[2] = -1, width * 16 + 1
        tables[3, 6], tables[4, 0] = -1, cache.shape[0]
        tables[5, 0] = -7  # a length of 0 uses no page
        say(f"attn_kv4 bad lengths and pages, width {width}")
        o = check(q, cache, 16, 1, tables, lens2, "f16", "bad")
        assert bool(torch.isnan(o[1:5]).all()) and not bool(torch.isnan(o[[0, 5, 6]]).any())


def test_empty_calls():
    g = rng(8)
    q, cache, tables = setup(g, [5], 16, 4, 1, 64, "f16")
    c = torch.from_numpy(cache).cuda()
    say("attn_kv4 no rows, no table")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    o = qmm.qmm_attn_kv4(q[:0].cuda(), c, 16, 1, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), none)
    assert o.shape == (0, 4, 64)
    lens = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    o = qmm.qmm_attn_kv4(torch.cat([q, q]).cuda(), c, 16, 1, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), lens)
    assert bool((o[0] == 0).all()) and bool(torch.isnan(o[1]).all())


@pytest.mark.parametrize("dim", [64, 128])
def test_places_past_the_length_hold_anything(dim):
    g = rng(9, dim)
    lens = [37, 64, 81, 300]
    q, cache, tables = setup(g, lens, 32, 8, 2, dim, "f16")
    clean = run(q, cache, 32, 2, tables, lens)
    bad = cache.copy()
    for i, n in enumerate(lens):
        for u in range(n, -(-n // 32) * 32):
            for h in range(2):
                slot = int(tables[i, u // 32]) * 32 + u % 32
                for which, v in ((0, np.nan), (1, np.nan)):
                    scales_at(bad, 32, 2, dim, slot, h, which)[:] = v if u % 3 else np.inf
    say(f"attn_kv4 stale places {dim}")
    assert torch.equal(run(q, bad, 32, 2, tables, lens), clean)


@pytest.mark.parametrize("dim", [64, 128])
def test_nonfinite_blocks(dim):
    """A key that is a NaN reaches all outputs of its rows, a value's block its own 32 elements, of its head alone."""
    g = rng(10, dim)
    lens = [90, 90]
    q, cache, tables = setup(g, lens, 16, 4, 2, dim, "f16")
    scales_at(cache, 16, 2, dim, int(tables[0, 2]) * 16 + 3, 0, 0)[1] = np.nan
    scales_at(cache, 16, 2, dim, int(tables[1, 4]) * 16 + 9, 1, 1)[0] = np.nan
    say(f"attn_kv4 NaN blocks {dim}")
    o = run(q, cache, 16, 2, tables, lens)
    want = np.zeros((2, 4, dim), bool)
    want[0, :2] = True
    want[1, 2:, :32] = True
    assert np.array_equal(np.isnan(f64(o)), want)
    q[1, 0, 5] = float("inf")
    q[0, 3, 0] = float("nan")
    want[1, 0] = want[0, 3] = True
    o = run(q, cache, 16, 2, tables, lens)
    assert np.array_equal(np.isnan(f64(o)), want)


@pytest.mark.parametrize("kind,size", [("bf16", 1e30), ("bf16", 3e38), ("bf16", 1e-30), ("bf16", 1e-39), ("f16", 6e4),
                                       ("f16", 1e-7)])
def test_query_sizes(kind, size):
    """Queries at the ends of their type: scores of any size, one key's weight 1 or all keys' the same."""
    g = rng(11)
    lens = [200, 40]
    q, cache, tables = setup(g, lens, 16, 4, 1, 128, kind)
    q = rounded(np.clip(f64(q), -1, 1) * size, kind)
    say(f"attn_kv4 queries of {size} {kind}")
    o = run(q, cache, 16, 1, tables, lens)
    want, err = S.attn_kv4(f64(q), cache, 16, 1, tables, lens, 128 ** -0.5, kind)
    if size > 1e20:  # far beyond fp32's steps: the largest score's value, if no other is near
        err = np.where(err > 1, 2.0 ** -7 * np.abs(want) + 2.0 ** -7, err)
    assert_within(o, want, err, "query size")


@pytest.mark.parametrize("sizes", [(60000.0, 1e-4), (1e-4, 60000.0), (6e-8, 6e-8), (1.0, 0.0)])
@pytest.mark.parametrize("dim", [64, 128])
def test_value_scales_of_all_sizes(sizes, dim):
    """Scales that change by a factor of 10^8 along the sequence, the keys there attended to or not."""
    g = rng(12, dim)
    lens = [640, 200]
    q, cache, tables = setup(g, lens, 64, 2, 1, dim, "bf16")
    for i, n in enumerate(lens):
        for u in range(n):
            s = scales_at(cache, 64, 1, dim, int(tables[i, u // 64]) * 64 + u % 64, 0, 1)
            s[:] = s * np.float16(sizes[0]) if u < 70 else s * np.float16(sizes[1])
    say(f"attn_kv4 value scales {sizes}")
    check(q, cache, 64, 1, tables, lens, "bf16", "value scales")
    check(q, cache, 64, 1, tables, lens, "bf16", "value scales, sharp", scale=4.0)


def test_sharp_and_flat_scores():
    g = rng(13)
    lens = [700, 64]
    q, cache, tables = setup(g, lens, 16, 8, 2, 64, "f16")
    for scale in (1e-30, 1e-3, 1.0, 30.0, 1e4):
        say(f"attn_kv4 scale {scale}")
        check(q, cache, 16, 2, tables, lens, "f16", "scale", scale=scale)


def test_largest_values():
    """A mean of equal largest values is that value, whatever the weights' rounding."""
    g = rng(14)
    lens = [333]
    q, cache, tables = setup(g, lens, 16, 4, 1, 64, "f16")
    for u in range(333):
        p, at, t = S.place(int(tables[0, u // 16]) * 16 + u % 16, 16, 1, 0, 64)
        tile = cache[p, at:at + 18 * 64]
        tile[512:1024] = 0  # codes 0: -8 d
        scales_at(cache, 16, 1, 64, int(tables[0, u // 16]) * 16 + u % 16, 0, 1)[:] = 8188.0
    say("attn_kv4 largest values")
    o = run(q, cache, 16, 1, tables, lens)
    assert bool((o.float() <= -65504 * (1 - 2.0 ** -10)).all()) and bool(torch.isfinite(o).all())


def test_repeats_streams_and_graphs():
    g = rng(15)
    lens = [1000, 77, 0]
    page, heads, dim = 32, 2, 128
    q, cache, tables = setup(g, lens, page, 8, heads, dim, "f16", width=64)
    c, t = torch.from_numpy(cache).cuda(), torch.from_numpy(tables).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qd = q.cuda()
    first = qmm.qmm_attn_kv4(qd, c, page, heads, t, n)
    assert torch.equal(first, qmm.qmm_attn_kv4(qd, c, page, heads, t, n))
    say("attn_kv4 on two streams")
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [qmm.qmm_attn_kv4(qd, c, page, heads, t, n, stream=s) for s in sides for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    say("attn_kv4 captured")
    ws = torch.empty(qmm.qmm_attn_kv4_workspace_bytes(3, 8, heads, dim, 64, page), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(qd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.qmm_attn_kv4(qd, c, page, heads, t, n, O=o, workspace=ws)
    for lens2 in ([1000, 77, 0], [1, 0, 5], [999, 64, 0]):
        n.copy_(torch.tensor([min(a, b) for a, b in zip(lens2, (1000, 77, 0))], dtype=torch.int32))
        ws.fill_(255)  # whatever an earlier call left there
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, qmm.qmm_attn_kv4(qd, c, page, heads, t, n)), lens2
