"""qmm_attn_kv4 where rows of different lengths are divided into ranges of one
length: more rows than lanes, rows that the division leaves whole, rows of
nothing and rows that the tables do not hold, in a workspace of exactly its size."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
from attn_util import rng, say
from test_gpu_attn_kv4 import check, run, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("rows,hq,heads,dim,longest", [(63, 4, 4, 64, 900), (64, 2, 1, 128, 700), (65, 1, 1, 64, 600),
                                                       (200, 2, 2, 64, 400),
                                                       (200, 2, 2, 64, 800), (130, 20, 1, 128, 500)])
def test_many_ragged_rows(rows, hq, heads, dim, longest, wide):
    """In tables as wide as the longest row, and in wide ones, whose rows are divided."""
    g = rng(90, rows, dim)
    say(f"attn_kv4 units {rows} {hq} {heads} {dim} {wide}")
    lens = [int(x) for x in np.where(g.random(rows) < 0.2, g.integers(0, longest, rows), g.integers(0, 40, rows))]
    lens[0], lens[-1], lens[rows // 2] = 0, longest, longest
    q, cache, tables = setup(g, lens, 32, hq, heads, dim, "f16", width=100 if wide else None)
    need = qmm.qmm_attn_kv4_workspace_bytes(rows, hq, heads, dim, tables.shape[1], 32)
    assert (need > 0) == wide
    check(q, cache, 32, heads, tables, lens, "f16", "ragged")


def test_one_long_row_among_short_ones():
    """Most of the ranges are one row's."""
    g = rng(91)
    lens = [1, 20000, 16, 0, 300]
    say("attn_kv4 one long row")
    q, cache, tables = setup(g, lens, 256, 2, 1, 64, "bf16")
    check(q, cache, 256, 1, tables, lens, "bf16", "long row")


def test_rows_that_the_table_does_not_hold():
    """Lengths of rubbish count as no keys in the division; the other rows are right."""
    g = rng(92)
    lens = [500, 333, 41, 700, 0, 64]
    say("attn_kv4 lengths outside")
    q, cache, tables = setup(g, lens, 16, 4, 2, 64, "f16")
    bad = [500, -1, 41, 2 ** 31 - 1, 0, -2 ** 31]
    o = check(q, cache, 16, 2, tables, bad, "f16", "outside")
    assert torch.isnan(o[1]).all() and torch.isnan(o[3]).all() and torch.isnan(o[5]).all() and (o[4] == 0).all()


@pytest.mark.parametrize("rows,hq,heads,dim", [(3, 8, 2, 128), (70, 4, 2, 64), (1, 40, 1, 128)])
def test_workspace_of_its_size(rows, hq, heads, dim):
    g = rng(93, rows)
    say(f"attn_kv4 workspace {rows} {hq} {heads} {dim}")
    lens = [int(x) for x in g.integers(0, 2000, rows)]
    q, cache, tables = setup(g, lens, 64, hq, heads, dim, "f16", width=40)
    need = qmm.qmm_attn_kv4_workspace_bytes(rows, hq, heads, dim, 40, 64)
    assert 0 < need <= qmm.qmm_attn_kv4_workspace_max_bytes(dim)
    buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    got = run(q, cache, 64, heads, tables, lens, workspace=buf[:need])
    assert torch.equal(got, run(q, cache, 64, heads, tables, lens))
    assert (buf[need:] == 0xA5).all()
    with pytest.raises(qmm.QmmError):
        run(q, cache, 64, heads, tables, lens, workspace=buf[:need - 16])


def test_binding_refusals():
    """What a call may not be given, with tensors of the GPU; nothing is enqueued."""
    say("serve binding refusals")
    d = "cuda"
    cache = torch.zeros(4, qmm.qmm_kv4_page_bytes(16, 2, 64), dtype=torch.uint8, device=d)
    k, i = torch.zeros(3, 2, 64, device=d), lambda *s: torch.zeros(*s, dtype=torch.int32, device=d)
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device=d)
    w = torch.zeros(4, 32, 20, dtype=torch.uint8, device=d)
    x, r = torch.zeros(2, 32, device=d), torch.zeros(4, 32, device=d)
    z, u = torch.zeros(3, 50, device=d), torch.zeros(3, device=d)
    Q4 = qmm.QMM_TYPE_Q4_0
    append = lambda **kw: qmm.qmm_kv4_append(**{**dict(K=k, V=k, cache=cache, page_tokens=16, slots=i(3)), **kw})
    attn = lambda **kw: qmm.qmm_attn_kv4(**{**dict(Q=q, cache=cache, page_tokens=16, n_kv_heads=2, tables=i(3, 2),
                                                   lengths=i(3)), **kw})
    moe = lambda **kw: qmm.qmm_moe(**{**dict(X=x, router=r, gate=w, up=w, type_in=Q4, down=w, type_out=Q4, n_used=2), **kw})
    sample = lambda **kw: qmm.qmm_sample(**{**dict(logits=z, u=u), **kw})
    append(), attn(), moe(), sample()
    for call, bad in ((append, [dict(K=k[0]), dict(V=k[:2]), dict(V=k.half()), dict(K=k.int()), dict(cache=cache[:, :-4]),
                                dict(cache=cache.int()), dict(page_tokens=32), dict(page_tokens=20), dict(slots=i(2)),
                                dict(slots=i(3).long()), dict(positions=i(3)), dict(freqs=[1.0]),
                                dict(positions=i(4), freqs=[1.0]), dict(positions=i(3), freqs=[100.0]),
                                dict(weight=u), dict(norm=True, weight=u), dict(pairs="quarters"), dict(eps=-1.0)]),
                      (attn, [dict(Q=q.float()), dict(Q=q[..., ::2]), dict(Q=q[:, :3]), dict(tables=i(2, 2)),
                              dict(tables=i(3, 2).long()), dict(tables=i(2, 3).t()), dict(lengths=i(4)), dict(scale=0.0),
                              dict(O=q.bfloat16()), dict(O=q[:2]), dict(workspace=u), dict(n_kv_heads=3)]),
                      (moe, [dict(X=x.double()), dict(X=x[:, ::2]), dict(X=torch.zeros(17, 32, device=d)), dict(router=r[:, :16]),
                             dict(router=r.half()), dict(gate=w[:3]), dict(up=w[:, :16]), dict(down=w[:, :, :16]),
                             dict(n_used=5), dict(n_used=0), dict(type_in=77), dict(Y=x.half()), dict(ids=i(2, 3)),
                             dict(weights=x), dict(workspace=cache[:1, :64])]),
                      (sample, [dict(logits=z.int()), dict(logits=z.t()), dict(logits=u), dict(u=u[:2]), dict(u=u.double()),
                                dict(top_k=u), dict(top_p=i(3)), dict(tokens=i(3).long()), dict(tokens=i(2)),
                                dict(probs=u.half()), dict(temperature=u[:1]), dict(workspace=cache[:1, :64])])):
        for kw in bad:
            with pytest.raises((TypeError, ValueError, qmm.QmmError)):
                call(**kw)
                pytest.fail(f"accepted {list(kw)}")
    torch.cuda.synchronize()
