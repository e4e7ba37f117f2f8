"""qmm_moe on the GPU against the 64-bit definition: the choice exactly, every
output within the bound that the stated numerics give."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.qmm_oracle as O
import oracle.serve_oracle as S
from attn_util import assert_within, f64, rng, rounded, say
from block_quantized_matmul_amd import synth

pytestmark = pytest.mark.gpu

Q = {"q4_0": qmm.QMM_TYPE_Q4_0, "q4_1": qmm.QMM_TYPE_Q4_1, "q5_0": qmm.QMM_TYPE_Q5_0, "q5_1": qmm.QMM_TYPE_Q5_1,
     "q8_0": qmm.QMM_TYPE_Q8_0, "q4_k": qmm.QMM_TYPE_Q4_K}


def stack(g, qtype, experts, rows, k, pad=0):
    """(bytes [experts][rows][nb1], weights) with nb1 a multiple of 4."""
    nb1 = (synth.dense_row_bytes(qtype, k) + 3) // 4 * 4 + pad
    w = synth.make_weights(qtype, experts * rows, k, nb1, g)
    vals = O.dequantize(w, qtype, experts * rows, k, nb1).astype(np.float64)
    return torch.from_numpy(w).view(experts, rows, nb1), vals.reshape(experts, rows, k)


def layer(g, n, experts, k, ff, tin, tout, kind="f32", pad=0):
    x = rounded(g.standard_normal((n, k)), kind)
    router = rounded(g.standard_normal((experts, k)) / np.sqrt(k), "f32")
    gate, gv = stack(g, Q[tin], experts, ff, k, pad)
    up, uv = stack(g, Q[tin], experts, ff, k, pad)
    down, dv = stack(g, Q[tout], experts, k, ff, pad)
    return x, router, gate, up, down, gv, uv, dv


def run(x, router, gate, up, down, tin, tout, used, **kw):
    ids = torch.full((x.shape[0], used), -9, dtype=torch.int32, device="cuda")
    w = torch.full((x.shape[0], used), -9.0, device="cuda")
    y = qmm.qmm_moe(x.cuda(), router.cuda(), gate.cuda(), up.cuda(), Q[tin], down.cuda(), Q[tout], used, ids=ids, weights=w,
                    **kw)
    torch.cuda.synchronize()
    return y, ids, w


def check(x, router, gate, up, down, gv, uv, dv, tin, tout, used, renormalise=True, what="moe"):
    y, ids, w = run(x, router, gate, up, down, tin, tout, used, renormalise=renormalise)
    want, err, wids, ww = S.moe(f64(x), f64(router), gv, uv, dv, used, renormalise)
    assert np.array_equal(ids.cpu().numpy(), wids), what
    assert_within(w, ww, 16 * S.E32 * ww + 2.0 ** -149, what + " weights")
    assert_within(y, want, err, what)
    return y


@pytest.mark.parametrize("tin", list(Q))
@pytest.mark.parametrize("n", [1, 5, 16])
def test_types(tin, n):
    """Every type for gate and up and for down, one column tile and two."""
    g = rng(40, n, Q[tin])
    tout = list(Q)[(list(Q).index(tin) + n) % 6]
    say(f"moe types {tin} {tout} {n}")
    check(*layer(g, n, 5, 512, 256, tin, tout), tin, tout, 2)


@pytest.mark.parametrize("k,ff", [(256, 256), (32, 32), (288, 352), (64, 1408), (2048, 96), (544, 2080)])
@pytest.mark.parametrize("tin,tout", [("q4_0", "q8_0"), ("q5_0", "q4_0"), ("q5_1", "q4_1"), ("q8_0", "q5_0")])
def test_sizes(k, ff, tin, tout):
    """Row groups and quads that are filled in part, rows of an odd number of blocks."""
    g = rng(41, k, ff)
    say(f"moe sizes {k} {ff} {tin} {tout}")
    check(*layer(g, 3, 4, k, ff, tin, tout), tin, tout, 2)


@pytest.mark.parametrize("n,experts,used", [(1, 1, 1), (2, 3, 3), (8, 8, 1), (9, 8, 2), (16, 2, 1), (4, 70, 6), (3, 512, 32),
                                            (16, 130, 9)])
def test_choices(n, experts, used):
    g = rng(42, n, experts)
    say(f"moe choices {n} {experts} {used}")
    check(*layer(g, n, experts, 64, 64, "q4_0", "q4_0"), "q4_0", "q4_0", used)


def test_not_renormalised_fp16_and_padded_rows():
    g = rng(43)
    say("moe not renormalised, fp16, padded")
    check(*layer(g, 6, 12, 512, 768, "q4_k", "q4_k", kind="f16", pad=16), "q4_k", "q4_k", 3, renormalise=False)
    check(*layer(g, 6, 12, 96, 160, "q4_0", "q5_1", kind="f16", pad=12), "q4_0", "q5_1", 3)


def test_views_of_one_tensor():
    """gate and up as halves of one stack of rows, and as one and the same."""
    g = rng(44)
    x, router, gate, up, down, gv, uv, dv = layer(g, 4, 6, 256, 128, "q4_0", "q4_0")
    both = torch.cat([gate, up], 1).cuda()
    say("moe views")
    y = qmm.qmm_moe(x.cuda(), router.cuda(), both[:, :128], both[:, 128:], Q["q4_0"], down.cuda(), Q["q4_0"], 2)
    assert torch.equal(y, run(x, router, gate, up, down, "q4_0", "q4_0", 2)[0])
    y = qmm.qmm_moe(x.cuda(), router.cuda(), both[:, 128:], both[:, :128], Q["q4_0"], down.cuda(), Q["q4_0"], 2)
    want, err, _, _ = S.moe(f64(x), f64(router), uv, gv, dv, 2)
    assert_within(y, want, err, "up before gate")
    same = gate.cuda()
    y = qmm.qmm_moe(x.cuda(), router.cuda(), same, same, Q["q4_0"], down.cuda(), Q["q4_0"], 2)
    want, err, _, _ = S.moe(f64(x), f64(router), gv, gv, dv, 2)
    assert_within(y, want, err, "gate is up")


def test_ties_take_the_first():
    g = rng(45)
    x, router, gate, up, down, gv, uv, dv = layer(g, 3, 9, 64, 64, "q4_0", "q4_0")
    router[4] = router[1]
    router[7] = router[1]
    router[2] = router[8]
    x[2] = 0  # all logits zero
    say("moe ties")
    check(x, router, gate, up, down, gv, uv, dv, "q4_0", "q4_0", 4)


def test_nonfinite_and_large_tokens():
    """A token's infinity, NaN or value beyond fp16 makes its own row non-finite and leaves the others' bits."""
    g = rng(46)
    x, router, gate, up, down, gv, uv, dv = layer(g, 7, 8, 256, 128, "q4_0", "q8_0")
    clean, _, _ = run(x, router, gate, up, down, "q4_0", "q8_0", 2)
    bad = x.clone()
    bad[1, 17], bad[3, 200], bad[5, 0] = float("nan"), float("inf"), 70000.0
    say("moe non-finite tokens")
    y, ids, _ = run(bad, router, gate, up, down, "q4_0", "q8_0", 2)
    for t in range(7):
        if t in (1, 3, 5):
            assert not bool(torch.isfinite(y[t]).any()), t
        else:
            want, err, _, _ = S.moe(f64(bad[t:t + 1]), f64(router), gv, uv, dv, 2)
            assert_within(y[t:t + 1], want, err, "finite token")
    assert bool((ids >= 0).all()) and bool((ids < 8).all())
    assert torch.equal(clean, run(x, router, gate, up, down, "q4_0", "q8_0", 2)[0])


@pytest.mark.parametrize("size", [1e-6, 1e-3, 300.0])
def test_small_and_large_activations(size):
    """Up to the stated limit: an activation between the products beyond 65504 makes the token's row non-finite."""
    g = rng(47)
    x, router, gate, up, down, gv, uv, dv = layer(g, 2, 4, 256, 256, "q4_0", "q4_0")
    say(f"moe activations of {size}")
    x = x * size
    ids, w = S.choice(f64(x), f64(router), 2)
    h = max(abs(w[t, i] * np.maximum(gv[e] @ f64(x)[t], 0) * (uv[e] @ f64(x)[t])).max() for t in range(2) for i, e in enumerate(ids[t]))
    if h < 65504:
        check(x, router, gate, up, down, gv, uv, dv, "q4_0", "q4_0", 2)
    else:
        assert h > 65600
        y, _, _ = run(x, router, gate, up, down, "q4_0", "q4_0", 2)
        assert not bool(torch.isfinite(y).all())


def test_repeats_streams_workspaces_and_graphs():
    g = rng(48)
    x, router, gate, up, down, gv, uv, dv = layer(g, 3, 8, 512, 608, "q4_0", "q4_0")
    first, _, _ = run(x, router, gate, up, down, "q4_0", "q4_0", 2)
    d = [t.cuda() for t in (x, router, gate, up, down)]
    torch.cuda.synchronize()

    def call(**kw):
        return qmm.qmm_moe(d[0], d[1], d[2], d[3], Q["q4_0"], d[4], Q["q4_0"], 2, **kw)

    say("moe on two streams")
    outs = [call(stream=s) for s in (torch.cuda.Stream(), torch.cuda.Stream()) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    say("moe captured")
    ws = torch.empty(qmm.qmm_moe_workspace_bytes(3, 512, 608, 8, 2), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(Y=y, workspace=ws)
    for step in range(3):
        d[0].copy_(rounded(g.standard_normal((3, 512)), "f32"))
        ws.fill_(255)  # whatever an earlier call left there
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, call()), step


def test_no_tokens():
    g = rng(49)
    x, router, gate, up, down, *_ = layer(g, 1, 2, 64, 64, "q4_0", "q4_0")
    y, _, _ = run(x[:0], router, gate, up, down, "q4_0", "q4_0", 1)
    assert y.shape == (0, 64)
