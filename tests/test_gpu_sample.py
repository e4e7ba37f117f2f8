"""qmm_sample on the GPU against the definition in 80 bits: the tokens exactly,
but where a decision lies within 2^-38 of its border."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.serve_oracle as S
from attn_util import f64, rng, rounded, say

pytestmark = pytest.mark.gpu
NEAR = 2.0 ** -38  # sums of 2^17 weights, each off by 2^-45 of the largest and 2^-46 of itself


def run(z, u, **kw):
    n = z.shape[0]
    kw = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32).cuda() for k, v in kw.items()}
    probs = torch.full((n,), -9.0, device="cuda")
    t = qmm.qmm_sample(z if z.is_cuda else z.cuda(), torch.tensor(u, dtype=torch.float32).cuda(), probs=probs, **kw)
    torch.cuda.synchronize()
    return t.cpu().numpy(), probs.cpu().numpy()


def check(z, u, what, **kw):
    tokens, probs = run(z, u, **kw)
    v = f64(z)
    far = 0
    for i in range(len(u)):
        row = {k: (int(x[i]) if k == "top_k" else float(np.float32(x[i]))) for k, x in kw.items()}
        want, p, near = S.sample(v[i], float(np.float32(u[i])), **row)
        if near <= NEAR:
            continue
        far += 1
        assert tokens[i] == want, (what, i, int(tokens[i]), want, row, u[i], near)
        if want >= 0:
            assert abs(float(probs[i]) - p) <= 2.0 ** -23 * p, (what, i, float(probs[i]), p)
        else:
            assert np.isnan(probs[i])
    assert far >= len(u) * 3 // 4, f"{what}: too many rows at a border"
    return tokens


def settings(g, n):
    return dict(temperature=np.where(g.random(n) < 0.1, 0.0, 0.3 + 1.5 * g.random(n)),
                top_k=np.where(g.random(n) < 0.4, 0, g.integers(1, 300, n)),
                top_p=np.where(g.random(n) < 0.3, 1.0, 0.5 + 0.5 * g.random(n)),
                min_p=np.where(g.random(n) < 0.5, 0.0, 0.2 * g.random(n)))


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 63, 1000, 2048, 2049, 32000, 130001])
def test_vocabularies(kind, vocab):
    g = rng(60, vocab)
    n = 12
    say(f"sample {kind} {vocab}")
    z = rounded((0.3 + 3 * g.random((n, 1))) * g.standard_normal((n, vocab)), kind)
    check(z, g.random(n), "vocabulary", **settings(g, n))


@pytest.mark.parametrize("only", ["temperature", "top_k", "top_p", "min_p", None])
def test_each_setting_alone(only):
    g = rng(61)
    n = 40
    z = rounded(2 * g.standard_normal((n, 3000)), "f32")
    kw = settings(g, n)
    say(f"sample {only} alone")
    check(z, g.random(n), only, **({only: kw[only]} if only else {}))


def test_many_rows_at_strides():
    g = rng(62)
    n, vocab = 700, 301
    wide = rounded(3 * g.standard_normal((n, 400)), "f32")
    say("sample many rows")
    dev = wide.cuda()[:, 17:17 + vocab]
    kw = settings(g, n)
    u = g.random(n)
    tokens = check(wide[:, 17:17 + vocab].contiguous(), u, "rows", **kw)
    assert np.array_equal(run(dev, u, **kw)[0], tokens)
    say("sample one row for all random numbers")
    one = dev[:1].expand(n, vocab)
    t, _ = run(one, u)
    v = f64(wide[0, 17:17 + vocab])
    assert all(t[i] == S.sample(v, float(np.float32(u[i])))[0] for i in range(0, n, 7))


def test_ties():
    """Equal logits: the order is the index's, limits may cut through them."""
    g = rng(63)
    n, vocab = 60, 5000
    z = torch.zeros(n, vocab)
    z[20:40] = torch.from_numpy(g.integers(-3, 3, (20, vocab)).astype(np.float32))
    z[40:] = torch.from_numpy(np.round(g.standard_normal((20, vocab)) * 4).astype(np.float32) / 8)
    z[3, 5::3] = -0.0
    kw = dict(temperature=np.full(n, 1.0), top_k=g.choice([0, 1, 7, 4999, 5000, 6000], n), top_p=g.choice([1.0, 0.37, 0.9], n),
              min_p=g.choice([0.0, 0.3, 1.0], n))
    say("sample ties")
    check(z, g.random(n), "ties", **kw)


def test_edges_of_u_and_settings():
    g = rng(64)
    vocab = 2500
    z = rounded(2 * g.standard_normal((1, vocab)), "f32")
    us = [0.0, -1.0, float("nan"), 1.0, 2.0, float("inf"), 0.99999994, 1e-45, 0.5]
    say("sample edges of u")
    check(z.expand(len(us), vocab).contiguous(), us, "u")
    n = 12
    zz = z.expand(n, vocab).contiguous()
    u = [0.0, 0.3, 0.999] * 4
    nan, inf = float("nan"), float("inf")
    say("sample edges of settings")
    check(zz, u, "top_p", top_p=[0.0, -1.0, 1e-30, 0.99999994, 1.0, 1.5, nan, inf, 0.5, 0.1, 0.9, 0.01])
    check(zz, u, "min_p", min_p=[0.0, -1.0, 1e-30, 1.0, 2.0, nan, inf, 0.5, 1e-45, 0.1, 0.9, 0.01])
    check(zz, u, "top_k", top_k=[-1, -2 ** 31, 0, 1, 2, vocab, vocab + 1, 2 ** 31 - 1, vocab - 1, 3, 4, 5])
    check(zz, u, "temperature", temperature=[nan, -1.0, 0.0, 1e-45, 1e-30, 1e-3, 100.0, 1e30, 3e38, 0.1, 1.0, 10.0])
    t, p = run(zz[:4], [0.0, 0.25, 0.5, 0.9999], temperature=[inf] * 4)
    order = np.argsort(-f64(z[0]), kind="stable")
    assert list(t) == [order[0], order[625], order[1250], order[int(np.float32(0.9999) * vocab)]]
    assert np.allclose(p, 1 / vocab, rtol=2.0 ** -23)


def test_infinities_and_nans():
    g = rng(65)
    vocab = 1500
    n = 10
    z = rounded(2 * g.standard_normal((n, vocab)), "f32")
    inf, nan = float("inf"), float("nan")
    z[0] = -inf
    z[1] = nan
    z[2] = -inf
    z[2, 777] = -3e38
    z[3, :700] = nan
    z[4, ::2] = -inf
    z[5, 3] = z[5, 900] = inf
    z[6, 3], z[6, 8] = 3.4e38, -3.4e38
    z[7] = -inf
    z[7, 1490:] = 5.0
    z[8, :] = 1e-42
    z[9, 5] = 3e38
    say("sample infinities and NaNs")
    for u in (0.0, 0.6, 0.99):
        t = check(z, [u] * n, "infinities")
        assert t[0] == t[1] == -1 and t[2] == 777 and t[5] in (3, 900)
    check(z, g.random(n), "infinities with limits", top_k=[5] * n, top_p=[0.8] * n, min_p=[0.01] * n)
    check(z, g.random(n), "infinities, hot", temperature=[1e30] * n, top_p=[0.7] * n)


def test_tiny_and_close_logits():
    """Logits that differ in their last bits only, and in the far small range."""
    g = rng(66)
    n, vocab = 20, 4000
    base = np.float32(13.7).view(np.uint32) + g.integers(0, 3000, (n, vocab))
    z = torch.from_numpy(base.astype(np.uint32).view(np.float32).copy())
    z[10:] = torch.from_numpy((g.integers(-2000, 2000, (10, vocab)) * 1e-42).astype(np.float32))
    kw = settings(g, n)
    kw["min_p"] = np.zeros(n)  # (all weights are within 2^-10 of 1)
    say("sample close logits")
    check(z, g.random(n), "close", **kw)


def test_frequencies():
    """A grid of random numbers meets every token as often as its probability says."""
    g = rng(67)
    vocab, n = 16, 4096
    z = rounded(g.standard_normal((1, vocab)), "f32")
    u = (np.arange(n) + 0.5) / n
    say("sample frequencies")
    t, _ = run(z.expand(n, vocab), u)
    p = np.exp(f64(z[0]))
    assert np.abs(np.bincount(t, minlength=vocab) - n * p / p.sum()).max() <= 1


def test_repeats_streams_and_graphs():
    g = rng(68)
    n, vocab = 5, 9001
    z = rounded(2 * g.standard_normal((n, vocab)), "f32").cuda()
    u = torch.rand(n, device="cuda")
    kw = dict(temperature=torch.full((n,), 0.8, device="cuda"), top_k=torch.full((n,), 50, dtype=torch.int32, device="cuda"),
              top_p=torch.full((n,), 0.95, device="cuda"), min_p=torch.full((n,), 0.02, device="cuda"))
    first = qmm.qmm_sample(z, u, **kw)
    torch.cuda.synchronize()
    say("sample on two streams")
    outs = [qmm.qmm_sample(z, u, stream=s, **kw) for s in (torch.cuda.Stream(), torch.cuda.Stream()) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    say("sample captured")
    tokens = torch.empty(n, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.qmm_sample(z, u, tokens=tokens, **kw)
    for step in range(4):
        u.copy_(torch.rand(n))
        z.copy_(torch.randn(n, vocab))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(tokens, qmm.qmm_sample(z, u, **kw)), step
    empty = qmm.qmm_sample(z[:0], u[:0])
    assert empty.shape == (0,)
