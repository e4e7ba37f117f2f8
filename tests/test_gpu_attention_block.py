"""The operators of include/qmm_attn.h as a layer runs them, together with the
MUL_MATs: q, k and v products (with adapters on q), norm and rotation into a
cache, attention, and the output product; first for a batch of prompts, then
for decode steps on a shared prefix, captured into a graph and replayed.

Every stage is compared with its 64-bit definition on the stage's own inputs,
so no error is excused by an earlier one.
"""
import numpy as np
import torch

import pytest

import block_quantized_matmul_amd as qmm
from block_quantized_matmul_amd import synth
import oracle.attn_oracle as A
import oracle.qmm_oracle as O
from attn_util import assert_within, f64, rng, say

pytestmark = pytest.mark.gpu

Q4 = qmm.QMM_TYPE_Q4_0
WIDTH, HQ, HKV, DIM, RANK, ADAPTERS = 256, 8, 2, 64, 8, 3
FREQS = [10000.0 ** (-i / 32) for i in range(32)]


class Layer:
    def __init__(self):
        r = rng(8)
        nb1 = synth.dense_row_bytes(Q4, WIDTH)
        self.host, self.w = {}, {}
        for name, rows, k in (("q", HQ * DIM, WIDTH), ("k", HKV * DIM, WIDTH), ("v", HKV * DIM, WIDTH),
                              ("o", WIDTH, HQ * DIM)):
            self.host[name] = synth.make_weights(Q4, rows, k, synth.dense_row_bytes(Q4, k), r)
            self.w[name] = torch.from_numpy(self.host[name]).cuda()
        assert self.host["q"].shape[1] == nb1
        self.a = torch.from_numpy(r.standard_normal((ADAPTERS, RANK, WIDTH)) / 16).half().cuda()
        self.b = torch.from_numpy(r.standard_normal((ADAPTERS, HQ * DIM, RANK))).half().cuda()
        self.nq = torch.from_numpy((1 + 0.1 * r.standard_normal(DIM)).astype(np.float32)).cuda()
        self.nk = torch.from_numpy((1 + 0.1 * r.standard_normal(DIM)).astype(np.float32)).cuda()

    def products(self, x, ids):
        y = {n: qmm.qmm_matmul(self.w[n], Q4, WIDTH, x) for n in ("q", "k", "v")}
        plain = y["q"].clone()
        qmm.qmm_lora(x, self.a, self.b, ids, base=y["q"], Y=y["q"])
        return plain, y

    def heads(self, y, q, kc, vc, positions, slots):
        n = y["q"].shape[0]
        qmm.qmm_norm_rope([qmm.qmm_head_part(y["q"].view(n, HQ, DIM), q, norm=True, weight=self.nq, rotate=True),
                           qmm.qmm_head_part(y["k"].view(n, HKV, DIM), kc, norm=True, weight=self.nk, rotate=True,
                                             slotted=True),
                           qmm.qmm_head_part(y["v"].view(n, HKV, DIM), vc, slotted=True)],
                          positions=positions, freqs=FREQS, slots=slots)

    def output(self, o):
        return qmm.qmm_matmul_x16(self.w["o"], Q4, HQ * DIM, o.reshape(o.shape[0], HQ * DIM))

    def check_matmul(self, name, x, y, k):
        w = self.host[name]
        ref, s = O.matmul(w, Q4, w.shape[0], k, w.shape[1], x.cpu().numpy())
        assert O.within_tolerance(y.cpu().numpy(), ref, s).all(), name

    def check_front(self, x, ids, plain, y, q, kc, vc, positions, slots, before):
        self.check_matmul("q", x, plain, WIDTH)
        self.check_matmul("k", x, y["k"], WIDTH)
        self.check_matmul("v", x, y["v"], WIDTH)
        want, err = A.lora(f64(x), f64(self.a), f64(self.b), ids.cpu().numpy(), None, f64(plain))
        assert_within(y["q"], want, err, "adapters")
        n, pos, at = x.shape[0], positions.cpu().numpy(), slots.cpu().numpy()
        want, err = A.norm_rope(f64(y["q"]).reshape(n, HQ, DIM), f64(self.nq), True, 1e-6, pos, FREQS, "halves", "f16")
        assert_within(q, want, err, "queries")
        for name, cache, old, p, w in (("k", kc, before[0], pos, f64(self.nk)), ("v", vc, before[1], None, None)):
            want, err = A.norm_rope(f64(y[name]).reshape(n, HKV, DIM), w, w is not None, 1e-6, p, FREQS, "halves", "f16")
            full, ferr = f64(old), np.zeros(old.shape)
            full[at], ferr[at] = want, err
            assert_within(cache, full, ferr, name + " cache")


def _ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def test_prompts_then_decode_on_a_shared_prefix():
    r = rng(9)
    layer = Layer()
    # the prompts of three requests, the first of which (30 tokens) becomes the shared prefix
    lens = [30, 21, 40]
    n = sum(lens)
    x = torch.from_numpy(r.standard_normal((n, WIDTH)).astype(np.float32)).cuda()
    ids = _ints(np.repeat([0, -1, 2], lens))
    positions = _ints(np.concatenate([np.arange(i) for i in lens]))
    kc, vc = (torch.zeros(n, HKV, DIM, dtype=torch.float16, device="cuda") for _ in range(2))
    q = torch.zeros(n, HQ, DIM, dtype=torch.float16, device="cuda")
    say("attention block: prompts")
    before = (kc.clone(), vc.clone())
    plain, y = layer.products(x, ids)
    layer.heads(y, q, kc, vc, positions, _ints(np.arange(n)))
    starts = [0, 30, 51, 91]
    o = qmm.qmm_attn_prompt(q, kc, vc, _ints(starts))
    out = layer.output(o)
    torch.cuda.synchronize()
    layer.check_front(x, ids, plain, y, q, kc, vc, positions, _ints(np.arange(n)), before)
    want, err = A.attn_prompt(f64(q), f64(kc), f64(vc), starts, DIM ** -0.5, "f16")
    assert_within(o, want, err, "prompt attention")
    layer.check_matmul("o", o.reshape(n, -1), out, HQ * DIM)

    # five sequences continue from the prefix, each token into its own cache; steps run as a graph
    b, cap, steps = 5, 8, 4
    pk, pv = kc[:30], vc[:30]
    own_k, own_v = (torch.full((b, cap, HKV, DIM), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    x = torch.zeros((b, WIDTH), device="cuda")
    ids, lengths, slots, positions = _ints([0, 1, -1, 2, 1]), _ints([0] * b), _ints([0] * b), _ints([0] * b)
    q, o = (torch.zeros(b, HQ, DIM, dtype=torch.float16, device="cuda") for _ in range(2))
    out = torch.zeros(b, WIDTH, device="cuda")
    plain = {}

    def step():
        plain["q"], plain["y"] = layer.products(x, ids)
        layer.heads(plain["y"], q, own_k.view(b * cap, HKV, DIM), own_v.view(b * cap, HKV, DIM), positions, slots)
        qmm.qmm_attn_shared(q, pk, pv, own_k, own_v, lengths, O=o)
        qmm.qmm_matmul_x16(layer.w["o"], Q4, HQ * DIM, o.view(b, HQ * DIM), Y=out)

    def set_up(i):
        x.copy_(torch.from_numpy(rng(10, i).standard_normal((b, WIDTH)).astype(np.float32)))
        # sequence 3 sits out step 2: its token is stored nowhere and its cache does not grow
        grows = np.array([1, 1, 1, 0 if i == 2 else 1, 1])
        lens_now = np.array([sum(1 for j in range(i + 1) if not (s == 3 and j == 2)) for s in range(b)])
        lengths.copy_(_ints(lens_now))
        slots.copy_(_ints(np.where(grows == 1, np.arange(b) * cap + lens_now - 1, -1)))
        positions.copy_(_ints(30 + lens_now - 1))

    say("attention block: decode step, eager and captured")
    set_up(0)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    own_k.fill_(float("nan")), own_v.fill_(float("nan"))
    for i in range(steps):
        set_up(i)
        before = own_k.clone(), own_v.clone()
        step()
        torch.cuda.synchronize()
        eager = [t.clone() for t in (q, o, out, own_k, own_v)]
        own_k.copy_(before[0]), own_v.copy_(before[1])
        for t in (q, o, out):
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for e, t, name in zip(eager, (q, o, out, own_k, own_v), ("q", "o", "out", "k", "v")):
            assert torch.equal(torch.nan_to_num(e, nan=99.0), torch.nan_to_num(t, nan=99.0)), (i, name)
        lens_now = lengths.cpu().numpy()
        want, err = A.attn_shared(f64(q), f64(pk), f64(pv), f64(own_k), f64(own_v), lens_now, DIM ** -0.5, "f16")
        assert_within(o, want, err, f"decode attention, step {i}")
        layer.check_matmul("o", o.reshape(b, -1), out, HQ * DIM)
        stored = [int(s) for s in slots.cpu().numpy() if s >= 0]
        new = own_k.view(b * cap, HKV, DIM)[stored]
        assert bool(torch.isfinite(new).all())
        # caches hold what the step put there, and nothing else changed
        keep = torch.ones(b * cap, dtype=torch.bool)
        keep[stored] = False
        keep = keep.cuda()
        for now, old in ((own_k, before[0]), (own_v, before[1])):
            a, c = now.view(b * cap, -1)[keep], old.view(b * cap, -1)[keep]
            assert torch.equal(torch.nan_to_num(a, nan=99.0), torch.nan_to_num(c, nan=99.0))


def test_two_streams_at_once():
    """Two calls of each operator on two streams, with workspaces and outputs of their own, give what they give alone."""
    r = rng(11)
    x = torch.from_numpy(r.standard_normal((600, 512)).astype(np.float32)).cuda()
    a = torch.from_numpy(r.standard_normal((4, 16, 512)) / 20).half().cuda()
    b = torch.from_numpy(r.standard_normal((4, 300, 16))).half().cuda()
    ids = _ints(r.integers(0, 4, 600))
    q = torch.from_numpy(r.standard_normal((40, 8, 64))).half().cuda()
    pk, pv = (torch.from_numpy(r.standard_normal((3000, 2, 64))).half().cuda() for _ in range(2))
    kv = torch.from_numpy(r.standard_normal((2, 3000, 2, 64))).half().cuda()
    qq = torch.from_numpy(r.standard_normal((3000, 8, 64))).half().cuda()
    starts = _ints([0, 1000, 3000])
    say("two streams")

    def work(s):
        return [qmm.qmm_lora(x, a, b, ids, stream=s), qmm.qmm_attn_shared(q, pk, pv, None, None, None, stream=s),
                qmm.qmm_attn_prompt(qq, kv[0], kv[1], starts, stream=s)]

    alone = work(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for _ in range(4):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            results.append(work(s))
    torch.cuda.synchronize()
    for res in results:
        for got, want in zip(res, alone):
            assert torch.equal(got, want)


def test_memory_of_another_stream():
    """What a call on another stream allocates is not memory that pending work of the current stream still writes."""
    r = rng(12)
    x = torch.from_numpy(r.standard_normal((700, 512)).astype(np.float32)).cuda()
    a = torch.from_numpy(r.standard_normal((2, 8, 512)) / 20).half().cuda()
    b = torch.from_numpy(r.standard_normal((2, 1024, 8))).half().cuda()
    ids = _ints(r.integers(0, 2, 700))
    say("another stream's memory")
    want = qmm.qmm_lora(x, a, b, ids)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    dropped = [torch.empty(700, 1024, device="cuda") for _ in range(4)]
    dropped += [torch.empty(qmm.qmm_lora_workspace_bytes(700, 512, 8), dtype=torch.uint8, device="cuda")
                for _ in range(4)]
    torch.cuda._sleep(30_000_000)  # some 15 ms
    for t in dropped:
        t.fill_(7)
    del dropped, t
    got = qmm.qmm_lora(x, a, b, ids, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
