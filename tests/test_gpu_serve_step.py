"""The operators of include/qmm_serve.h as a served model runs them, together
with the MUL_MATs and qmm_norm_rope: a decode step from the tokens of the last
one to the next (q, k and v products, norm and rotation, the append, attention,
the output product, the expert layer, logits, the choice of a token), first
eagerly, then as a captured graph that is replayed while sequences grow over
pages' ends, one of them empty.

Every stage is compared with its 64-bit definition on the stage's own inputs,
so no error is excused by an earlier one.
"""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.attn_oracle as A
import oracle.qmm_oracle as O
import oracle.serve_oracle as S
from attn_util import assert_within, f64, rng, say
from block_quantized_matmul_amd import synth

pytestmark = pytest.mark.gpu

Q4, Q8 = qmm.QMM_TYPE_Q4_0, qmm.QMM_TYPE_Q8_0
B, WIDTH, HQ, HKV, DIM, FF, EXPERTS, USED, VOCAB = 5, 256, 8, 2, 64, 192, 6, 2, 700
PAGE, PAGES, TABLE = 16, 24, 100  # (a table of 1600 tokens, so that rows are split)
FREQS = [10000.0 ** (-i / 32) for i in range(32)]


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def floats(a):
    return torch.tensor(np.asarray(a), dtype=torch.float32).cuda()


class Model:
    def __init__(self):
        r = rng(70)
        self.host, self.w = {}, {}
        for name, rows, k in (("q", HQ * DIM, WIDTH), ("k", HKV * DIM, WIDTH), ("v", HKV * DIM, WIDTH),
                              ("o", WIDTH, HQ * DIM), ("logits", VOCAB, WIDTH)):
            self.host[name] = synth.make_weights(Q4, rows, k, synth.dense_row_bytes(Q4, k), r)
            self.w[name] = torch.from_numpy(self.host[name]).cuda()
        self.values, self.stack = {}, {}
        for name, t, rows, k in (("gate", Q4, FF, WIDTH), ("up", Q4, FF, WIDTH), ("down", Q8, WIDTH, FF)):
            nb1 = synth.dense_row_bytes(t, k)
            nb1 += nb1 % 4
            w = synth.make_weights(t, EXPERTS * rows, k, nb1, r)
            self.values[name] = O.dequantize(w, t, EXPERTS * rows, k, nb1).astype(np.float64).reshape(EXPERTS, rows, k)
            self.stack[name] = torch.from_numpy(w).view(EXPERTS, rows, nb1).cuda()
        self.router = floats(r.standard_normal((EXPERTS, WIDTH)) / 16)
        self.nq, self.nk = (floats(1 + 0.1 * r.standard_normal(DIM)) for _ in range(2))
        self.embed = floats(r.standard_normal((VOCAB, WIDTH)))
        # sequences of 15, 0 (an idle row), 30, 31 and 1 tokens so far; their pages in any order
        self.lengths = ints([15, 0, 30, 31, 1])
        self.live = ints([1, 0, 1, 1, 1])
        order = r.permutation(PAGES)[:4 * 5].reshape(4, 5)
        tables = np.full((B, TABLE), -1, np.int32)
        for i, row in enumerate((0, 2, 3, 4)):
            tables[row, :5] = order[i]
        self.tables = ints(tables)
        self.cache = torch.zeros(PAGES, qmm.qmm_kv4_page_bytes(PAGE, HKV, DIM), dtype=torch.uint8, device="cuda")
        self.tokens = ints([3, 9, 27, 81, 243])
        self.u = floats([0.1, 0.9, 0.5, 0.0, 0.7])
        self.settings = dict(temperature=floats([0.8, 1.0, 0.0, 1.3, 0.5]), top_k=ints([0, 5, 9, 40, 100]),
                             top_p=floats([0.9, 1.0, 1.0, 0.95, 0.7]), min_p=floats([0.0, 0.0, 0.0, 0.05, 0.0]))

    def fill(self):
        """Keys and values of the tokens so far, appended as a prompt's would be."""
        r = rng(71)
        n = [int(x) for x in self.lengths.cpu()]
        rows = np.repeat(np.arange(B), n)
        pos = np.concatenate([np.arange(x) for x in n])
        slots = self.tables.cpu().numpy()[rows, pos // PAGE] * PAGE + pos % PAGE
        k, v = (torch.from_numpy(r.standard_normal((len(rows), HKV, DIM))).half().cuda() for _ in range(2))
        qmm.qmm_kv4_append(k, v, self.cache, PAGE, ints(slots), positions=ints(pos), freqs=FREQS, norm=True, weight=self.nk)

    def step(self):
        """One step. What it computes on the way is kept to be looked at."""
        s = {"x": self.embed[self.tokens.long()]}
        for name in "qkv":
            s[name] = qmm.qmm_matmul(self.w[name], Q4, WIDTH, s["x"])
        at = self.lengths
        s["queries"] = torch.zeros(B, HQ, DIM, dtype=torch.float16, device="cuda")
        qmm.qmm_norm_rope([qmm.qmm_head_part(s["q"].view(B, HQ, DIM), s["queries"], norm=True, weight=self.nq, rotate=True)],
                          positions=at, freqs=FREQS)
        page = torch.gather(self.tables, 1, (at // PAGE).long().view(B, 1)).view(B)
        s["slots"] = torch.where(self.live > 0, page * PAGE + at % PAGE, -1).to(torch.int32)
        s["before"] = self.cache.clone()
        s["positions"] = at.clone()
        qmm.qmm_kv4_append(s["k"].view(B, HKV, DIM), s["v"].view(B, HKV, DIM), self.cache, PAGE, s["slots"],
                           positions=s["positions"], freqs=FREQS, norm=True, weight=self.nk)
        s["after"] = self.cache.clone()
        self.lengths += self.live
        s["lengths"] = self.lengths.clone()
        s["o"] = qmm.qmm_attn_kv4(s["queries"], self.cache, PAGE, HKV, self.tables, s["lengths"])
        s["attended"] = qmm.qmm_matmul_x16(self.w["o"], Q4, HQ * DIM, s["o"].view(B, HQ * DIM))
        s["ids"] = torch.zeros(B, USED, dtype=torch.int32, device="cuda")
        s["weights"] = torch.zeros(B, USED, device="cuda")
        s["y"] = qmm.qmm_moe(s["attended"], self.router, self.stack["gate"], self.stack["up"], Q4, self.stack["down"], Q8,
                             USED, ids=s["ids"], weights=s["weights"])
        s["logits"] = qmm.qmm_matmul(self.w["logits"], Q4, WIDTH, s["y"])
        s["probs"] = torch.zeros(B, device="cuda")
        qmm.qmm_sample(s["logits"], self.u, probs=s["probs"], tokens=self.tokens, **self.settings)
        s["tokens"] = self.tokens.clone()
        return s

    def check_matmul(self, name, x, y):
        w = self.host[name]
        ref, bound = O.matmul(w, Q4, w.shape[0], x.shape[1], w.shape[1], x.float().cpu().numpy())
        assert O.within_tolerance(y.cpu().numpy(), ref, bound).all(), name

    def check(self, s):
        for name in "qkv":
            self.check_matmul(name, s["x"], s[name])
        pos = s["positions"].cpu().numpy()
        want, err = A.norm_rope(f64(s["q"]).reshape(B, HQ, DIM), f64(self.nq), True, 1e-6, pos, FREQS, "halves", "f16")
        assert_within(s["queries"], want, err, "queries")
        want = S.append(f64(s["k"]).reshape(B, HKV, DIM), f64(s["v"]).reshape(B, HKV, DIM), s["before"].cpu().numpy(), PAGE,
                        s["slots"].cpu().numpy(), positions=pos, freqs=FREQS, norm=True, weight=f64(self.nk))
        assert np.array_equal(s["after"].cpu().numpy(), want)
        want, err = S.attn_kv4(f64(s["queries"]), want, PAGE, HKV, self.tables.cpu().numpy(), s["lengths"].cpu().numpy(),
                               DIM ** -0.5, "f16")
        assert_within(s["o"], want, err, "attention")
        assert (s["o"][1] == 0).all()  # the idle row
        self.check_matmul("o", s["o"].view(B, HQ * DIM), s["attended"])
        want, err, ids, w = S.moe(f64(s["attended"]), f64(self.router), *(self.values[x] for x in ("gate", "up", "down")), USED)
        assert np.array_equal(s["ids"].cpu().numpy(), ids)
        assert_within(s["weights"], w, 16 * S.E32 * w + 2.0 ** -149, "weights")
        assert_within(s["y"], want, err, "experts")
        self.check_matmul("logits", s["y"], s["logits"])
        z, set_ = f64(s["logits"]), {k: v.cpu().numpy() for k, v in self.settings.items()}
        for i in range(B):
            token, p, near = S.sample(z[i], float(self.u[i]), **{k: float(v[i]) if k != "top_k" else int(v[i])
                                                                 for k, v in set_.items()})
            if near > 2.0 ** -38:
                assert int(s["tokens"][i]) == token and abs(float(s["probs"][i]) - p) <= 2.0 ** -23 * p, i


def test_decode_steps_eager_and_captured():
    say("serve step: eager")
    m = Model()
    m.fill()
    state = [t.clone() for t in (m.cache, m.lengths, m.tokens)]
    eager = []
    for _ in range(4):
        s = m.step()
        torch.cuda.synchronize()
        m.check(s)
        eager.append({k: v.clone() for k, v in s.items()})

    say("serve step: captured")
    for t, old in zip((m.cache, m.lengths, m.tokens), state):
        t.copy_(old)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step()  # what the first call sets up is not part of the graph
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for t, old in zip((m.cache, m.lengths, m.tokens), state):
        t.copy_(old)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = m.step()
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        for name, want in eager[i].items():
            assert torch.equal(s[name], want), (i, name)


def test_two_steps_at_once():
    """Two models' steps on two streams, which share nothing but the weights' pages."""
    say("serve step: two streams")
    m = [Model(), Model()]
    m[1].u.copy_(floats([0.3, 0.2, 0.9, 0.6, 0.05]))
    for x in m:
        x.fill()
    state = [[t.clone() for t in (x.cache, x.lengths, x.tokens)] for x in m]
    want = [[x.step()["tokens"] for _ in range(3)] for x in m]
    for x, old in zip(m, state):
        for t, o in zip((x.cache, x.lengths, x.tokens), old):
            t.copy_(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(m[i].step()["tokens"])
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)
