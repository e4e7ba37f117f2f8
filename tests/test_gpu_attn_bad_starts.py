"""qmm_attn_prompt on starts that are not in order: a sequence whose two ends are
in order and which shares no token with another is computed, however many tiles
the sequences that do share tokens have between them."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.attn_oracle as O
from attn_util import f64, rng, rounded, say

pytestmark = pytest.mark.gpu

KEPT = 7.0


def _sequences(starts, n):
    return [(b, e) for b, e in zip(starts[:-1], starts[1:]) if 0 <= b <= e <= n]


def _alone(starts, n):
    """Which tokens lie in one sequence that shares none of its tokens, and which in none."""
    seqs = [s for s in _sequences(starts, n) if s[1] > s[0]]
    alone, held = np.zeros(n, bool), np.zeros(n, bool)
    for i, (b, e) in enumerate(seqs):
        held[b:e] = True
        if all(e <= b2 or e2 <= b for j, (b2, e2) in enumerate(seqs) if j != i):
            alone[b:e] = True
    return alone, ~held


def _check(starts, n, hq, hkv, dim, rows=None):
    r = rng(30, n, hq, len(starts))
    q, k, v = (rounded(r.standard_normal((n, h, dim)), "f16") for h in (hq, hkv, hkv))
    say(f"prompt {n} tokens, heads {hq}/{hkv} of {dim}, {len(starts) - 1} pairs of starts {starts[:9]}")
    dev = torch.tensor(starts, dtype=torch.int32).cuda()
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    alone, outside = _alone(starts, n)
    seq_of = {t: b for b, e in _sequences(starts, n) for t in range(b, e)}
    for _ in range(2):
        o = torch.full(q.shape, KEPT, dtype=q.dtype, device="cuda")
        qmm.qmm_attn_prompt(qd, kd, vd, dev, O=o)
        torch.cuda.synchronize()
        got = f64(o)
        assert (got[outside] == KEPT).all()
        at = np.flatnonzero(alone)
        assert at.size
        for t in at if rows is None else at[::max(1, at.size // rows)]:
            for h in range(hq):
                g = h * hkv // hq
                want, err = O.attend(f64(q[t, h]), f64(k[seq_of[t]:t + 1, g]), f64(v[seq_of[t]:t + 1, g]), dim ** -0.5, "f16")
                assert (np.abs(got[t, h] - want) <= err).all(), (t, h)


@pytest.mark.parametrize("starts,n,hq,hkv", [
    ([0, 100, 50, 100, 200], 200, 8, 1),                       # 18 tiles where disjoint sequences could have 16
    ([0, 1000, 0, 1000, 0, 1000, 1024], 1024, 4, 1),           # 97 and 38
    ([0, 1280, 0, 1280, 1290], 1290, 1, 1),
    ([1000, 1024, 0, 1000, 0, 1000, 0, 1000], 1024, 4, 2),     # the one alone comes first
    ([0, 300, -5, 700, 0, 300, 10 ** 9, 300, 0, 300, 700], 700, 2, 2),
])
def test_sequences_beside_overlapping_ones(starts, n, hq, hkv):
    _check(starts, n, hq, hkv, 64, rows=25)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_many_sequences_beside_overlapping_ones(where, dim):
    """More sequences than one step of the search takes, the overlapping ones among the first, middle or last of them."""
    n, m = 3000, 200
    good = [int(x) for x in np.linspace(1000, n, m)]
    many = [0, 1000] * 30
    starts = {"first": many + good, "middle": good[:100] + many + good[100:], "last": good + many}[where]
    _check(starts, n, 4, 1, dim, rows=40)


def test_tokens_each_their_own_sequence():
    """As many tiles as the bound for sequences in order allows."""
    n = 300
    _check(list(range(n + 1)), n, 2, 1, 64)
    _check([0] * 5 + list(range(n + 1)) + [n] * 70, n, 2, 1, 64, rows=60)
