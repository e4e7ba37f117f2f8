"""qmm_attn_prompt and qmm_attn_shared with finite scores of large magnitude.

Scaled scores of 2^20 and more (in base-2 units) leave fp32 no or few bits for
the differences that a softmax is made of, so whatever is subtracted from them
has to be the same number for every key of a row. Scores here are sums of
products that fp32 holds exactly (or equal for all keys that matter), so the
definition in 64 bits needs no allowance for them: what remains are the
rounding of a weight and of the output (a half step u of the type each), the
exponential and its argument (2^-20 of the largest weight in all: an argument -x
is off by 2 steps of 2^-24 of itself, which moves the weight 2^-x by less than
2^-23 of the largest, and the exponential by 2^-22 of itself, as do the few
rescalings), and sums in fp32.
"""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.attn_oracle as O
from attn_util import assert_within, rng, rounded, say

pytestmark = pytest.mark.gpu


def _attend(s, v, kind):
    """softmax(s) v from exact scores, and the bound above."""
    w = np.exp(s - s.max())
    w = w / w.sum()
    o, mag, u = w @ v, w @ np.abs(v), O.HALF_STEP[kind]
    # weights below the type's normal range are off by half a subnormal of it, relative to the largest weight
    err = (u + 2.0 ** -20 + (3 * len(s) + 64) * O.E32) * mag + O.SUBNORMAL[kind] * np.abs(v).sum(0)
    return o, err + u * (np.abs(o) + err) + O.SUBNORMAL[kind]


class Keys:
    """Keys and values of one KV head with their exact scores against one query."""

    def __init__(self, q, k, v, scores, scale):
        self.q, self.k, self.v, self.scores, self.scale = q, k, v, scores, scale


def ties(kind, dim, mag, signs, seed, scale=None):
    """Every element of the query and the keys is `mag`, with each key's sign: scores of +-S only."""
    scale = dim ** -0.5 if scale is None else scale
    n = len(signs)
    signs = np.asarray(signs, np.float64)
    v = rounded(rng(20, seed, n).standard_normal((n, dim)), kind)
    return Keys(rounded(np.full(dim, mag), kind), rounded(mag * signs[:, None] * np.ones((n, dim)), kind), v,
                signs * (dim * mag * mag * scale), scale)


def steps(kind, dim, base, n, scale, seed):
    """Scores base^2 + j with j = 0 .. 3: integers that fp32 holds, whose differences decide."""
    r = rng(21, seed, n)
    j = r.integers(0, 4, n)
    q, k = np.zeros(dim), np.zeros((n, dim))
    q[0], q[1], k[:, 0], k[:, 1] = base, 1.0, base, j
    return Keys(rounded(q, kind), rounded(k, kind), rounded(r.standard_normal((n, dim)), kind),
                (float(base) ** 2 + j) * scale, scale)


def cases(kind, dim, n):
    small, large = (8000.0, 60000.0) if kind == "f16" else (27648.0, 2.0 ** 40)
    r = rng(22, n)
    runs = np.where(np.arange(n) // 70 % 2 == 0, -1, 1)
    return {
        "equal": ties(kind, dim, small, np.ones(n), 1),
        "equal, larger": ties(kind, dim, 20000.0 if kind == "f16" else 40960.0, np.ones(n), 2),
        "equal, largest": ties(kind, dim, large, np.ones(n), 3),
        "equal, negative": ties(kind, dim, large, -np.ones(n), 4),
        "both signs": ties(kind, dim, small, r.choice([-1, 1], n), 5),
        "runs of both signs": ties(kind, dim, large, runs, 6),
        "last one larger": ties(kind, dim, small, np.where(np.arange(n) == n - 1, 1, -1), 7),
        # on both sides of 2^20 in base-2 units
        "steps from 2^18": steps(kind, dim, 512, n, 1.0, 8),
        "steps from 2^20": steps(kind, dim, 1024, n, 0.5, 9),
        "steps from 2^20, whole": steps(kind, dim, 1024, n, 1.0, 10),
        "steps from 2^22": steps(kind, dim, 2048, n, 8.0, 11),
        "steps from 2^22, scaled": steps(kind, dim, 2048, n, 2.0 ** -9, 12),
    }


NAMES = list(cases("f16", 64, 4))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("name", NAMES)
def test_prompt(kind, dim, name):
    """Rows see one key, a few, and keys of several blocks and tiles; two heads share them."""
    n, hq = 200, 2
    c = cases(kind, dim, n)[name]
    what = f"prompt {kind} dim={dim}, {name}"
    say(what)
    o = qmm.qmm_attn_prompt(c.q.expand(n, hq, dim).contiguous().cuda(), c.k[:, None].cuda(), c.v[:, None].cuda(),
                            torch.tensor([0, n], dtype=torch.int32).cuda(), scale=c.scale)
    torch.cuda.synchronize()
    v = c.v.double().numpy()
    want, err = np.zeros((n, hq, dim)), np.zeros((n, hq, dim))
    for t in range(n):
        want[t], err[t] = _attend(c.scores[:t + 1], v[:t + 1], kind)
    assert_within(o, want, err, what)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("prefix,cap,lengths", [(1, 0, [0]), (90, 70, [0, 1, 33, 70]), (0, 300, [1, 300, 64]),
                                                (1030, 70, [0, 1, 70]), (1100, 1000, [0, 999, 300])])
def test_shared(kind, dim, name, prefix, cap, lengths):
    """Keys in one launch, and in pieces of the prefix and of the caches; two heads share them."""
    hq, b = 2, len(lengths)
    c = cases(kind, dim, prefix + cap)[name]
    what = f"shared {kind} dim={dim} prefix={prefix} cap={cap}, {name}"
    say(what)
    k, v = c.k[:, None].cuda(), c.v[:, None].cuda()
    own = [None] * 3
    if cap:
        own = [x[prefix:].expand(b, cap, 1, dim).contiguous() for x in (k, v)]
        own.append(torch.tensor(lengths, dtype=torch.int32).cuda())
    o = qmm.qmm_attn_shared(c.q.expand(b, hq, dim).contiguous().cuda(), *((k[:prefix], v[:prefix]) if prefix else (None, None)),
                            *own, scale=c.scale)
    torch.cuda.synchronize()
    v = c.v.double().numpy()
    want, err = np.zeros((b, hq, dim)), np.zeros((b, hq, dim))
    for i, n in enumerate(lengths):
        want[i], err[i] = _attend(c.scores[:prefix + n], v[:prefix + n], kind)
    assert_within(o, want, err, what)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("large_first", [True, False])
def test_large_beside_ordinary_scores(kind, dim, large_first):
    """Keys of ordinary scores behind some of large negative ones, and ahead of some of large positive ones."""
    n, hq, at = 300, 4, 100
    r = rng(23, dim)
    q = rounded(np.abs(r.standard_normal((hq, dim))) + 0.1, kind)
    k, v = rounded(r.standard_normal((n, dim)) / 4, kind), rounded(r.standard_normal((n, dim)), kind)
    large = 60000.0 if kind == "f16" else 2.0 ** 100
    if large_first:
        k[:at] = -large
    else:
        k[n - at:] = large
    say(f"{kind} dim={dim}, large scores {'first' if large_first else 'last'}")
    args = (k[:, None].cuda(), v[:, None].cuda())
    prompt = qmm.qmm_attn_prompt(q.expand(n, hq, dim).contiguous().cuda(), *args,
                                 torch.tensor([0, n], dtype=torch.int32).cuda(), scale=1.0)
    direct = qmm.qmm_attn_shared(q[None].contiguous().cuda(), *args, None, None, None, scale=1.0)
    # the same keys four times over: in pieces
    pieces = qmm.qmm_attn_shared(q[None].contiguous().cuda(), *(x.repeat(4, 1, 1) for x in args), None, None, None,
                                 scale=1.0)
    torch.cuda.synchronize()
    q, k, v = q.double().numpy(), k.double().numpy(), v.double().numpy()

    def want(h, t):
        """The row of a query that sees keys 0 .. t."""
        if large_first:
            keys = slice(0, t + 1) if t < at else slice(at, t + 1)
        else:
            keys = slice(0, t + 1) if t < n - at else slice(n - at, t + 1)
        if (t < at) if large_first else (t >= n - at):  # equal scores
            return _attend(np.zeros(len(range(*keys.indices(n)))), v[keys], kind)
        return O.attend(q[h], k[keys], v[keys], 1.0, kind)

    rows = [[want(h, t) for h in range(hq)] for t in range(n)]
    assert_within(prompt, np.array([[o for o, _ in r] for r in rows]), np.array([[e for _, e in r] for r in rows]), "prompt")
    o, e = np.array([r[0] for r in rows[-1]]), np.array([r[1] for r in rows[-1]])
    assert_within(direct[0], o, e, "direct")
    # four times the keys: sums of four times the terms
    assert_within(pieces[0], o, e + 9 * n * O.E32 * np.abs(v).max(0), "pieces")


@pytest.mark.parametrize("power", [20, 60])
def test_large_scale_beside_a_nonfinite_later_value(power):
    """A scale that takes the queries (not the scores) to 2^90, or out of fp32's range, in rows that are computed key by
    key because a later token's value is not finite."""
    n, dim, starts = 100, 64, [0, 100]
    r = rng(24)
    q = rounded(2.0 ** 70 * r.standard_normal((n, 2, dim)), "bf16")
    k = rounded(2.0 ** (-70 - power) * r.standard_normal((n, 1, dim)), "bf16")
    v = rounded(r.standard_normal((n, 1, dim)), "bf16")
    scale = 2.0 ** power / 8
    want, err = O.attn_prompt(q.double().numpy(), k.double().numpy(), v.double().numpy(), starts, scale, "bf16")
    v[n - 1, 0, 3] = float("inf")
    say(f"prompt, scale {scale} beside an infinite later value")
    o = qmm.qmm_attn_prompt(q.cuda(), k.cuda(), v.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), scale=scale)
    torch.cuda.synchronize()
    assert_within(o[:n - 1], want[:n - 1], err[:n - 1], "rows before it")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_large_scores_beside_infinite_and_nonfinite(kind, dim):
    """Keys whose score is -infinity among large ones, and rows computed key by key for a later token's value."""
    n, mag = 150, 8000.0 if kind == "f16" else 2.0 ** 40
    signs = rng(25, dim).choice([-1, 1], n)
    c = ties(kind, dim, mag, signs, 26)
    c.k[5::7] = -float("inf")
    c.scores[5::7] = -np.inf
    v = c.v.clone()
    v[n - 1, 3] = float("nan")
    say(f"{kind} dim={dim}, large and infinite scores")
    args = c.q.expand(n, 2, dim).contiguous().cuda(), c.k[:, None].cuda()
    starts = torch.tensor([0, n], dtype=torch.int32).cuda()
    prompt = qmm.qmm_attn_prompt(*args, c.v[:, None].cuda(), starts)
    by_key = qmm.qmm_attn_prompt(*args, v[:, None].cuda(), starts)
    direct = qmm.qmm_attn_shared(args[0][:1], args[1], c.v[:, None].cuda(), None, None, None)
    pieces = qmm.qmm_attn_shared(args[0][:1], args[1].repeat(8, 1, 1), c.v[:, None].cuda().repeat(8, 1, 1), None, None, None)
    torch.cuda.synchronize()
    v = c.v.double().numpy()
    rows = [_attend(c.scores[:t + 1], v[:t + 1], kind) for t in range(n)]
    want, err = (np.repeat(np.array([r[i] for r in rows])[:, None], 2, 1) for i in (0, 1))
    assert_within(prompt, want, err, "tiles")
    assert_within(by_key[:n - 1], want[:n - 1], err[:n - 1], "key by key")
    assert_within(direct[0], want[-1], err[-1], "direct")
    assert_within(pieces[0], want[-1], err[-1] + 21 * n * O.E32 * np.abs(v).max(0), "pieces")
