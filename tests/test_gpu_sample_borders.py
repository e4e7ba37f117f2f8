"""qmm_sample on rows placed next to a border: two tokens whose shares, share of
top_p or ratio to min_p differ from the limit by little more than what the sums'
rounding may move it, so that weights less exact than stated choose another token."""
import numpy as np
import pytest
import torch

import oracle.serve_oracle as S
from attn_util import rng, say
from test_gpu_sample import NEAR, check, run

pytestmark = pytest.mark.gpu
FAR = 8 * NEAR


def beside(g, limit, inverse, value, n=2_000_000, least=100):
    """(differences, limits), both fp32: those of n random limits between which and value(difference) lie NEAR to FAR."""
    limits = limit(g, n).astype(np.float32)
    d = inverse(limits.astype(np.float64)).astype(np.float32)
    off = np.abs(value(d.astype(np.longdouble)) - limits.astype(np.longdouble))
    take = (off > 1.01 * NEAR) & (off < FAR) & (d > 0)
    assert take.sum() >= least
    closest = np.argsort(off[take], kind="stable")[:4000]
    return d[take][closest], limits[take][closest]


SHARE = (lambda p: np.log(p / (1 - p)), lambda d: 1 / (1 + np.exp(-d)))


def rows(d):
    return torch.from_numpy(np.stack([np.zeros_like(d), -d], -1))


@pytest.mark.parametrize("high", [0.7, 0.999])
def test_random_numbers_beside_a_share(high):
    g = rng(110, int(1000 * high))
    d, u = beside(g, lambda g, n: 0.5 + (high - 0.5) * g.random(n), *SHARE)
    say(f"sample {len(d)} rows beside a share")
    check(rows(d), u, "u beside a share")


def test_top_p_beside_a_share():
    g = rng(111)
    d, p = beside(g, lambda g, n: 0.5 + 0.4 * g.random(n), *SHARE)
    say(f"sample {len(d)} rows beside top_p")
    tokens = check(rows(d), np.full(len(d), 0.9999), "top_p beside a share", top_p=p)
    assert 0 < tokens.sum() < len(d)


def test_min_p_beside_a_weight():
    g = rng(112)
    d, p = beside(g, lambda g, n: 0.05 + 0.9 * g.random(n), lambda p: -np.log(p), lambda d: np.exp(-d))
    say(f"sample {len(d)} rows beside min_p")
    tokens = check(rows(d), np.full(len(d), 0.9999), "min_p beside a weight", min_p=p)
    assert 0 < tokens.sum() < len(d)


@pytest.mark.parametrize("z,u,token", [(-0.5360652804374695, 0.6308966279029846, 1), (-0.7634844779968262, 0.6821097731590271, 1),
                                       (-0.395387202501297, 0.5975788831710815, None)])
def test_two_tokens(z, u, token):
    z, u = float(np.float32(z)), float(np.float32(u))
    want, _, near = S.sample(np.array([0.0, z]), u)
    assert near > NEAR and (token is None or want == token)
    say(f"sample two tokens {z} {u}")
    assert run(torch.tensor([[0.0, z]]), [u])[0][0] == want


def test_many_tokens_beside_a_share():
    """The same two tokens in front of 3000 others of far smaller weight, whose sum is part of the border."""
    g = rng(113)
    n, vocab = 60, 3000
    z, u = np.zeros((n, vocab), np.float32), np.zeros(n, np.float32)
    z[:, 2:] = -12 - 3 * g.random((n, vocab - 2))
    rest = np.exp(z[:, 2:].astype(np.longdouble)).sum(-1)
    for i in range(n):
        d, limits = beside(g, lambda g, n: 0.5 + 0.3 * g.random(n), lambda p: -np.log(1 / p - 1 - float(rest[i])),
                           lambda d: 1 / (1 + np.exp(-d) + rest[i]), 50000, 1)
        z[i, 1], u[i] = -d[0], limits[0]
    say("sample many tokens beside a share")
    check(torch.from_numpy(z), u, "beside a share among many")
