"""qmm_attn_prompt and qmm_attn_shared on fp16 values up to the type's largest: an
output is a weighted mean of values, so it is never beyond the largest of them,
whatever the weights' rounding. An infinite value stays infinite."""
import math

import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.attn_oracle as O
from attn_util import f64, rng, rounded, say

pytestmark = pytest.mark.gpu

LARGEST = 65504.0


def _check(o, q, k, v, what, scale=None):
    """o [hq][dim] of one query over all keys of one KV head."""
    for h in range(o.shape[0]):
        want, err = O.attend(q[h], k, v, scale or o.shape[1] ** -0.5, "f16")
        assert np.isfinite(o[h]).all(), (what, h)
        assert (np.abs(o[h]) <= LARGEST).all() and (np.abs(o[h] - want) <= err).all(), (what, h)


def _inputs(n, hq, dim, seed):
    r = rng(40, n, seed)
    q, k = rounded(r.standard_normal((n, hq, dim)), "f16"), rounded(r.standard_normal((n, 1, dim)), "f16")
    # columns of the largest value, of its negative, of both in turn, and others
    v = np.full((n, 1, dim), LARGEST)
    v[..., 1::4] *= -1
    v[..., 2::4] *= np.where(np.arange(n) % 2, 1, -1)[:, None, None]
    v[..., 3::4] = r.standard_normal((n, 1, dim // 4))
    return q, k, rounded(v, "f16")


@pytest.mark.parametrize("dim", [64, 128])
def test_prompt(dim):
    n, hq = 150, 4
    q, k, v = _inputs(n, hq, dim, dim)
    say(f"prompt largest values dim={dim}")
    o = qmm.qmm_attn_prompt(q.cuda(), k.cuda(), v.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    o = f64(o)
    for t in range(n):
        _check(o[t], f64(q[t]), f64(k[:t + 1, 0]), f64(v[:t + 1, 0]), t)
    v[60, 0, 8] = float("inf")  # its rows by tiles, earlier ones row by row
    o = f64(qmm.qmm_attn_prompt(q.cuda(), k.cuda(), v.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda()))
    assert not np.isfinite(o[60:, :, 8]).any()
    v[60, 0, 8] = 1.0
    for t in range(60):
        _check(o[t], f64(q[t]), f64(k[:t + 1, 0]), f64(v[:t + 1, 0]), t)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("prefix,cap", [(3, 90), (1100, 90), (0, 150)])
def test_shared(dim, prefix, cap):
    b, hq = 5, 4
    q, k, v = _inputs(prefix + cap, hq, dim, prefix)
    lengths = [1 + i * (cap - 1) // (b - 1) for i in range(b)]
    say(f"shared largest values dim={dim} prefix={prefix} cap={cap}")
    kd, vd = k.cuda(), v.cuda()
    own = [x[prefix:].expand(b, cap, 1, dim).contiguous() for x in (kd, vd)]
    o = f64(qmm.qmm_attn_shared(q[:b].cuda(), *((kd[:prefix], vd[:prefix]) if prefix else (None, None)), *own,
                                torch.tensor(lengths, dtype=torch.int32).cuda()))
    for i, n in enumerate(lengths):
        _check(o[i], f64(q[i]), f64(k[:prefix + n, 0]), f64(v[:prefix + n, 0]), i)


# Of sixteen keys one has the weight 1, the others 1/2 + 2^-12 + 2^-15, which fp16 rounds up to 1/2 + 2^-11: their mean
# comes out (2^-11 - 2^-14) 7.5 / 8.5 = 3.8e-4 too large, and 65504 of that is 25. From 65520 on, fp16 has infinity.
SCALE = -math.log(0.5 + 2.0 ** -12 + 2.0 ** -15)


def _rounded_up(n, dim):
    q, k = torch.zeros(1, dim).half(), torch.zeros(n, 1, dim).half()
    q[0, 0], k[:, 0, 0] = 1.0, torch.where(torch.arange(n) % 16 == 0, 0.0, -1.0)
    v = torch.full((n, 1, dim), LARGEST).half()
    v[..., dim // 2:] = -LARGEST
    return q, k, v


@pytest.mark.parametrize("dim", [64, 128])
def test_weights_rounded_up(dim):
    n = 400
    q, k, v = _rounded_up(n, dim)
    say(f"weights rounded up, dim={dim}")
    qd = q.expand(n, 1, dim).contiguous().cuda()
    starts = torch.tensor([0, n - 1], dtype=torch.int32).cuda()
    o = f64(qmm.qmm_attn_prompt(qd, k.cuda(), v.cuda(), starts, scale=SCALE))
    for t in range(n - 1):
        _check(o[t], f64(q), f64(k[:t + 1, 0]), f64(v[:t + 1, 0]), t, SCALE)
    for m in (n, 5 * n):  # in one launch and in pieces
        q, k, v = _rounded_up(m, dim)
        o = f64(qmm.qmm_attn_shared(qd[:3], k.cuda(), v.cuda(), None, None, None, scale=SCALE))
        own = qmm.qmm_attn_shared(qd[:3], None, None, k[None].expand(3, m, 1, dim).cuda(), v[None].expand(3, m, 1, dim).cuda(),
                                  torch.tensor([m, m - 1, m // 2], dtype=torch.int32).cuda(), scale=SCALE)
        for i in range(3):
            _check(o[i], f64(q), f64(k[:, 0]), f64(v[:, 0]), (m, i), SCALE)
            e = [m, m - 1, m // 2][i]
            _check(f64(own)[i], f64(q), f64(k[:e, 0]), f64(v[:e, 0]), ("own", m, i), SCALE)
