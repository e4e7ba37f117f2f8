"""Buffers of the attention operators: one workspace, sized for the largest batch,
through calls of falling sizes, and an output in place of the queries."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
from attn_util import rng, say

pytestmark = pytest.mark.gpu


def _normal(r, *shape):
    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).cuda()


def test_shared_prefix():
    r = rng(50)
    q, pk, pv = _normal(r, 48, 4, 64).half(), _normal(r, 6000, 2, 64).half(), _normal(r, 6000, 2, 64).half()
    k, v = _normal(r, 48, 600, 2, 64).half(), _normal(r, 48, 600, 2, 64).half()
    lengths = torch.tensor([i * 12 for i in range(48)], dtype=torch.int32).cuda()
    ws = torch.full((qmm.qmm_attn_shared_workspace_max_bytes(48, 4, 64),), 0xFF, dtype=torch.uint8, device="cuda")
    for n, prefix in ((48, 6000), (33, 5000), (32, 6000), (31, 4097), (7, 6000), (1, 1025), (1, 3)):
        say(f"shared, kept workspace, {n} sequences on {prefix}")
        args = (q[:n], pk[:prefix], pv[:prefix], k[:n], v[:n], lengths[:n])
        got, want = qmm.qmm_attn_shared(*args, workspace=ws), qmm.qmm_attn_shared(*args)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_lora():
    r = rng(51)
    x, a, b = _normal(r, 1100, 1056), (_normal(r, 3, 40, 1056) / 32).half(), _normal(r, 3, 70, 40).half()
    ids = torch.from_numpy(r.integers(-1, 3, 1100).astype(np.int32)).cuda()
    ws = torch.full((qmm.qmm_lora_workspace_max_bytes(1100, 1056, 40),), 0xFF, dtype=torch.uint8, device="cuda")
    for n, k in ((1100, 1056), (705, 1056), (704, 1056), (513, 1024), (512, 1056), (300, 1056), (1, 32)):
        say(f"lora, kept workspace, {n} tokens of {k}")
        args = (x[:n, :k].contiguous(), a[..., :k].contiguous(), b, ids[:n])
        got, want = qmm.qmm_lora(*args, workspace=ws), qmm.qmm_lora(*args)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("prefix,cap", [(100, 50), (3000, 50), (0, 2000)])
def test_output_in_place_of_the_queries(prefix, cap):
    r = rng(52)
    q = _normal(r, 9, 8, 64).half()
    pk, pv = (_normal(r, prefix, 2, 64).half() if prefix else None for _ in range(2))
    k, v = (_normal(r, 9, cap, 2, 64).half() for _ in range(2))
    lengths = torch.tensor([i * cap // 8 for i in range(9)], dtype=torch.int32).cuda()
    say(f"shared, O in place of Q, prefix {prefix}, caches of {cap}")
    want = qmm.qmm_attn_shared(q, pk, pv, k, v, lengths)
    got = qmm.qmm_attn_shared(q, pk, pv, k, v, lengths, O=q)
    torch.cuda.synchronize()
    assert got is q and torch.equal(got, want)
