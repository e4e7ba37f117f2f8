"""qmm_moe where an expert's tokens are many (a second set for the ninth and on),
all, or one of 512 experts', in rows short and long, and in a workspace of its size."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
from attn_util import rng, say
from test_gpu_moe import Q, check, layer, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k,ff", [(64, 96), (512, 768), (288, 544)])
@pytest.mark.parametrize("n,experts,used", [(8, 1, 1), (9, 1, 1), (16, 1, 1), (16, 3, 3), (12, 2, 1), (10, 5, 4)])
def test_many_tokens_of_an_expert(k, ff, n, experts, used):
    g = rng(100, n, experts, k)
    say(f"moe sets {n} {experts} {used} {k} {ff}")
    check(*layer(g, n, experts, k, ff, "q4_0", "q8_0"), "q4_0", "q8_0", used)


@pytest.mark.parametrize("tin", list(Q))
def test_types_with_two_sets(tin):
    g = rng(101, Q[tin])
    tout = list(Q)[(list(Q).index(tin) + 1) % 6]
    say(f"moe two sets {tin} {tout}")
    check(*layer(g, 13, 2, 512, 256, tin, tout), tin, tout, 2)


def test_most_experts_and_choices():
    g = rng(102)
    say("moe 16 tokens, 32 of 512")
    check(*layer(g, 16, 512, 64, 32, "q4_0", "q4_0"), "q4_0", "q4_0", 32)


@pytest.mark.parametrize("n,experts,used,k,ff", [(1, 8, 2, 512, 256), (5, 20, 6, 256, 288), (16, 2, 2, 512, 512),
                                                 (16, 40, 3, 2048, 64)])
def test_workspace_of_its_size(n, experts, used, k, ff):
    g = rng(103, n)
    say(f"moe workspace {n} {experts} {used} {k} {ff}")
    x, router, gate, up, down = layer(g, n, experts, k, ff, "q4_0", "q4_0")[:5]
    need = qmm.qmm_moe_workspace_bytes(n, k, ff, experts, used)
    buf = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    want = run(x, router, gate, up, down, "q4_0", "q4_0", used)
    for _ in range(2):
        got = run(x, router, gate, up, down, "q4_0", "q4_0", used, workspace=buf[:need])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (buf[need:] == 0xFF).all()
