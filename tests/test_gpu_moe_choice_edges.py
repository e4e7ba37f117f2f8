"""qmm_moe's choice where logits are infinite, NaN or zeros of either sign."""
import numpy as np
import pytest
import torch

import oracle.serve_oracle as S
from attn_util import f64, rng, say
from test_gpu_moe import check, layer, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,experts", [(2, 6), (16, 34)])
def test_nan_is_below_infinity(n, experts):
    """Experts of logit -infinity come before those of a NaN, whatever their indexes; their weight is zero."""
    g = rng(160, n)
    x, router, gate, up, down, gv, uv, dv = layer(g, n, experts, 64, 64, "q4_0", "q4_0")
    x[:, 7] = x[:, 7].abs() + 0.5
    router[:, 7] = 0
    router[0] = router[2] = float("nan")
    router[3, 7] = router[experts - 1, 7] = float("-inf")
    say(f"moe NaN and -infinity {n} {experts}")
    used = experts - 2
    ids = S.choice(f64(x), f64(router), used)[0]
    assert (np.sort(ids[:, -2:], -1) == [3, experts - 1]).all()
    check(x, router, gate, up, down, gv, uv, dv, "q4_0", "q4_0", used)


def test_all_nan():
    """The first experts, with weights and outputs of NaN, which leave the other tokens alone."""
    g = rng(161)
    x, router, gate, up, down, gv, uv, dv = layer(g, 3, 5, 64, 64, "q4_0", "q4_0")
    router[:, 3] = 0
    clean = run(x, router, gate, up, down, "q4_0", "q4_0", 2)
    bad = x.clone()
    bad[1, 3] = float("inf")
    say("moe all NaN")
    y, ids, w = run(bad, router, gate, up, down, "q4_0", "q4_0", 2)
    assert ids[1].tolist() == [0, 1] and bool(torch.isnan(w[1]).all()) and not bool(torch.isfinite(y[1]).any())
    for a, b in zip(clean, (y, ids, w)):
        assert torch.equal(a[[0, 2]], b[[0, 2]])


def test_zeros_of_either_sign_are_equal():
    g = rng(162)
    x, router, gate, up, down, gv, uv, dv = layer(g, 2, 8, 64, 64, "q4_0", "q4_0")
    router[:] = 0
    router[2], router[5] = -0.0, -0.0
    say("moe zeros")
    check(x, router, gate, up, down, gv, uv, dv, "q4_0", "q4_0", 4)
