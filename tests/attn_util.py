"""Inputs and comparisons of the tests of include/qmm_attn.h's operators."""
import numpy as np
import torch

from gpu_util import say  # noqa: F401 - re-exported

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rng(*key):
    return np.random.Generator(np.random.PCG64(np.random.SeedSequence([77, *key])))


def rounded(a, kind):
    """The values of a (float64) rounded to the type, as a CPU tensor of the type."""
    return torch.from_numpy(np.ascontiguousarray(a)).to(TORCH[kind])


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def assert_within(got, want, err, what):
    """Every element of got (a tensor) within err of want; NaNs where want has them."""
    g = f64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(g), nan), f"{what}: NaN at {np.argwhere(np.isnan(g) != nan)[:5].tolist()}"
    off = np.abs(g - want) - err
    off[nan] = -1.0
    inf = np.isinf(want)
    off[inf] = np.where(g[inf] == want[inf], -1.0, np.inf)
    if (off > 0).any():
        i = np.unravel_index(int(np.argmax(off)), off.shape)
        raise AssertionError(f"{what}: {int((off > 0).sum())} of {off.size} outside; worst at {i}: {g[i]!r}, "
                             f"want {want[i]!r} within {err[i]:.3g}")
