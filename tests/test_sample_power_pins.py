"""The powers that qmm_sample's weights are made of, in the kernel's own steps:
its constants, read from the source, against 2^x in 50 digits."""
import os
import re
from decimal import Decimal, getcontext

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = open(os.path.join(HERE, "..", "block_quantized_matmul_amd", "csrc", "sample.hip")).read()


def test_polynomial():
    """Within 2^-46 of itself over the whole rest of a 64th of an octave, as the tests of the tokens take it to be."""
    getcontext().prec = 50
    a = [float(re.search(rf"\ba{i} = (-?[0-9.e-]+)", SOURCE)[1]) for i in range(1, 6)]
    worst = 0
    for rest in [0.5, -0.5, *np.random.default_rng(1).uniform(-0.5, 0.5, 500)]:
        rest, s = float(rest), 0.0
        for c in reversed(a):
            s = s * rest + c
        want = Decimal(2) ** (-Decimal(rest) / 64)
        worst = max(worst, abs(Decimal(rest * s + 1.0) / want - 1))
    assert worst < Decimal(2) ** -50


def test_table():
    """Products of the roots 2^-1/2, 2^-1/4, .. 2^-1/64, as the kernel makes its table."""
    getcontext().prec = 50
    roots = [float.fromhex(x) for x in re.search(r"kRoots\[\] = \{([^}]*)\}", SOURCE)[1].replace(" ", "").split(",")]
    assert len(roots) == 6
    for j in range(64):
        p = 2.0 ** 44
        for b, r in enumerate(roots):
            p *= r if j >> (5 - b) & 1 else 1.0
        assert abs(Decimal(p) / Decimal(2) ** (44 - Decimal(j) / 64) - 1) < Decimal(2) ** -50
