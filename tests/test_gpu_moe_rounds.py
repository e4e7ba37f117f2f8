"""qmm_moe at the sizes where gate's and up's workgroups are divided another way: as many
as run at once with this type's LDS, one set of rows more, and more than any division."""
import pytest

from attn_util import rng, say
from test_gpu_moe import Q, check, layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tin,ffs", [("q8_0", [4096, 4128, 8192, 8224, 16384, 16416]), ("q4_0", [6144, 6176, 16384, 16416])])
@pytest.mark.parametrize("n", [1, 3])
def test_rounds(tin, ffs, n):
    g = rng(170, n, Q[tin])
    for ff in ffs:
        say(f"moe rounds {tin} {ff} {n}")
        check(*layer(g, n, 2, 256, ff, tin, "q4_0"), tin, "q4_0", 2, what=f"{ff} rows")
