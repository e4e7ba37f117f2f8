"""qmm_sample in a workspace of exactly its size, at vocabularies around those where a
part of it ends; nothing in front of it or behind it is written."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
from attn_util import rng, rounded, say
from test_gpu_sample import check, settings

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("n,vocab", [(1, 1), (5, 7), (3, 16), (70, 17), (9, 100), (3, 8191), (2, 8193), (2, 16383),
                                     (2, 16385), (3, 40000)])
def test_exact_size(n, vocab, flat):
    """Ordinary rows, and ones whose elements are all in question: equal but for one, or one step apart."""
    g = rng(115, n, vocab)
    z = 3 * g.standard_normal((n, vocab))
    if flat:
        z = np.round(z) * 2.0 ** -20
        z[:, vocab // 2] = 9.0
    z, u, kw = rounded(z, "f32"), g.random(n), settings(g, n)
    need = qmm.qmm_sample_workspace_bytes(n, vocab)
    say(f"sample workspace {n} {vocab} {flat}")
    want = check(z, u, "workspace", **kw)
    buf = torch.full((4096 + need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    dev = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32).cuda() for k, v in kw.items()}
    for at in (4096, 16):  # (aligned to 16 bytes only)
        buf.fill_(0xA5)
        got = qmm.qmm_sample(z.cuda(), torch.tensor(u, dtype=torch.float32).cuda(), workspace=buf[at:at + need], **dev)
        assert np.array_equal(got.cpu().numpy(), want)
        assert bool((buf[:at] == 0xA5).all()) and bool((buf[at + need:] == 0xA5).all())
