"""qmm_sample where its ways differ: rows at the ends of a chunk of 8192, ranges
with many elements, many equal ones, and more than are looked at one by one."""
import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
from attn_util import rng, rounded, say
from test_gpu_sample import check, run, settings

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [8191, 8192, 8193, 8196, 16384, 16385, 40961, 524287])
def test_chunks(vocab):
    g = rng(80, vocab)
    n = 8 if vocab < 100000 else 3
    say(f"sample chunks {vocab}")
    check(rounded(2 * g.standard_normal((n, vocab)), "f32"), g.random(n), "chunks", **settings(g, n))


@pytest.mark.parametrize("flat", [0.01, 0.3])
def test_full_ranges(flat):
    """Nearly flat rows with one much larger logit: the others lie in few ranges."""
    g = rng(81, int(100 * flat))
    n, vocab = 6, 60000
    say(f"sample full ranges {flat}")
    z = flat * g.standard_normal((n, vocab))
    z[:, 777] = np.array([1.0, 4.0, 8.0, 12.0, 12.0, 30.0])
    kw = dict(top_k=np.array([0, 0, 500, 20000, 59999, 7]), top_p=np.array([0.9, 0.5, 1.0, 0.99, 1.0, 0.999]))
    check(rounded(z, "f32"), g.random(n), "full ranges", **kw)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("distinct,vocab", [(40, 8000), (12, 30000), (3, 9000), (2, 100000)])
def test_many_equal(kind, distinct, vocab):
    """Of equal logits the lower indexes come first, also where they are thousands."""
    g = rng(82, distinct, vocab)
    n = 6
    say(f"sample many equal {kind} {distinct} {vocab}")
    z = rounded(g.choice(np.arange(distinct) * 0.25, (n, vocab)), kind)
    kw = dict(top_k=np.array([0, 100, 5000, 0, 1, 2000]), top_p=np.array([1.0, 0.9, 0.6, 0.3, 1.0, 0.97]),
              temperature=np.array([1.0, 0.7, 2.0, 5.0, 1.0, 0.2]))
    check(z, g.random(n), "many equal", **kw)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [3873, 50000])
def test_top_k_ends_among_elements_without_a_weight(kind, vocab):
    """Peaked rows: a few likely tokens, all others below 2^-45 of the largest; and some of others on either side."""
    g = rng(85, vocab)
    n = 8
    say(f"sample peaked {kind} {vocab}")
    z = 2 * g.standard_normal((n, vocab))
    for i in range(n):
        z[i, g.permutation(vocab)[:5 + 9 * i]] += 60 + 3 * g.standard_normal(5 + 9 * i)
    kw = dict(top_k=np.array([200, 150, 23, 33, 40, 3000, 0, 60]), top_p=np.array([1.0, 0.9, 1.0, 0.99, 0.7, 1.0, 0.95, 1.0]),
              temperature=np.array([0.5, 0.7, 1.0, 1.0, 0.3, 1.0, 1.0, 1.9]),
              min_p=np.array([0.0, 0.0, 0.0, 0.01, 0.0, 0.05, 0.0, 0.0]))
    check(rounded(z, kind), g.random(n), "peaked", **kw)


def test_few_and_many_in_one_call():
    """Rows that go different ways, among them rows without a probability."""
    g = rng(83)
    vocab = 20000
    say("sample few and many")
    z = np.stack([10 * g.standard_normal(vocab), 0.01 * g.standard_normal(vocab), np.full(vocab, 1.5), np.full(vocab, -np.inf),
                  np.where(g.random(vocab) < 0.3, np.inf, 0.0), g.standard_normal(vocab), np.full(vocab, np.nan),
                  1e30 * g.standard_normal(vocab), 1e-30 * g.standard_normal(vocab)])
    kw = dict(top_k=np.array([0, 3, 0, 5, 9, 40, 1, 0, 0]), top_p=np.array([0.9, 1.0, 0.5, 0.5, 0.8, 0.95, 1.0, 0.9, 0.9]))
    check(rounded(z, "f32"), g.random(len(z)), "few and many", **kw)


def test_workspace_is_the_callers():
    """A workspace with anything in it, used by call after call of different sizes; nothing behind it is written."""
    g = rng(84)
    say("sample workspace")
    need = qmm.qmm_sample_workspace_bytes(7, 30000)
    buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for n, vocab in ((7, 30000), (3, 100), (7, 30000), (1, 16385)):
        z = rounded(3 * g.standard_normal((n, vocab)), "f32").cuda()
        u, kw = g.random(n), settings(g, n)
        want = run(z, u, **kw)
        got = torch.empty(n, dtype=torch.int32, device="cuda")
        dev = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32).cuda() for k, v in kw.items()}
        qmm.qmm_sample(z, torch.tensor(u, dtype=torch.float32).cuda(), tokens=got, workspace=buf[:need], **dev)
        assert np.array_equal(got.cpu().numpy(), want[0])
    assert (buf[need:] == 0xA5).all()
    with pytest.raises(qmm.QmmError):
        qmm.qmm_sample(z, torch.zeros(1, device="cuda"), workspace=buf[:64])
