"""Host-side checks of include/qmm_serve.h's entry points and their binding (no
GPU needed), the size limits that the header states, and pins of the 64-bit
definitions that the GPU tests compare with.

Pointers passed here are fake (never dereferenced): validation happens on the
host first, and zero-sized calls return before any launch.
"""
import ctypes
import math
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.serve_oracle as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qmm_serve.h")
NULL = ctypes.c_void_p(0)
Q4, Q4K, Q8 = qmm.QMM_TYPE_Q4_0, qmm.QMM_TYPE_Q4_K, qmm.QMM_TYPE_Q8_0


def P(i, off=0):
    return ctypes.c_void_p(0x100000 * i + off)


def heads(data=0x100000, token=1024, head=128):
    return ctypes.byref(qmm.qmm_heads_desc(data, 0, token, head))


@pytest.fixture(scope="module")
def L():
    qmm.qmm_kv4_page_bytes(16, 1, 64)  # declares the argument types
    return qmm.lib()


def test_header_matches_library_and_binding(L):
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"^(?:int|int64_t)\s+(qmm_[a-z_0-9]+)\s*\(", text, re.M)))
    assert names == ["qmm_attn_kv4", "qmm_attn_kv4_workspace_bytes", "qmm_kv4_append", "qmm_kv4_page_bytes",
                     "qmm_kv4_read", "qmm_moe", "qmm_moe_workspace_bytes", "qmm_sample", "qmm_sample_workspace_bytes"]
    for name in names:
        assert hasattr(L, name) and hasattr(qmm, name), name
    constants = re.findall(r"#define (QMM_[A-Z_0-9]+) (\d+)", text)
    assert len(constants) == 5
    for name, val in constants:
        assert getattr(qmm, name) == int(val), name


def test_page_bytes(L):
    for page in (16, 32, 64, 128, 256):
        for dim in (64, 128):
            assert qmm.qmm_kv4_page_bytes(page, 3, dim) == 3 * page * 2 * (dim // 2 + 2 * dim // 32)
    for bad in ((0, 1, 64), (8, 1, 64), (24, 1, 64), (512, 1, 64), (-16, 1, 64), (16, 0, 64), (16, -1, 64), (16, 1, 96),
                (16, 1 << 31, 64)):
        assert L.qmm_kv4_page_bytes(*bad) == qmm.QMM_ERR_SHAPE, bad
        with pytest.raises(qmm.QmmError):
            qmm.qmm_kv4_page_bytes(*bad)


def _append(L, t=0, K=heads(), V=heads(), n=5, hkv=2, dim=128, norm=0, w=NULL, eps=1e-6, pos=P(2), freqs=(0.5, 0.25),
            n_freqs=None, pairs=0, slots=P(3), cache=P(4), pages=7, page=32):
    fp = None if freqs is None else (ctypes.c_double * len(freqs))(*freqs)
    n_freqs = len(freqs or ()) if n_freqs is None else n_freqs
    return L.qmm_kv4_append(t, K, V, n, hkv, dim, norm, w, eps, pos, fp, n_freqs, pairs, slots, cache, pages, page, NULL)


def test_append_validation(L):
    E = qmm
    for bad in (dict(t=3), dict(t=-1), dict(pairs=2), dict(pairs=-1)):
        assert _append(L, **bad) == E.QMM_ERR_TYPE, bad
    for bad in (dict(K=None), dict(V=None), dict(K=heads(0)), dict(V=heads(0)), dict(pos=NULL), dict(slots=NULL),
                dict(cache=NULL), dict(freqs=None, n_freqs=2)):
        assert _append(L, **bad) == E.QMM_ERR_NULL, bad
    for bad in (dict(n=-1), dict(n=1 << 31), dict(hkv=0), dict(dim=32), dict(dim=96), dict(dim=256), dict(n_freqs=65),
                dict(n_freqs=-1), dict(eps=-1e-9), dict(eps=math.nan), dict(eps=math.inf), dict(freqs=(64.5,)),
                dict(freqs=(math.nan,)), dict(pages=0), dict(pages=-1), dict(pages=1 << 26), dict(page=8), dict(page=48),
                dict(page=512), dict(n=(1 << 31) - 1, hkv=1 << 20), dict(K=heads(token=1 << 60)),
                dict(V=heads(head=1 << 61))):
        assert _append(L, **bad) == E.QMM_ERR_SHAPE, bad
    for bad in (dict(K=heads(token=-1)), dict(V=heads(head=-128))):
        assert _append(L, **bad) == E.QMM_ERR_STRIDE, bad
    for bad in (dict(K=heads(0x100002)), dict(V=heads(0x100001), t=1), dict(pos=P(2, 2)), dict(slots=P(3, 1)),
                dict(w=P(5, 2)), dict(cache=P(4, 8))):
        assert _append(L, **bad) == E.QMM_ERR_ALIGN, bad
    # empty calls, with nothing behind their pointers; strides of axes of one element do not matter
    assert _append(L, n=0, K=None, V=None, pos=NULL, slots=NULL) == E.QMM_OK
    assert _append(L, n=1, hkv=1, K=heads(0x100000, -5, -7), slots=NULL) == E.QMM_ERR_NULL


def _read(L, t=0, K=heads(), V=heads(), n=5, hkv=2, dim=128, slots=P(3), cache=P(4), pages=7, page=32):
    return L.qmm_kv4_read(t, K, V, n, hkv, dim, slots, cache, pages, page, NULL)


def test_read_validation(L):
    E = qmm
    assert _read(L, t=3) == E.QMM_ERR_TYPE
    for bad in (dict(K=heads(0)), dict(V=heads(0)), dict(slots=NULL), dict(cache=NULL)):
        assert _read(L, **bad) == E.QMM_ERR_NULL, bad
    for bad in (dict(n=-1), dict(n=1 << 31), dict(dim=100), dict(pages=0), dict(page=17)):
        assert _read(L, **bad) == E.QMM_ERR_SHAPE, bad
    for bad in (dict(K=heads(token=-1)), dict(V=heads(head=127)), dict(K=heads(token=255)), dict(K=heads(head=0)),
                dict(V=heads(token=0))):  # (rows that share elements)
        assert _read(L, **bad) == E.QMM_ERR_STRIDE, bad
    for bad in (dict(K=heads(0x100002)), dict(slots=P(3, 2)), dict(cache=P(4, 4))):
        assert _read(L, **bad) == E.QMM_ERR_ALIGN, bad
    assert _read(L, n=0, slots=NULL) == E.QMM_OK
    assert _read(L, K=None, V=None, slots=NULL) == E.QMM_OK
    assert _read(L, K=heads(token=128, head=640), slots=NULL) == E.QMM_ERR_NULL  # heads outside, tokens inside


def _attn(L, t=1, Q=heads(), O=heads(0x900000), n=3, hq=8, hkv=2, dim=128, cache=P(4), pages=7, page=32, tables=P(5),
          stride=64, width=64, lengths=P(6), scale=0.1, ws=P(7), ws_bytes=1 << 40):
    return L.qmm_attn_kv4(t, Q, O, n, hq, hkv, dim, cache, pages, page, tables, stride, width, lengths, scale, ws,
                          ws_bytes, NULL)


def test_attention_validation(L):
    E = qmm
    for t in (0, 3, -1):
        assert _attn(L, t=t) == E.QMM_ERR_TYPE
    for bad in (dict(Q=None), dict(O=None), dict(Q=heads(0)), dict(O=heads(0)), dict(cache=NULL), dict(tables=NULL),
                dict(lengths=NULL)):
        assert _attn(L, **bad) == E.QMM_ERR_NULL, bad
    for bad in (dict(n=-1), dict(n=1 << 24), dict(n=1 << 22, hq=4, hkv=4), dict(hq=7), dict(hq=0), dict(hkv=0),
                dict(hkv=16), dict(dim=32), dict(page=20), dict(width=-1), dict(width=1 << 26), dict(pages=0),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=2.0 ** 127)):
        assert _attn(L, **bad) == E.QMM_ERR_SHAPE, bad
    for bad in (dict(Q=heads(token=1028)), dict(O=heads(0x900000, head=132)), dict(Q=heads(token=-8)), dict(stride=-1),
                dict(O=heads(0x900000, head=64)), dict(O=heads(0x900000, token=0)), dict(stride=1 << 62)):
        assert _attn(L, **bad) == E.QMM_ERR_STRIDE, bad
    for bad in (dict(Q=heads(0x100008)), dict(O=heads(0x900002)), dict(cache=P(4, 8)), dict(tables=P(5, 2)),
                dict(lengths=P(6, 1)), dict(ws=P(7, 8))):
        assert _attn(L, **bad) == E.QMM_ERR_ALIGN, bad
    need = L.qmm_attn_kv4_workspace_bytes(3, 8, 2, 128, 64, 32)
    assert need > 0
    assert _attn(L, ws=NULL) == E.QMM_ERR_WORKSPACE and _attn(L, ws_bytes=need - 1) == E.QMM_ERR_WORKSPACE
    assert _attn(L, n=0, Q=None, O=None, tables=NULL, lengths=NULL, ws=NULL) == E.QMM_OK


def test_attention_workspaces(L):
    W = L.qmm_attn_kv4_workspace_bytes
    assert W(0, 8, 2, 128, 9, 32) == 0 and W(5, 8, 2, 128, 0, 32) == 0
    assert W(1, 8, 2, 128, 1, 256) == 0  # nothing to divide
    for dim in (64, 128):
        most = qmm.qmm_attn_kv4_workspace_max_bytes(dim)
        assert most < 9.1e6
        largest = 0
        for hq, hkv in ((1, 1), (8, 1), (33, 1), (64, 2), (40, 8), (32, 32), (128, 128), (96, 3), (1000, 10), (1023, 1023)):
            for n in list(range(1, 70)) + [100, 127, 128, 129, 255, 500, 511, 512, 1000, 1023, 1024, 5000]:
                for width in (1, 2, 3, 100, 1 << 18):
                    need = W(n, hq, hkv, dim, width, 256)
                    assert 0 <= need <= most, (n, hq, hkv, dim, width, need)
                    largest = max(largest, need)
        assert largest > most / 3  # a bound, but no wild one
    assert W(1, 32, 8, 128, 1000, 64) > W(1024, 32, 8, 128, 1000, 64) == 0  # why there is one
    with pytest.raises(ValueError):
        qmm.qmm_attn_kv4_workspace_max_bytes(96)


def _moe(L, X=P(1), xt=0, n=3, k=256, router=P(2), experts=8, used=2, gate=P(3), up=P(4), ti=Q4, ff=512, s1=144, s2=512 * 144,
         down=P(5), to=Q4, d1=288, d2=256 * 288, Y=P(6), ids=NULL, weights=NULL, ws=P(7), ws_bytes=1 << 40):
    return L.qmm_moe(X, xt, n, k, router, experts, used, 1, gate, up, ti, ff, s1, s2, down, to, d1, d2, Y, ids, weights, ws,
                     ws_bytes, NULL)


def test_moe_validation(L):
    E = qmm
    for bad in (dict(xt=2), dict(xt=-1), dict(ti=99), dict(to=-1)):
        assert _moe(L, **bad) == E.QMM_ERR_TYPE, bad
    for bad in (dict(X=NULL), dict(router=NULL), dict(gate=NULL), dict(up=NULL), dict(down=NULL), dict(Y=NULL)):
        assert _moe(L, **bad) == E.QMM_ERR_NULL, bad
    for bad in (dict(n=-1), dict(n=17), dict(k=0), dict(k=48), dict(k=1 << 24), dict(ff=0), dict(ff=500), dict(experts=0),
                dict(experts=513), dict(used=0), dict(used=9), dict(used=33, experts=64),
                dict(experts=512, s2=1 << 58)):
        assert _moe(L, **bad) == E.QMM_ERR_SHAPE, bad
    for bad in (dict(s1=140), dict(s1=146), dict(s2=512 * 144 - 4), dict(s2=512 * 144 + 2), dict(d1=284), dict(d1=290),
                dict(d2=256 * 288 - 4), dict(d1=1 << 61)):
        assert _moe(L, **bad) == E.QMM_ERR_STRIDE, bad
    assert _moe(L, ti=Q4K, k=128, s1=80) < 0  # a Q4_K row holds multiples of 256
    for bad in (dict(X=P(1, 2)), dict(router=P(2, 1)), dict(gate=P(3, 2)), dict(up=P(4, 2)), dict(down=P(5, 2)),
                dict(Y=P(6, 2)), dict(ids=P(8, 2)), dict(weights=P(9, 2)), dict(ws=P(7, 8))):
        assert _moe(L, **bad) == E.QMM_ERR_ALIGN, bad
    need = L.qmm_moe_workspace_bytes(3, 256, 512, 8, 2)
    assert _moe(L, ws=NULL) == E.QMM_ERR_WORKSPACE and _moe(L, ws_bytes=need - 1) == E.QMM_ERR_WORKSPACE
    assert _moe(L, n=0, X=NULL, router=NULL, gate=NULL, up=NULL, down=NULL, Y=NULL, ws=NULL) == E.QMM_OK


def test_moe_workspace_grows_with_every_size(L):
    W = L.qmm_moe_workspace_bytes
    for bad in ((17, 32, 32, 1, 1), (1, 33, 32, 1, 1), (1, 32, 1 << 24, 1, 1), (1, 32, 32, 513, 1), (1, 32, 32, 4, 5)):
        assert W(*bad) == qmm.QMM_ERR_SHAPE, bad
    steps = ([1, 2, 3, 4, 5, 8, 9, 12, 16], [32, 64, 288, 1024, 2048, 2080, 4096, 4128, 8192, 8224, 16384, 65536, (1 << 24) - 32],
             [32, 96, 1408, 14336], [8, 9, 64, 512], [1, 2, 6, 8])
    base = [3, 2048, 1408, 64, 6]
    for n in steps[0]:
        for axis in range(1, 5):
            before = 0
            for v in steps[axis]:
                size = list(base)
                size[0], size[axis] = n, v
                need = W(*size)
                assert need >= before > -1, size
                before = need
    for k in steps[1]:
        before = 0
        for n in steps[0]:
            need = W(n, k, 1408, 64, 6)
            assert need > before
            before = need
    assert W(0, 32, 32, 1, 1) == 0


def _sample(L, z=P(1), t=0, n=3, vocab=100, stride=100, u=P(2), temp=NULL, k=NULL, p=NULL, m=NULL, tokens=P(3), probs=NULL,
            ws=P(4), ws_bytes=1 << 50):
    return L.qmm_sample(z, t, n, vocab, stride, u, temp, k, p, m, tokens, probs, ws, ws_bytes, NULL)


def test_sample_validation(L):
    E = qmm
    assert _sample(L, t=3) == E.QMM_ERR_TYPE
    for bad in (dict(z=NULL), dict(u=NULL), dict(tokens=NULL)):
        assert _sample(L, **bad) == E.QMM_ERR_NULL, bad
    for bad in (dict(n=-1), dict(n=1 << 22), dict(vocab=0), dict(vocab=-1), dict(vocab=524288), dict(stride=1 << 60)):
        assert _sample(L, **bad) == E.QMM_ERR_SHAPE, bad
    assert _sample(L, stride=-1) == E.QMM_ERR_STRIDE
    for bad in (dict(z=P(1, 2)), dict(z=P(1, 1), t=1), dict(u=P(2, 2)), dict(temp=P(5, 2)), dict(k=P(5, 1)), dict(p=P(5, 3)),
                dict(m=P(5, 2)), dict(tokens=P(3, 2)), dict(probs=P(5, 2)), dict(ws=P(4, 8))):
        assert _sample(L, **bad) == E.QMM_ERR_ALIGN, bad
    W = L.qmm_sample_workspace_bytes
    assert _sample(L, ws=NULL) == E.QMM_ERR_WORKSPACE and _sample(L, ws_bytes=W(3, 100) - 1) == E.QMM_ERR_WORKSPACE
    assert _sample(L, n=0, z=NULL, u=NULL, tokens=NULL, ws=NULL) == E.QMM_OK
    assert _sample(L, n=1, stride=-3, ws=NULL) == E.QMM_ERR_WORKSPACE  # one row has no stride
    assert W(0, 100) == 0 and W(1 << 22, 100) == W(1, 524288) == W(-1, 5) == W(1, 0) == E.QMM_ERR_SHAPE
    for vocab in (1, 8192, 8193, 32000, 130001, 524287):
        assert W(2, vocab) == 2 * W(1, vocab) and W(1, vocab) >= W(1, max(1, vocab - 8192)) and W(1, vocab) % 8 == 0


def test_the_header_is_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "sizes.c", tmp_path / "sizes"
    src.write_text('#include <stdio.h>\n#include "qmm_serve.h"\nint main(void) {\n'
                   'printf("%lld %lld\\n", (long long)qmm_attn_kv4_workspace_max_bytes(64),\n'
                   '       (long long)qmm_attn_kv4_workspace_max_bytes(128));\nreturn 0;\n}\n')
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [qmm.qmm_attn_kv4_workspace_max_bytes(d) for d in (64, 128)]


def test_binding_refuses_cpu_tensors():
    f, i = torch.zeros, lambda *s: torch.zeros(*s, dtype=torch.int32)
    cache = torch.zeros(2, qmm.qmm_kv4_page_bytes(16, 1, 64), dtype=torch.uint8)
    w = torch.zeros(4, 32, 20, dtype=torch.uint8)
    for call in (lambda: qmm.qmm_kv4_append(f(2, 1, 64), f(2, 1, 64), cache, 16, i(2)),
                 lambda: qmm.qmm_kv4_read(cache, 16, i(2), 1, 64),
                 lambda: qmm.qmm_attn_kv4(f(2, 1, 64).half(), cache, 16, 1, i(2, 2), i(2)),
                 lambda: qmm.qmm_moe(f(2, 32), f(4, 32), w, w, Q4, w, Q4, 2),
                 lambda: qmm.qmm_sample(f(2, 9), f(2))):
        with pytest.raises(TypeError, match="GPU tensor"):
            call()


# ---- the 64-bit definitions

def test_oracle_blocks():
    x = np.zeros(32)
    x[3], x[9], x[20] = 4.0, -8.0, 8.0  # the first of the largest magnitudes is negative: d = 1
    d, codes = S.quantise(x)
    assert d == 0x3C00 and codes[3] == 12 and codes[9] == 0 and codes[20] == 15 and codes[0] == 8
    d, codes = S.quantise(np.zeros(32))
    assert d == 0 and (codes == 8).all()
    d, codes = S.quantise(np.where(np.arange(32) == 5, np.inf, 1.0))
    assert d == 0x7E00 and (codes == 8).all()


def test_oracle_append_and_read_are_one_cache():
    g = np.random.default_rng(5)
    for page, heads_, dim in ((16, 2, 64), (64, 3, 128)):
        cache = np.zeros((2, S.page_bytes(page, heads_, dim)), np.uint8)
        k, v = g.standard_normal((2, 9, heads_, dim))
        slots = g.permutation(2 * page)[:9].astype(np.int32)
        new = S.append(k, v, cache, page, slots)
        assert cache.max() == 0
        rk, rv = S.read(new, page, slots, heads_, dim)[:2]
        for got, x in ((rk, k), (rv, v)):
            # a step is at most an eighth of a block's largest magnitude: half of one, and a whole at the end of the codes
            largest = np.abs(x.reshape(9, heads_, -1, 32)).max(-1, keepdims=True)
            assert (np.abs(got - x).reshape(9, heads_, -1, 32) <= largest * (0.125 * 1.001)).all()
        other = S.read(new, page, np.setdiff1d(np.arange(2 * page), slots).astype(np.int32), heads_, dim)[0]
        assert (other == 0).all()
        outside = S.read(new, page, np.array([-1, 2 * page], np.int32), heads_, dim)[0]
        assert np.isnan(outside).all()


def test_oracle_choice():
    router = np.eye(4)
    router[3] = np.nan
    ids, w = S.choice(np.array([[1.0, 3.0, 3.0, 9.0]]), router, 2)
    assert list(np.asarray(ids)[0]) == [1, 2] and np.allclose(np.asarray(w)[0], 0.5)


def test_oracle_sampling():
    z = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    for u, token in ((0.0, 1), (0.399, 1), (0.401, 3), (0.699, 3), (0.701, 2), (0.899, 2), (0.901, 0)):
        assert S.sample(z, u)[0] == token, u
    assert S.sample(z, 0.99, top_k=2)[0] == 3
    assert S.sample(z, 0.99, top_p=0.5)[0] == 3   # 0.4 does not reach a half, 0.7 does
    assert S.sample(z, 0.99, min_p=0.6)[0] == 3   # 0.3 / 0.4 stays, 0.2 / 0.4 does not
    assert S.sample(z, 0.99, temperature=0.0)[0] == 1
    assert S.sample(np.full(5, -np.inf), 0.5)[0] == -1
