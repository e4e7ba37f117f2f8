"""Host-side checks of include/qmm_attn.h's entry points and their binding (no
GPU needed), and pins of the 64-bit definitions the GPU tests compare with.

Pointers passed here are fake (never dereferenced): validation happens on the
host first, and zero-sized calls return before any launch.
"""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import block_quantized_matmul_amd as qmm
import oracle.attn_oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qmm_attn.h")
NULL = ctypes.c_void_p(0)


def P(i, off=0):
    return ctypes.c_void_p(0x10000 * i + off)


@pytest.fixture(scope="module")
def L():
    qmm.qmm_lora_workspace_bytes(1, 32, 1)  # declares the argument types
    return qmm.lib()


def test_header_matches_library_and_binding(L):
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"^(?:int|int64_t)\s+(qmm_[a-z_0-9]+)\s*\(", text, re.M)))
    assert names == ["qmm_attn_prompt", "qmm_attn_shared", "qmm_attn_shared_workspace_bytes", "qmm_lora",
                     "qmm_lora_workspace_bytes", "qmm_norm_rope"]
    for name in names:
        assert hasattr(L, name) and hasattr(qmm, name), name
    for name, val in re.findall(r"#define (QMM_[A-Z_0-9]+) (\d+)", text):
        assert getattr(qmm, name) == int(val), name
    assert ctypes.sizeof(qmm.qmm_heads_desc) == 32 and ctypes.sizeof(qmm.qmm_head_part_desc) == 96


def _lora(L, X=P(1), xt=0, n=3, k=64, A=P(2), B=P(3), ad=4, rank=8, rows=16, scales=NULL, ids=P(4), base=NULL, Y=P(5),
          ws=P(6), ws_bytes=1 << 40):
    return L.qmm_lora(X, xt, n, k, A, B, ad, rank, rows, scales, ids, base, Y, ws, ws_bytes, NULL)


def test_lora_validation(L):
    E = qmm
    for name in ("X", "A", "B", "ids", "Y"):
        assert _lora(L, **{name: NULL}) == E.QMM_ERR_NULL, name
    assert _lora(L, xt=2) == E.QMM_ERR_TYPE and _lora(L, xt=-1) == E.QMM_ERR_TYPE
    for bad in (dict(k=0), dict(k=40), dict(k=-32), dict(k=1 << 24), dict(n=-1), dict(n=1 << 25), dict(rank=0),
                dict(rank=257), dict(rows=-1), dict(rows=1 << 31), dict(ad=-1), dict(ad=1 << 31)):
        assert _lora(L, **bad) == E.QMM_ERR_SHAPE, bad
    for bad in (dict(X=P(1, 8)), dict(A=P(2, 8)), dict(B=P(3, 1)), dict(scales=P(7, 2)), dict(ids=P(4, 2)),
                dict(base=P(8, 2)), dict(Y=P(5, 2)), dict(ws=P(6, 8))):
        assert _lora(L, **bad) == E.QMM_ERR_ALIGN, bad
    need = L.qmm_lora_workspace_bytes(3, 64, 8)
    assert need > 0
    assert _lora(L, ws=NULL) == E.QMM_ERR_WORKSPACE and _lora(L, ws_bytes=need - 1) == E.QMM_ERR_WORKSPACE
    # empty calls, with nothing behind their pointers
    assert _lora(L, n=0, X=NULL, ids=NULL, Y=NULL, ws=NULL) == E.QMM_OK
    assert _lora(L, rows=0, B=NULL, Y=NULL) == E.QMM_OK


def test_lora_workspace_sizes(L):
    W = L.qmm_lora_workspace_bytes
    assert W(0, 64, 8) == 0
    for n, k, rank in ((1, 32, 1), (1, 4096, 16), (512, 4096, 16), (513, 4096, 16), (2048, 11008, 64), (3, 1 << 23, 256)):
        assert W(n, k, rank) % (4 * n * rank) == 0 and W(n, k, rank) >= 4 * n * rank
        assert W(n, k, rank) <= 4 * n * rank * 512  # ranges of k stay few
    for bad in ((-1, 64, 8), (1 << 25, 64, 8), (4, 48, 8), (4, 1 << 24, 8), (4, 64, 0), (4, 64, 257)):
        assert W(*bad) == qmm.QMM_ERR_SHAPE


def _part(**kw):
    d = dict(X=0x10000, x_type=0, x_token_stride=256, x_head_stride=128, Y=0x20000, y_type=1, y_row_stride=256,
             y_head_stride=128, n_heads=2, norm=1, weight=0x30000, rotate=1, slotted=0)
    d.update(kw)
    return qmm.qmm_head_part_desc(**d)


def _rope(L, *parts, n=5, dim=128, eps=1e-6, pos=P(4), freqs=None, n_freqs=64, pairs=0, slots=P(5), n_slots=9,
          n_parts=None):
    parts = parts or (_part(),)
    arr = (qmm.qmm_head_part_desc * 4)(*parts)
    freqs = [0.5] * 256 if freqs is None else freqs
    f = (ctypes.c_double * max(1, len(freqs)))(*freqs)
    return L.qmm_norm_rope(arr, len(parts) if n_parts is None else n_parts, n, dim, eps, pos, f, n_freqs, pairs, slots,
                           n_slots, NULL)


def test_norm_rope_validation(L):
    E = qmm
    for bad in (dict(n_parts=-1), dict(n_parts=5), dict(n=-1), dict(n=1 << 31), dict(dim=0), dict(dim=7), dict(dim=514),
                dict(n_freqs=-1), dict(n_freqs=65), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(n_slots=-1), dict(freqs=[0.5] * 63 + [float("nan")]), dict(freqs=[0.5] * 63 + [64.5]),
                dict(freqs=[-float("inf")] * 64)):
        assert _rope(L, **bad) == E.QMM_ERR_SHAPE, bad
    assert _rope(L, pairs=2) == E.QMM_ERR_TYPE
    assert L.qmm_norm_rope(None, 1, 5, 128, 0.0, P(4), None, 0, 0, NULL, 0, NULL) == E.QMM_ERR_NULL
    assert L.qmm_norm_rope(None, 0, 5, 128, 0.0, NULL, None, 0, 0, NULL, 0, NULL) == E.QMM_OK
    assert _rope(L, pos=P(4, 2)) == E.QMM_ERR_ALIGN and _rope(L, slots=P(5, 2)) == E.QMM_ERR_ALIGN
    assert _rope(L, pos=NULL) == E.QMM_ERR_NULL            # a rotated part without positions
    assert _rope(L, n_freqs=0) == E.QMM_ERR_NULL           # or frequencies
    for status, kw in ((E.QMM_ERR_NULL, dict(X=None)), (E.QMM_ERR_NULL, dict(Y=None)),
                       (E.QMM_ERR_TYPE, dict(x_type=3)), (E.QMM_ERR_TYPE, dict(y_type=-1)),
                       (E.QMM_ERR_SHAPE, dict(n_heads=-1)), (E.QMM_ERR_SHAPE, dict(x_token_stride=1 << 58)),
                       (E.QMM_ERR_STRIDE, dict(x_token_stride=-256)), (E.QMM_ERR_STRIDE, dict(y_head_stride=-128)),
                       (E.QMM_ERR_STRIDE, dict(y_row_stride=128)),      # rows of two heads overlap
                       (E.QMM_ERR_STRIDE, dict(y_head_stride=64)), (E.QMM_ERR_STRIDE, dict(y_row_stride=0)),
                       (E.QMM_ERR_ALIGN, dict(X=0x10002)), (E.QMM_ERR_ALIGN, dict(Y=0x20001)),
                       (E.QMM_ERR_ALIGN, dict(weight=0x30002))):
        assert _rope(L, _part(), _part(**kw)) == status, kw
    assert _rope(L, _part(slotted=1), slots=NULL) == E.QMM_ERR_NULL
    # nothing to do: no tokens, no heads, or no slots
    assert _rope(L, _part(X=None, Y=None), n=0) == E.QMM_OK
    assert _rope(L, _part(X=None, Y=None, n_heads=0)) == E.QMM_OK
    assert _rope(L, _part(Y=None, slotted=1, rotate=0), n_slots=0) == E.QMM_OK


def _h(i, tok, head, seq=0, off=0):
    return qmm.qmm_heads_desc(0x100000 * i + off, seq, tok, head)


def _prompt(L, t=1, Q=None, K=None, V=None, O_=None, n=10, hq=4, hkv=2, dim=64, starts=P(7), seqs=2, scale=0.125):
    return L.qmm_attn_prompt(t, Q or _h(1, 256, 64), K or _h(2, 128, 64), V or _h(3, 128, 64), O_ or _h(4, 256, 64), n,
                             hq, hkv, dim, starts, seqs, scale, NULL)


def test_attn_prompt_validation(L):
    E = qmm
    assert _prompt(L, t=0) == E.QMM_ERR_TYPE and _prompt(L, t=3) == E.QMM_ERR_TYPE
    for bad in (dict(n=-1), dict(n=1 << 31), dict(hq=0), dict(hkv=0), dict(hq=3), dict(dim=32), dict(dim=96),
                dict(dim=256), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(seqs=-1), dict(seqs=1 << 31), dict(n=1 << 29, hq=8, hkv=8),
                # more workgroups than a launch holds
                dict(n=1 << 24, seqs=1 << 24, hq=32, Q=_h(1, 2048, 64), O_=_h(4, 2048, 64))):
        assert _prompt(L, **bad) == E.QMM_ERR_SHAPE, bad
    assert _prompt(L, starts=NULL) == E.QMM_ERR_NULL and _prompt(L, starts=P(7, 2)) == E.QMM_ERR_ALIGN
    for name, ok in (("Q", (256, 64)), ("K", (128, 64)), ("V", (128, 64)), ("O_", (256, 64))):
        assert _prompt(L, **{name: qmm.qmm_heads_desc(None, 0, *ok)}) == E.QMM_ERR_NULL
        assert _prompt(L, **{name: _h(5, ok[0], ok[1], off=8)}) == E.QMM_ERR_ALIGN
        assert _prompt(L, **{name: _h(5, ok[0] + 4, ok[1])}) == E.QMM_ERR_STRIDE
        assert _prompt(L, **{name: _h(5, ok[0], 60)}) == E.QMM_ERR_STRIDE
        assert _prompt(L, **{name: _h(5, -ok[0], ok[1])}) == E.QMM_ERR_STRIDE
        assert _prompt(L, **{name: _h(5, (1 << 25) + 8, ok[1])}) == E.QMM_ERR_STRIDE
        assert _prompt(L, **{name: _h(5, ok[0], 1 << 58)}) == E.QMM_ERR_SHAPE
    for strides in ((128, 64), (256, 32), (0, 64), (256, 0)):   # an output whose heads overlap
        assert _prompt(L, O_=_h(4, *strides)) == E.QMM_ERR_STRIDE
    assert _prompt(L, n=0, Q=qmm.qmm_heads_desc(), starts=NULL) == E.QMM_OK
    assert _prompt(L, seqs=0, starts=NULL) == E.QMM_OK


def _shared(L, t=1, Q=None, PK=None, PV=None, prefix=100, K=None, V=None, cap=20, lengths=P(9), O_=None, n=3, hq=4,
            hkv=2, dim=64, scale=0.125, ws=P(8), ws_bytes=1 << 40):
    return L.qmm_attn_shared(t, Q or _h(1, 256, 64), PK or _h(2, 128, 64), PV or _h(3, 128, 64), prefix,
                             K or _h(4, 128, 64, 2560), V or _h(5, 128, 64, 2560), cap, lengths, O_ or _h(6, 256, 64), n,
                             hq, hkv, dim, scale, ws, ws_bytes, NULL)


def test_scale_times_log2_e_has_to_fit(L):
    for scale in (2.0 ** 127, 3e38):
        assert _prompt(L, scale=scale) == qmm.QMM_ERR_SHAPE
        assert _shared(L, scale=scale) == qmm.QMM_ERR_SHAPE


def test_attn_shared_validation(L):
    E = qmm
    assert _shared(L, t=0) == E.QMM_ERR_TYPE
    for bad in (dict(n=-1), dict(prefix=-1), dict(cap=-1), dict(prefix=1 << 31), dict(cap=1 << 31), dict(hq=3),
                dict(hkv=0), dict(dim=80), dict(scale=0.0), dict(scale=float("inf")), dict(n=1 << 30, hq=2, hkv=2),
                dict(n=1 << 23, hq=4, hkv=4)):
        assert _shared(L, **bad) == E.QMM_ERR_SHAPE, bad
    for name in ("Q", "PK", "PV", "K", "V", "O_"):
        ok = (256, 64) if name in ("Q", "O_") else (128, 64)
        assert _shared(L, **{name: qmm.qmm_heads_desc(None, 2560, *ok)}) == E.QMM_ERR_NULL, name
        assert _shared(L, **{name: _h(7, ok[0], ok[1], 2560, off=4)}) == E.QMM_ERR_ALIGN, name
        assert _shared(L, **{name: _h(7, ok[0] + 2, ok[1], 2560)}) == E.QMM_ERR_STRIDE, name
    assert _shared(L, K=_h(4, 128, 64, 2561)) == E.QMM_ERR_STRIDE
    assert _shared(L, V=_h(4, 128, 64, -8)) == E.QMM_ERR_STRIDE
    assert _shared(L, lengths=NULL) == E.QMM_ERR_NULL and _shared(L, lengths=P(9, 1)) == E.QMM_ERR_ALIGN
    assert _shared(L, O_=_h(6, 128, 64)) == E.QMM_ERR_STRIDE
    big = dict(prefix=5000, cap=2000, K=_h(4, 128, 64, 1 << 20), V=_h(5, 128, 64, 1 << 20))
    need = L.qmm_attn_shared_workspace_bytes(3, 5000, 2000, 4, 2, 64)
    assert need > 0 and need % (4 * 65 * 12) == 0
    assert _shared(L, **big, ws=NULL) == E.QMM_ERR_WORKSPACE
    assert _shared(L, **big, ws_bytes=need - 1) == E.QMM_ERR_WORKSPACE
    assert _shared(L, **big, ws=P(8, 4)) == E.QMM_ERR_ALIGN
    assert _shared(L, n=0, Q=qmm.qmm_heads_desc(), lengths=NULL, ws=NULL) == E.QMM_OK


def test_attn_shared_workspace_sizes(L):
    W = L.qmm_attn_shared_workspace_bytes
    assert W(0, 100, 100, 4, 2, 64) == 0
    assert W(4, 500, 192, 32, 8, 128) == 0            # few keys: no partial results
    assert W(4, 0, 0, 32, 8, 128) == 0
    one = 4 * 129 * 48 * 32                           # one piece of 48 sequences and 32 heads of 128
    assert W(48, 32000, 0, 32, 8, 128) % one == 0 and 2 * one <= W(48, 32000, 0, 32, 8, 128) <= 64 * one
    for bad in ((-1, 1, 1, 4, 2, 64), (1, -1, 1, 4, 2, 64), (1, 1, -1, 4, 2, 64), (1, 1, 1, 4, 3, 64), (1, 1, 1, 4, 2, 65),
                (1, 1, 1, 0, 1, 64), (1 << 31, 1, 1, 1, 1, 64)):
        assert W(*bad) == qmm.QMM_ERR_SHAPE, bad


def test_binding_refuses_cpu_tensors():
    f = torch.zeros
    with pytest.raises(TypeError, match="GPU tensor"):
        qmm.qmm_lora(f(2, 32), f(1, 4, 32).half(), f(1, 8, 4).half(), f(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="GPU tensor"):
        qmm.qmm_norm_rope([qmm.qmm_head_part(f(2, 1, 64), f(2, 1, 64))])
    with pytest.raises(TypeError, match="GPU tensor"):
        qmm.qmm_attn_prompt(f(2, 1, 64).half(), f(2, 1, 64).half(), f(2, 1, 64).half(), f(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="GPU tensor"):
        qmm.qmm_attn_shared(f(2, 1, 64).half(), f(9, 1, 64).half(), f(9, 1, 64).half(), None, None, None)
    with pytest.raises(TypeError, match="GPU tensor"):
        qmm.qmm_lora(None, None, None, None)
    assert qmm.qmm_norm_rope([]) == []
    with pytest.raises(ValueError):
        qmm.qmm_norm_rope([qmm.qmm_head_part(None, None)] * 5)
    with pytest.raises(ValueError):
        qmm.qmm_norm_rope([qmm.qmm_head_part(None, None)], pairs="quarters")


# ---------------------------------------------- pins of the definitions

def test_attention_by_hand():
    # scores log 3 and 0 after scaling: weights 3/4 and 1/4
    q, k = np.array([2.0, 0.0]), np.array([[math.log(3.0), 5.0], [0.0, -7.0]])
    v = np.array([[4.0, 0.0], [0.0, 8.0]])
    o, err = O.attend(q, k, v, 0.5, "f16")
    assert np.allclose(o, [3.0, 2.0], rtol=1e-15) and (err > 0).all() and (err < 0.02).all()
    q3 = np.tile(q, (3, 2, 1))
    o, _ = O.attn_prompt(q3, np.stack([k, k, k])[:, :1], np.stack([v, v, v])[:, :1], [0, 1, 3], 0.5, "f16")
    assert np.allclose(o[0], v[0]) and np.allclose(o[1], v[0]) and np.allclose(o[2], v[0])  # equal keys
    o, _ = O.attn_shared(q[None, None], k[:1, None], v[:1, None], k[None, 1:, None], v[None, 1:, None], [1], 0.5, "f16")
    assert np.allclose(o[0, 0], [3.0, 2.0])
    o, _ = O.attn_shared(q[None, None], k[:1, None], v[:1, None], k[None, 1:, None], v[None, 1:, None], [0], 0.5, "f16")
    assert np.allclose(o[0, 0], v[0])
    o, _ = O.attn_shared(q[None, None], None, None, k[None, :, None], v[None, :, None], [0], 0.5, "f16")
    assert (o == 0).all()
    o, _ = O.attn_shared(q[None, None], None, None, k[None, :, None], v[None, :, None], [3], 0.5, "f16")
    assert np.isnan(o).all()


def test_rotation_and_norm_by_hand():
    x = np.array([[[3.0, 4.0, 1.0, 2.0]]])
    quarter = [math.pi / 2]
    y, _ = O.norm_rope(x, positions=np.array([1]), freqs=quarter, pairs="halves")
    assert np.allclose(y, [[[-4.0, 3.0, 1.0, 2.0]]])      # elements 0 and 1 = i and i + n_freqs
    y, _ = O.norm_rope(x, positions=np.array([2]), freqs=quarter, pairs="neighbours")
    assert np.allclose(y, [[[-3.0, -4.0, 1.0, 2.0]]])
    y, _ = O.norm_rope(x, positions=np.array([1]), freqs=[math.pi / 2, 0.0], pairs="halves")
    assert np.allclose(y, [[[-1.0, 4.0, 3.0, 2.0]]])
    y, _ = O.norm_rope(x, np.array([1.0, 2.0, 1.0, 1.0]), True, 0.0)
    assert np.allclose(y, x / math.sqrt(7.5) * [1, 2, 1, 1])


def test_adapters_by_hand():
    a = np.array([[[1.0, 2.0]], [[0.0, -1.0]]])       # two adapters of rank 1
    b = np.array([[[3.0]], [[5.0]]])
    y, err = O.lora(np.array([[1.0, 1.0]] * 4), a, b, [0, 1, -1, 2], np.array([1.0, 2.0]), np.full((4, 1), 10.0))
    assert y[0, 0] == 19.0 and y[1, 0] == 0.0 and y[2, 0] == 10.0 and np.isnan(y[3, 0]) and (err >= 0).all()


def test_the_bounds_catch_planted_mistakes():
    """A key left out, a wrong scale, a weight too many, a pair rotated the wrong way: all outside the bounds."""
    r = np.random.Generator(np.random.PCG64(5))
    q, k, v = r.standard_normal(64), r.standard_normal((50, 64)), r.standard_normal((50, 64))
    o, err = O.attend(q, k, v, 0.125, "bf16")
    for wrong in (O.attend(q, k[:-1], v[:-1], 0.125, "bf16")[0], O.attend(q, k, v, 0.13, "bf16")[0],
                  O.attend(q, np.vstack([k, k[:1]]), np.vstack([v, v[:1]]), 0.125, "bf16")[0]):
        assert (np.abs(wrong - o) > err).any()
    x = r.standard_normal((2, 1, 64))
    f = [10000.0 ** (-i / 32) for i in range(32)]
    y, err = O.norm_rope(x, None, True, 1e-6, np.array([3, 70000]), f, "halves", "bf16")
    for wrong in (O.norm_rope(x, None, True, 1e-6, np.array([-3, 70000]), f, "halves", "bf16")[0],
                  O.norm_rope(x, None, True, 1e-6, np.array([3, 70000]), f, "neighbours", "bf16")[0],
                  O.norm_rope(x, None, False, 1e-6, np.array([3, 70000]), f, "halves", "bf16")[0],
                  O.norm_rope(x, None, True, 1e-6, np.array([3, 70001]), f, "halves", "bf16")[0]):
        assert (np.abs(wrong - y) > err).any()
    x, a, b = r.standard_normal((1, 64)), r.standard_normal((2, 4, 64)), r.standard_normal((2, 8, 4))
    y, err = O.lora(x, a, b, [0])
    assert (np.abs(O.lora(x, a, b, [1])[0] - y) > err).all()
    assert (np.abs(O.lora(x, a[:, :3], b[:, :, :3], [0])[0] - y) > err).any()
