"""The size limits that include/qmm_attn.h states, at the limits (no GPU needed:
what is within them is stopped by a missing workspace or pointer)."""
import ctypes

import pytest

import block_quantized_matmul_amd as qmm

NULL = ctypes.c_void_p(0)


def P(i):
    return ctypes.c_void_p(0x100000 * i)


@pytest.fixture(scope="module")
def L():
    qmm.qmm_lora_workspace_bytes(1, 32, 1)  # declares the argument types
    return qmm.lib()


def _heads(heads, dim=64):
    return qmm.qmm_heads_desc(0x100000, 1 << 22, heads * dim, dim)


def _shared(L, n, hq, hkv, prefix, cap):
    kv = _heads(hkv)
    return L.qmm_attn_shared(1, _heads(hq), kv, kv, prefix, kv, kv, cap, P(2), _heads(hq), n, hq, hkv, 64, 0.125, NULL, 0,
                             NULL)


def test_shared_takes_up_to_2_22_rows(L):
    for hq, hkv in ((1, 1), (2, 2), (8, 8), (8, 1), (64, 2), (1 << 10, 1), (1 << 10, 1 << 10)):
        n = (1 << 22) // hq
        for prefix, cap in ((1 << 30, 1 << 30), ((1 << 31) - (1 << 20) - 1, 0), (2000, 1), (1, 2000)):
            assert qmm.qmm_attn_shared_workspace_bytes(n, prefix, cap, hq, hkv, 64) > 0, (n, hq, hkv, prefix, cap)
            assert _shared(L, n, hq, hkv, prefix, cap) == qmm.QMM_ERR_WORKSPACE, (n, hq, hkv, prefix, cap)
        assert _shared(L, (1 << 24) // hq, hq, hkv, 2000, 2000) == qmm.QMM_ERR_SHAPE
        assert _shared(L, n, hq, hkv, (1 << 31) - (1 << 20), 0) == qmm.QMM_ERR_SHAPE
    # 2^23 rows of one kind of piece each, one workgroup a row: too many for a launch
    assert _shared(L, 1 << 22, 2, 2, 2000, 2000) == qmm.QMM_ERR_SHAPE


def test_prompt_workgroups(L):
    def prompt(n, seqs, hq, hkv, starts=P(2)):
        return L.qmm_attn_prompt(1, _heads(hq), _heads(hkv), _heads(hkv), _heads(hq), n, hq, hkv, 64, starts, seqs, 0.125,
                                 NULL)

    # (n group / 128 + min(seqs, n)) hkv of 2^24 and, where the starts are missing, of less
    for n, seqs, hq, hkv in ((1 << 24, 1 << 24, 1, 1), (1 << 20, 1 << 20, 16, 16), (1 << 23, 1 << 23, 32, 2)):
        assert prompt(n, seqs, hq, hkv) == qmm.QMM_ERR_SHAPE, (n, seqs, hq, hkv)
        assert prompt(n, 1, hq, hkv, starts=NULL) == qmm.QMM_ERR_NULL


def test_norm_rope_heads(L):
    def rope(heads, X=0x100000):
        part = qmm.qmm_head_part_desc(X=X, x_type=0, x_token_stride=0, x_head_stride=0, Y=0x200000, y_type=0,
                                      y_row_stride=heads * 64, y_head_stride=64, n_heads=heads, norm=1)
        return L.qmm_norm_rope(ctypes.byref(part), 1, 5, 64, 1e-6, NULL, None, 0, 0, NULL, 0, NULL)

    assert rope((1 << 24) + 1) == qmm.QMM_ERR_SHAPE
    assert rope(1 << 24, X=None) == qmm.QMM_ERR_NULL
