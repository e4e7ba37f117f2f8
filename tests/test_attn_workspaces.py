"""Workspaces kept for calls of different sizes (no GPU needed): what a call needs
may be more for a smaller batch, and the *_workspace_max_bytes functions bound it."""
import os
import random
import shutil
import subprocess

import pytest

import block_quantized_matmul_amd as qmm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_workspace_for_the_largest_batch_serves_smaller_ones():
    heads = [(32, 8, 128), (32, 8, 64), (8, 8, 64), (40, 1, 128), (33, 1, 64), (64, 2, 128), (1, 1, 64)]
    r = random.Random(3)
    for hq, hkv, dim in heads:
        need_of = {}
        for n in list(range(1, 130)) + [200, 255, 256, 257, 600, 1000, 4096]:
            most = qmm.qmm_attn_shared_workspace_max_bytes(n, hq, dim)
            assert most >= qmm.qmm_attn_shared_workspace_max_bytes(n - 1, hq, dim)
            for prefix, cap in ((0, 2048), (1, 2000), (500, 32000), (32000, 0), (32000, 2048), (16384, 16384), (1025, 1),
                                (1 << 30, 1 << 30), (r.randint(0, 70000), r.randint(0, 70000))):
                need = qmm.qmm_attn_shared_workspace_bytes(n, prefix, cap, hq, hkv, dim)
                assert 0 <= need <= most, (n, prefix, cap, hq, hkv, dim, need, most)
                need_of[n, prefix, cap] = need
        if (hq, hkv, dim) == (32, 8, 128):  # why: 32 sequences need more than 48
            assert need_of[32, 32000, 2048] > need_of[48, 32000, 2048]


def test_a_workspace_for_the_largest_token_count_serves_smaller_ones():
    for k in (32, 512, 4096, 8192, 8224, 11008, 131072, 200000, (1 << 24) - 32):
        for rank in (1, 16, 32, 33, 64, 256):
            for n in list(range(1, 700, 7)) + [511, 512, 513, 704, 705, 1024, 2048, 2049, 8192, 40000, (1 << 25) - 1]:
                most = qmm.qmm_lora_workspace_max_bytes(n, k, rank)
                need = qmm.qmm_lora_workspace_bytes(n, k - k % 32, rank)
                assert 0 < need <= most, (n, k, rank, need, most)
                assert most >= qmm.qmm_lora_workspace_max_bytes(n - 1, k, rank)
                assert most >= qmm.qmm_lora_workspace_max_bytes(n, max(32, k - 32), rank)
    assert qmm.qmm_lora_workspace_bytes(2048, 4096, 16) > qmm.qmm_lora_workspace_bytes(2049, 4096, 16)


def test_the_header_is_c_and_says_the_same(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lora = [(1, 32, 1), (512, 4096, 16), (513, 4096, 16), (513, 200000, 16), (40000, 11008, 64), (3, 8224, 256)]
    shared = [(1, 1, 64), (48, 32, 128), (4096, 33, 64)]
    lines = [f'printf("%lld\\n", (long long)qmm_lora_workspace_max_bytes({n}, {k}, {r}));' for n, k, r in lora]
    lines += [f'printf("%lld\\n", (long long)qmm_attn_shared_workspace_max_bytes({n}, {h}, {d}));' for n, h, d in shared]
    src, exe = tmp_path / "sizes.c", tmp_path / "sizes"
    src.write_text('#include <stdio.h>\n#include "qmm_attn.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0;\n}\n")
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == ([qmm.qmm_lora_workspace_max_bytes(*x) for x in lora]
                   + [qmm.qmm_attn_shared_workspace_max_bytes(*x) for x in shared])
