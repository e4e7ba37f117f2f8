"""The host code of include/qmm_serve.h's entry points under AddressSanitizer
and UndefinedBehaviorSanitizer, built and run as tests/test_host_sanitizers.py
does for the rest of the library (whose objects it links, for the block types'
sizes): tests/host_sanitize/serve_abi_driver.cpp calls every entry point with
invalid and extreme arguments, and nothing is launched.
"""
import hashlib
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

import test_host_sanitizers as base
from test_host_sanitizers import CSRC, FLAGS, INCLUDE, ROOT, SAN, _hipcc, _run

DRIVER = os.path.join(ROOT, "tests", "host_sanitize", "serve_abi_driver.cpp")
BUILD = os.path.join(ROOT, "tests", "host_sanitize", "_build", "serve")
SOURCES = ["serve_api", "kv4", "attn_kv4", "moe", "sample"]


def _build(hipcc):
    base._build(hipcc)
    os.makedirs(BUILD, exist_ok=True)
    h = hashlib.sha256(" ".join(FLAGS).encode())
    for path in ([os.path.join(CSRC, x) for x in sorted(os.listdir(CSRC)) if x.endswith((".hip", ".h"))]
                 + [os.path.join(INCLUDE, x) for x in ("qmm.h", "qmm_attn.h", "qmm_serve.h")] + [DRIVER]):
        h.update(open(path, "rb").read())
    stamp, exe = os.path.join(BUILD, "inputs.sha256"), os.path.join(BUILD, "driver")
    if os.path.exists(exe) and os.path.exists(stamp) and open(stamp).read() == h.hexdigest():
        return exe
    objs = [os.path.join(BUILD, s + ".o") for s in SOURCES]
    jobs = [[hipcc, *FLAGS, "-c", os.path.join(CSRC, s + ".hip"), "-o", o] for s, o in zip(SOURCES, objs)]
    drv = os.path.join(BUILD, "driver.o")
    jobs.append([hipcc, *FLAGS, "-x", "c++", "-c", DRIVER, "-o", drv])
    with ThreadPoolExecutor(min(len(jobs), os.cpu_count() or 1)) as ex:
        list(ex.map(_run, jobs))
    _run([hipcc, "--offload-arch=gfx950", *SAN, drv, *objs, *[os.path.join(base.BUILD, s + ".o") for s in base.SOURCES],
          "-o", exe])
    with open(stamp, "w") as f:
        f.write(h.hexdigest())
    return exe


def test_abi_checks_under_host_sanitizers():
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not found")
    exe = _build(hipcc)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert res.returncode == 0, f"driver failed ({res.returncode}):\n{res.stdout}\n{res.stderr[-6000:]}"
    assert "abi checks ok" in res.stdout
