"""The host code of the bf16 expert products, the gradient clipping and the single-token products under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): the library's sources compiled as for gfx950 with both
sanitizers on the host pass, and random and limit-value arguments from tests/experts_abi_fuzz.c."""
from __future__ import annotations

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests.test_host_sanitizers import COMMON, CSRC, HIPCC, ROCM_INCLUDE, ROOT, SAN, SOURCES

EXPERTS_SOURCES = SOURCES + ["experts_api.hip", "bf16_gemm.hip", "grad_clip.hip", "gemv_nvfp4.hip"]


def test_experts_abi_validation_is_clean_under_asan_and_ubsan(tmp_path):
    if not os.path.exists(HIPCC) or shutil.which("gcc") is None:
        pytest.skip("hipcc or gcc not available")

    def run(*cmd, **kw):
        r = subprocess.run(list(cmd), capture_output=True, text=True, **kw)
        assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-3000:])
        return r.stdout

    def compile_one(src):
        obj = str(tmp_path / (os.path.splitext(src)[0] + ".o"))
        run(HIPCC, *COMMON, *SAN, "-c", os.path.join(CSRC, src), "-o", obj)
        return obj

    with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, EXPERTS_SOURCES))
    drv, exe = str(tmp_path / "fuzz.o"), str(tmp_path / "fuzz")
    run(HIPCC, "-x", "c", "-std=c11", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", ROCM_INCLUDE,
        *SAN, "-c", os.path.join(ROOT, "tests", "experts_abi_fuzz.c"), "-o", drv)
    run(HIPCC, "--offload-arch=gfx950", *SAN, *objs, drv, "-o", exe)
    out = run(exe, "30000", env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
                                     UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1"), timeout=600)
    assert out.startswith("ok "), out
