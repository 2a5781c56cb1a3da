"""The host code of the expert, gated activation and grouped weight-gradient entry
points under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only; device code
is built as usual): extreme sizes, strides and leading dimensions."""

import concurrent.futures
import os
import subprocess

import pytest

from blockwise_scaled_fp8_amd import build
from tests.test_abi_sanitizers import CLANGXX, CSRC, HIPCC, HOST_ONLY_SANITIZE, INCLUDE, LIB_FLAGS, ROCM, ROOT, _run


def test_expert_entry_points_under_asan_and_ubsan(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)):
        pytest.skip("hipcc / clang++ not installed")
    cmds = [[HIPCC, *LIB_FLAGS, "-x", "hip", "-c", os.path.join(CSRC, s), "-o", str(tmp_path / (s + ".o"))]
            for s in build.SOURCES]
    cmds.append([CLANGXX, "-O1", "-g", "-std=c++17", *HOST_ONLY_SANITIZE, "-D__HIP_PLATFORM_AMD__",
                 "-I", os.path.join(ROCM, "include"), "-I", INCLUDE, "-c",
                 os.path.join(ROOT, "tests", "moe_abi_sanitize_driver.cpp"), "-o", str(tmp_path / "driver.o")])
    with concurrent.futures.ThreadPoolExecutor(max_workers=4) as ex:
        list(ex.map(_run, cmds))
    exe = tmp_path / "driver"
    _run([CLANGXX, *HOST_ONLY_SANITIZE, str(tmp_path / "driver.o"), *[str(tmp_path / (s + ".o")) for s in build.SOURCES],
          "-L", os.path.join(ROCM, "lib"), "-lamdhip64", f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}", "-lpthread",
          "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600,
                       env={**os.environ, "ASAN_OPTIONS": "halt_on_error=1", "UBSAN_OPTIONS": "halt_on_error=1"})
    if r.returncode == 77:
        pytest.skip(r.stdout.strip())
    report = r.stdout + r.stderr
    assert "Sanitizer" not in report and "runtime error" not in report, report[-6000:]
    assert r.returncode == 0 and " 0 failures" in r.stdout, report[-6000:]
