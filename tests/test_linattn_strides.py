"""Distances between rows at the limits of what the kernels reach, and tables that
start at any element: the argument checks of linattn.h on the host, with kernels
replaced by stubs."""
import os
import shutil
import subprocess

import pytest

from tests.test_linattn_sanitized import CSRC, HERE, ROCM, ROOT

pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(f"{ROCM}/lib/libamdhip64.so"),
                                reason="needs g++ and the HIP runtime library")


def test_distances_under_asan_and_ubsan(tmp_path):
    exe = str(tmp_path / "linattn_strides_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{ROOT}/include", f"-I{CSRC}",
           *[os.path.join(HERE, f) for f in ("linattn_strides_driver.cpp", "linattn_stub.cpp", "kernel_stub.cpp")],
           *[os.path.join(CSRC, f) for f in ("linattn_api.cpp", "wkv6_api.cpp")],
           f"-L{ROCM}/lib", f"-Wl,-rpath,{ROCM}/lib", "-lamdhip64", "-lpthread", "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                         env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1", UBSAN_OPTIONS="print_stacktrace=1"))
    out = run.stdout + run.stderr
    assert run.returncode == 0 and "all distances hold" in out, out[-4000:]
