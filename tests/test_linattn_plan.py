"""The launches of the attention calls at sizes up to their limits, on the host
(linear_attention_rnn_amd/csrc/linattn_plan.h), and the refusal of those that
no launch holds."""
import os
import shutil
import subprocess

import pytest

from linear_attention_rnn_amd import linattn, wkv6
from tests.test_linattn_abi import UNSUPPORTED, bwd, refused
from tests.test_linattn_sanitized import CSRC, HERE, ROCM, ROOT


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(f"{ROCM}/lib/libamdhip64.so"),
                    reason="needs g++ and the HIP runtime library")
def test_plans_under_asan_and_ubsan(tmp_path):
    exe = str(tmp_path / "linattn_plan_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{ROOT}/include", f"-I{CSRC}",
           *[os.path.join(HERE, f) for f in ("linattn_plan_driver.cpp", "linattn_stub.cpp", "kernel_stub.cpp")],
           *[os.path.join(CSRC, f) for f in ("linattn_api.cpp", "wkv6_api.cpp")],
           f"-L{ROCM}/lib", f"-Wl,-rpath,{ROCM}/lib", "-lamdhip64", "-lpthread", "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                         env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1", UBSAN_OPTIONS="print_stacktrace=1"))
    out = run.stdout + run.stderr
    assert run.returncode == 0 and "all plans hold" in out, out[-4000:]


@pytest.mark.skipif(not os.path.exists(wkv6.LIB_PATH), reason="libwkv6.so not built")
@pytest.mark.parametrize("kw", [dict(B=1398097, H=1), dict(B=2 ** 21, H=1, K=72, V=72), dict(B=1, H=2 ** 21, T=1000)])
def test_gradients_that_no_launch_holds_are_refused(kw):
    kw = dict(dict(T=1, K=128, V=128, dtype=0, grad=0, s_in=0, ds_out=0, ds_in=0), **kw)
    refused(bwd(**kw), UNSUPPORTED, "launch")
    assert linattn.lib().linattn_bwd_workspace_bytes(kw["B"], kw["T"], kw["H"], kw["K"], kw["V"], 0, 0, 0) == 0
