"""The serving operators' C-ABI layer (serve_api.cpp: argument checks and dispatch) built for the host with
AddressSanitizer and UndefinedBehaviorSanitizer and driven on the CPU, with host stand-ins for the HIP runtime and the
kernel launchers as in test_host_sanitizers.py.  Device code is not part of this build."""

import os
import shutil
import subprocess

import pytest

from tests.test_host_sanitizers import CSRC, ROOT, SAN

SOURCES = [os.path.join(CSRC, "api.cpp"), os.path.join(CSRC, "workspace.cpp"), os.path.join(CSRC, "serve_api.cpp"),
           os.path.join(SAN, "hip_stub.cpp"), os.path.join(SAN, "kernel_stub.cpp"),
           os.path.join(SAN, "serve_kernel_stub.cpp"), os.path.join(SAN, "serve_driver.cpp")]


def test_serving_c_abi_layer_under_asan_and_ubsan(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.isdir("/opt/rocm/include/hip"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = str(tmp_path / "serve_sanitize")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, *SOURCES, "-o", exe, "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, f"sanitizer build failed:\n{' '.join(cmd)}\n{r.stderr[-4000:]}"
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-6000:]
    assert "serve sanitize driver: ok" in r.stdout
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out[-6000:]
