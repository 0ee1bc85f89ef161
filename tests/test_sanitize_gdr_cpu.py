"""Host-side AddressSanitizer + UndefinedBehaviorSanitizer run of the gated
delta rule's C-ABI layer (gdr_api.cpp as plain host C++, kernel launchers
stubbed out), through tests/sanitize/gdr_host_driver.cpp.  CPU only: no GPU
code is built with a sanitizer."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None
                    or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")),
                    reason="needs g++ and the ROCm headers")
def test_gdr_host_layer_under_asan_ubsan(tmp_path):
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-fno-omit-frame-pointer", "-g", "-O1"]
    csrc = os.path.join(ROOT, "gated_delta_rule_95_amd", "csrc")
    exe = tmp_path / "gdr_host_driver"
    cmd = ["g++", "-std=c++17", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROCM, "include"),
           "-I" + os.path.join(ROOT, "include"), "-I" + csrc, os.path.join(csrc, "gdr_api.cpp"),
           os.path.join(csrc, "kda_api.cpp"), os.path.join(ROOT, "tests", "sanitize", "gdr_host_driver.cpp"),
           "-o", str(exe), "-L" + os.path.join(ROCM, "lib"), "-lamdhip64",
           "-Wl,-rpath," + os.path.join(ROCM, "lib")] + san
    subprocess.run(cmd, check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "sanitized gated delta rule host checks passed" in r.stdout
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr
