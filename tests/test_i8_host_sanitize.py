"""The 8-bit side's host code (argument checks, launch plans, workspace carving)
under AddressSanitizer and UndefinedBehaviorSanitizer, with recorders in place of the
kernel launches (no GPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verify_dspk_amd", "csrc")
ROCM_INC = "/opt/rocm/include"


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM_INC), reason="needs g++ and the ROCm headers")
def test_8bit_host_code_under_sanitizers(tmp_path):
    exe = tmp_path / "i8_host_check"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INC, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(ROOT, "tests", "host_check", "i8_host_check.cpp"), os.path.join(CSRC, "i8_api.cpp"),
           "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1"))
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "host check ok" in r.stdout and "runtime error" not in r.stderr
