"""Launch shapes of the cache and tree calls for every size the argument checks
let through (no GPU): under sanitizers with recorders in place of the launches,
and through the library, where a call that is too large has to be refused
before a launch."""
import ctypes
import os
import shutil
import subprocess

import pytest

from speculative_decoding_verify_dspk_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verify_dspk_amd", "csrc")
ROCM_INC = "/opt/rocm/include"
P, EUNSUPPORTED = 0x100000, -2


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM_INC), reason="needs g++ and the ROCm headers")
def test_launch_shapes_under_sanitizers(tmp_path):
    exe = tmp_path / "attn_launch_check"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INC, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(ROOT, "tests", "host_check", "attn_launch_check.cpp"), os.path.join(CSRC, "attn_api.cpp"),
           "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1"))
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "launch check ok" in r.stdout and "runtime error" not in r.stderr


@pytest.mark.parametrize("b,kv_heads,max_rows,total_rows", [
    (1, 1, (1 << 31) - 1, (1 << 31) - 1),          # the sum with a block's positions passes 32 bits
    (1, 1, 1 << 30, 1 << 30),                      # 2^24 workgroups of 256 threads
    (512, 8, 100000, 110000),                      # ragged: few rows, many that a request might have
])
def test_calls_past_one_launch_are_refused(b, kv_heads, max_rows, total_rows):
    L = binding.lib()
    c = binding.KVCacheDesc(kv_heads, 64, 64, 16, 1 << 20, P, 2 * P, None, None)
    B = binding.AttnBatchDesc(b, max_rows, total_rows, 4, 5 * P, 3 * P, 4 * P)
    prep = binding.QKPrepDesc(1e-6, None, None, None, 0, 0, None)
    ld = kv_heads * 64
    c, B, prep = (ctypes.byref(x) for x in (c, B, prep))
    if b == 1:                                     # without q the ragged call above still fits
        assert L.dspk_kv_append(c, B, P, ld, P, ld, 1, None) == EUNSUPPORTED
        assert L.dspk_kv_read(c, B, P, ld, P, ld, 1, None) == EUNSUPPORTED
    assert L.dspk_qkv_norm_rope_append(c, B, prep, P, 32 * 64, P, ld, P, ld, 1, 32, 2 * P, 32 * 64, None) == EUNSUPPORTED
    assert "too many rows" in L.dspk_last_error().decode()


def test_tree_calls_past_one_launch_are_refused():
    L = binding.lib()
    for b in (1 << 26, (1 << 31) - 1):
        assert L.dspk_tree_layout(P, b, 4, P, 2 * P, 3 * P, None) == EUNSUPPORTED
        assert L.dspk_accept_tree_greedy(P, P, P, b, 4, 2 * P, 3 * P, 4 * P, None) == EUNSUPPORTED
