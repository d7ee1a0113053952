"""One workspace for 8-bit products and expert layers in turn: neither leaves anything in the
other's arrival counters."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from i8util import codes, dev, host, scales
from speculative_decoding_verify_dspk_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verify_dspk_amd", "csrc")
ROCM_INC = "/opt/rocm/include"
SPLIT = [(18, 130, 6500), (64, 130, 2100), (130, 1500, 9000), (200, 8200, 9000), (300, 640, 4000)]     # m, n, k


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM_INC), reason="needs g++ and the ROCm headers")
def test_sums_begin_behind_every_counter(tmp_path):
    exe = tmp_path / "buffer"
    cmd = ["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INC, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(ROOT, "tests", "host_check", "i8_buffer_check.cpp"), os.path.join(CSRC, "i8_api.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([str(exe)] + [str(v) for s in SPLIT for v in s], capture_output=True, text=True, timeout=60)
    counters, *plans = r.stdout.split("\n")[:-1]
    assert len(plans) == len(SPLIT)
    for shape, line in zip(SPLIT, plans):
        splits, sums = map(int, line.split())
        assert splits > 1 and sums >= int(counters), shape


@pytest.mark.gpu
def test_products_and_expert_layers_in_turn():
    import torch
    from test_gpu_moe import Layer
    # layers whose 16 columns of y are shared by several workgroups, and one without
    layers = [Layer(2048, 768, 16, 3, seed=1), Layer(2048, 2048, 9, 16, seed=2), Layer(512, 96, 32, 17, seed=3)]
    tops = [8, 1, 8]
    need = max([binding.i8_workspace_bytes(n, k, m) for m, n, k in SPLIT] +
               [binding.moe_workspace_bytes(L.hidden, L.inter, L.experts, L.m, top) for L, top in zip(layers, tops)])
    ws, rng = binding.alloc_workspace(need), np.random.default_rng(0)
    products = []
    for m, n, k in SPLIT:
        c, s, w, sw = codes(rng, m, k), scales(rng, m), codes(rng, n, k), scales(rng, n)
        x = torch.zeros(m, -(-k // 16) * 16, dtype=torch.int8, device="cuda")
        x[:, :k] = dev(c)
        W, want, y = binding.Int8Weight(dev(w), dev(sw)), torch.zeros(m, n, device="cuda"), torch.zeros(m, n, device="cuda")
        binding.i8_gemm(W, x, dev(s), m, want)                       # without a workspace: one workgroup per sum
        products.append((W, x, dev(s), m, y, want))
    choices = [L.choice(top) for L, top in zip(layers, tops)]
    wants = [L.run(*choice) for L, choice in zip(layers, choices)]   # with workspaces of their own
    for turn in range(3):
        for i, (W, x, s, m, y, want) in enumerate(products):
            y.zero_()
            binding.i8_gemm(W, x, s, m, y, ws)
            L, choice = layers[(i + turn) % 3], choices[(i + turn) % 3]
            assert np.array_equal(L.run(*choice, ws=ws), wants[(i + turn) % 3])
            assert torch.equal(y, want)
            assert not ws[:6400].any(), "counters left"
    torch.cuda.synchronize()
    assert host(ws[:6400]).sum() == 0


def test_the_largest_over_every_call_is_what_a_buffer_needs():
    """Fewer rows may need more, for products and for expert layers: a buffer of the largest
    m's size is refused for a smaller one, which names the size it needs."""
    lib, P, n, k = binding.lib(), 0x100000, 2560, 4096
    sizes = {m: binding.i8_workspace_bytes(n, k, m) for m in range(1, 600)}
    most = max(sizes, key=sizes.get)
    assert sizes[most] > sizes[599]
    w = binding.Int8WeightDesc(n, k, 1, P, P)
    got = lib.dspk_i8_gemm(ctypes.byref(w), P, k, P, most, P, 0, n, P, sizes[599], None)
    assert got == -1 and f"workspace of {sizes[most]} bytes" in lib.dspk_last_error().decode()
    assert binding.moe_workspace_bytes(2048, 768, 128, 16, 32) > binding.moe_workspace_bytes(2048, 768, 128, 17, 32)
