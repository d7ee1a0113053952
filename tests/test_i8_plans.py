"""Every kernel that the products of 8-bit rows can take: sizes that reach each of
them, checked on the host, and their results to the bit."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from i8util import bf16, codes, dev, host, scales

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verify_dspk_amd", "csrc")
ROCM_INC = "/opt/rocm/include"

# (m, n, k): kernel, whether K is split, and of 256 x 256 tiles whether some are whole (1)
# or in quarters (2)
PLANS = {(7, 130, 300): (0, False, 0), (5, 4112, 96): (1, False, 0), (18, 130, 150): (2, False, 0),
         (18, 4100, 150): (3, False, 0), (40, 130, 150): (4, False, 0), (40, 4100, 150): (5, False, 0),
         (31, 8200, 1100): (6, False, 0), (18, 130, 6500): (6, True, 0), (130, 130, 150): (7, False, 0),
         (64, 130, 2100): (7, True, 0), (200, 4100, 150): (8, False, 0), (130, 1500, 9000): (8, True, 0),
         (1560, 2570, 150): (9, False, 0), (200, 8200, 9000): (9, True, 0), (390, 20500, 300): (10, False, 1),
         (200, 8200, 4200): (10, False, 2), (1560, 10300, 150): (10, False, 3)}


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM_INC), reason="needs g++ and the ROCm headers")
def test_sizes_reach_every_kernel(tmp_path):
    exe = tmp_path / "plans"
    cmd = ["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INC, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(ROOT, "tests", "host_check", "i8_plan_check.cpp"), os.path.join(CSRC, "i8_api.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([str(exe)] + [str(v) for shape in PLANS for v in shape], capture_output=True, text=True, timeout=60)
    got = {}
    for shape, line in zip(PLANS, r.stdout.split("\n")):
        kind, splits, whole, groups = map(int, line.split())
        got[shape] = kind, splits > 1, (whole > 0) + 2 * (groups > whole) if kind == 10 else 0
    assert got == PLANS
    assert {p[0] for p in PLANS.values()} == set(range(11))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", list(PLANS))
def test_every_kernel(m, n, k):
    import torch

    from speculative_decoding_verify_dspk_amd import binding
    rng = np.random.default_rng(m + n + k)
    c, s, w, ws = codes(rng, m, k), scales(rng, m), codes(rng, n, k), scales(rng, n)
    x = torch.full((m, -(-k // 16) * 16 + 32), -77, dtype=torch.int8, device="cuda")
    x[:, :k] = dev(c)
    # |sums| <= 13000 * 2^14 < 2^53: exact in fp64, in any order
    want = (c.astype(np.float64) @ w.astype(np.float64).T).astype(np.float32) * s[:, None] * ws[None]
    y = torch.full((m + 1, n + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    work = binding.alloc_workspace(binding.i8_workspace_bytes(n, k, m))
    W = binding.Int8Weight(dev(w), dev(ws))
    for _ in range(2):
        y[:m, :n] = 0
        binding.i8_gemm(W, x[:, :k], dev(s), m, y, work)
        got = host(y)
        assert np.array_equal(got[:m, :n], bf16(want))
        assert (got[m] == 7).all() and (got[:m, n:] == 7).all()
    assert not work[:4096].any(), "arrivals left"
