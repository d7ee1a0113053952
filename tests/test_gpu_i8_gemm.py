"""Products of 8-bit rows with 8-bit weights: the bits of the definition in fp32."""
import numpy as np
import pytest

from i8util import bf16, codes, dev, host, scales
from oracle import layer8
from speculative_decoding_verify_dspk_amd import binding

pytestmark = pytest.mark.gpu


def _x(rng, m, k, pad=0):
    """Codes in rows whose padding is poison, and their scales."""
    import torch
    c, s = codes(rng, m, k), scales(rng, m)
    t = torch.full((m, -(-k // 16) * 16 + 16 * pad), -77, dtype=torch.int8, device="cuda")
    t[:, :k] = dev(c)
    return c, s, t[:, :k], dev(s)


def _want(c, s, w, ws):
    """float(sum) * x_scale * w_scale, each step in fp32."""
    return layer8.sums(c, w).astype(np.float32) * s[:, None] * ws[None]


def _workspace(n, k, m):
    return binding.alloc_workspace(binding.i8_workspace_bytes(n, k, m))


SHAPES = [(1, 1, 1), (1, 16, 64), (2, 17, 65), (3, 5, 130), (16, 48, 200), (17, 33, 777), (32, 160, 1024), (33, 100, 63),
          (64, 64, 640), (65, 31, 128), (100, 257, 321), (128, 128, 128), (129, 300, 513), (200, 1000, 95),
          (257, 520, 1100), (300, 129, 2049), (513, 640, 256), (1, 2560, 9728), (6, 2560, 9728), (1030, 700, 300),
          (20, 2570, 9999), (50, 2560, 9728), (100, 1000, 9000), (260, 500, 8200), (700, 999, 5000), (777, 4100, 777)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_product_is_the_definitions_bits(m, n, k, kind):
    import torch
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    c, s, x, sd = _x(rng, m, k, pad=m % 3)
    w, ws = codes(rng, n, k), scales(rng, n)
    W = binding.Int8Weight(dev(w), dev(ws))
    want = _want(c, s, w, ws)
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    ld = n + (m + n) % 5                              # odd leading dimensions among them
    for work in (None, _workspace(n, k, m)):
        y = torch.full((m + 1, ld), 7.0, dtype=dt, device="cuda")
        binding.i8_gemm(W, x, sd, m, y, work)
        got = host(y)
        assert np.array_equal(got[:m, :n], want if kind == "f32" else bf16(want))
        assert (got[m] == 7).all() and (got[:m, n:] == 7).all()
    assert not work[:4096].any(), "arrivals left"


@pytest.mark.parametrize("n,k", [(300, 1000), (2560, 2560), (640, 20000)])
def test_a_rows_bits_do_not_depend_on_the_rows_beside_it(n, k):
    """What makes a verify pass exact: the same row alone, in a round, and in a prompt."""
    import torch
    rng = np.random.default_rng(k)
    m = 600
    c, s, x, sd = _x(rng, m, k)
    W = binding.Int8Weight(dev(codes(rng, n, k)), dev(scales(rng, n)))
    whole = torch.empty(m, n, device="cuda")
    binding.i8_gemm(W, x, sd, m, whole, _workspace(n, k, m))
    for take in (1, 5, 16, 17, 32, 33, 64, 65, 128, 200, 400):
        for work in (None, _workspace(n, k, take)):
            y = torch.empty(take, n, device="cuda")
            binding.i8_gemm(W, x[100:], sd[100:], take, y, work)
            assert torch.equal(y, whole[100:100 + take]), take


def test_largest_sums():
    """The longest K at the extreme codes: sums next to 2^31."""
    import torch
    k, m, n = 131071, 18, 20
    for a, b in ((-128, -128), (-128, 127), (127, 127)):
        x = torch.full((m, -(-k // 16) * 16), a, dtype=torch.int8, device="cuda")[:, :k]
        W = binding.Int8Weight(torch.full((n, k), b, dtype=torch.int8, device="cuda"), torch.ones(n, device="cuda"))
        for take in (1, m):
            y = torch.empty(take, n, device="cuda")
            binding.i8_gemm(W, x, torch.ones(m, device="cuda"), take, y, _workspace(n, k, take))
            assert (y == float(np.float32(a * b * k))).all()


def test_rows_without_a_scale_stay_alone():
    import torch
    rng = np.random.default_rng(0)
    for m in (5, 40, 300):
        c, s, x, sd = _x(rng, m, 320)
        w, ws = codes(rng, 70, 320), scales(rng, 70)
        sd[2], ws[9] = float("nan"), np.inf
        y = torch.empty(m, 70, device="cuda")
        binding.i8_gemm(binding.Int8Weight(dev(w), dev(ws)), x, sd, m, y)
        got = host(y)
        assert np.isnan(got[2]).all()
        ok = np.delete(np.delete(got, 2, 0), 9, 1)
        assert np.array_equal(ok, np.delete(np.delete(_want(c, s, w, ws), 2, 0), 9, 1))


def test_packing_of_slices_and_several_weights():
    """A weight's codes at any address and leading dimension; several weights in one call."""
    import torch
    rng = np.random.default_rng(4)
    big = codes(rng, 50, 333)
    d = dev(big)
    c, s, x, sd = _x(rng, 7, 300)
    ws = scales(rng, 40)
    W = binding.Int8Weight(d[7:47, 13:313], dev(ws))
    y = torch.empty(7, 40, device="cuda")
    binding.i8_gemm(W, x, sd, 7, y)
    assert np.array_equal(host(y), _want(c, s, big[7:47, 13:313], ws))
    three, sc = codes(rng, 3, 35, 90), scales(rng, 3, 35)
    W = binding.Int8Weight(dev(three), dev(sc))
    assert W.count == 3 and W.tiles.numel() == binding.i8_tiled_bytes(35, 90, 3)
    t = W.tiles.cpu().numpy().view(np.int8).reshape(3, 3, 2, 4, 16, 16)
    for g in range(3):
        for col in range(48):
            for r in range(128):
                want = three[g, col, r] if col < 35 and r < 90 else 0
                assert t[g, col // 16, r // 64, r % 64 // 16, col % 16, r % 16] == want


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_weights_from_rows(kind):
    import torch
    from oracle import attention as oa
    w = np.random.default_rng(2).normal(0, 0.05, (3, 50, 70)).astype(np.float32)
    w = w if kind == "f32" else bf16(w)
    t = torch.zeros(150, 80, dtype=torch.float32 if kind == "f32" else torch.bfloat16, device="cuda")
    t[:, :70] = dev(w.reshape(150, 70))
    one = binding.Int8Weight.quantize(t[:50, :70])
    code, scale = oa.quantise_rows(w[0])
    assert np.array_equal(host(one.scales), scale)
    c, s, x, sd = _x(np.random.default_rng(3), 4, 70)
    y = torch.empty(4, 50, device="cuda")
    binding.i8_gemm(one, x, sd, 4, y)
    assert np.array_equal(host(y), _want(c, s, code, scale))


def test_calls_in_a_graph_and_on_two_streams():
    """Captured and replayed with eager calls between, and two streams at once with a workspace each."""
    import torch
    rng = np.random.default_rng(6)
    n, k = 640, 4000
    W = binding.Int8Weight(dev(codes(rng, n, k)), dev(scales(rng, n)))
    for m in (3, 150, 300):
        c, s, x, sd = _x(rng, m, k)
        want = torch.empty(m, n, device="cuda")
        binding.i8_gemm(W, x, sd, m, want, _workspace(n, k, m))
        y, work = torch.zeros(m, n, device="cuda"), _workspace(n, k, m)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.i8_gemm(W, x, sd, m, y, work)
        for _ in range(3):
            y.zero_()
            g.replay()
            assert torch.equal(y, want)
            binding.i8_gemm(W, x, sd, m, y, work)
            torch.cuda.synchronize()
            assert torch.equal(y, want)
        sides = [torch.cuda.Stream() for _ in range(2)]
        outs, spaces = [torch.zeros_like(want) for _ in sides], [_workspace(n, k, m) for _ in sides]
        torch.cuda.synchronize()
        for _ in range(10):
            for st, o, sp in zip(sides, outs, spaces):
                binding.i8_gemm(W, x, sd, m, o, sp, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


def test_one_workspace_serves_calls_of_all_sizes():
    import torch
    rng = np.random.default_rng(8)
    sizes = [(300, 640, 4000), (40, 16, 9000), (130, 300, 640), (1, 2560, 512), (700, 130, 2000)]
    work = binding.alloc_workspace(max(binding.i8_workspace_bytes(n, k, m) for m, n, k in sizes))
    for turn in range(2):
        for m, n, k in sizes:
            c, s, x, sd = _x(rng, m, k)
            w, ws = codes(rng, n, k), scales(rng, n)
            y = torch.empty(m, n, device="cuda")
            binding.i8_gemm(binding.Int8Weight(dev(w), dev(ws)), x, sd, m, y, work)
            assert np.array_equal(host(y), _want(c, s, w, ws)), (turn, m, n, k)


def test_no_rows():
    import torch
    W = binding.Int8Weight(torch.ones(20, 70, dtype=torch.int8, device="cuda"), torch.ones(20, device="cuda"))
    binding.i8_gemm(W, torch.zeros(0, 80, dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda"), 0,
                    torch.zeros(0, 20, device="cuda"))
