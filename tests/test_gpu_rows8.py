"""Norm with the residual's addition, activation, and rows to 8 bits and back,
against fp64 on the same inputs."""
import numpy as np
import pytest

from i8util import BF16, F32, assert_codes, bf16, blank, host, padding_kept, rows
from oracle import attention as oa
from oracle import layer8
from speculative_decoding_verify_dspk_amd import binding

pytestmark = pytest.mark.gpu

# Relative error of y in fp32.  norm: s is one sum (1 rounding, twice in y: in s and
# in the mean, where it counts half); the squares are added by at most 32 terms in a
# lane, 6 + 4 steps over lanes and waves (one rounding each, and one of each
# square), all positive, halved by the root; then mean, eps, root, reciprocal and
# the two products of y: 1 + 0.5 + (32 + 10 + 1) / 2 + 7 < 32 roundings.
NORM = 32 * F32
# silu: exp by the hardware's power of 2, off by a step (two half steps), and the
# correction of its argument (1); 1 + exp (1); the hardware's reciprocal, off by a step
# (2); the products with gate and up (2).
SILU = 8 * F32


def far_below(gate, up):
    """exp(-gate) passes fp32's largest number, below 2^128, for gates under -88.7, and the
    activation is -0 there instead of gate * exp(gate) * up with exp(gate) < 2^-127.96; a
    quotient below 2^-126 is off by half of 2^-149 times up, less than the difference to 2^-127."""
    return 2.0 ** -127 * np.abs(np.asarray(gate, np.float64) * up)

SHAPES = [(1, 1), (1, 2560), (2, 7), (3, 8), (5, 64), (4, 511), (6, 520), (3, 4097), (2, 8193), (2, 16390), (1, 32768),
          (700, 129), (1100, 2048)]


def _types(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _values(rng, m, n, kind, std=1.0):
    x = rng.normal(0, std, (m, n)).astype(np.float32)
    x[:, ::37] *= 20                                # a few far columns, as in a residual stream
    return x if kind == "f32" else bf16(x)


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("xt,rt", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_norm_with_residual(m, n, xt, rt):
    import torch
    rng = np.random.default_rng(m * 40000 + n)
    x, r = _values(rng, m, n, xt), _values(rng, m, n, rt, 3.0)
    w = rng.normal(1, 0.3, n).astype(np.float32)
    xd, rd = rows(x, _types(xt), 1), rows(r, _types(rt), 2)
    ro, out = blank(m, n, _types(rt)), blank(m, n, torch.bfloat16, 1)
    c8, sc = blank(m, n, torch.int8), torch.zeros(m, device="cuda")
    binding.add_rmsnorm(xd, rd, ro, torch.from_numpy(w).cuda(), m, n, eps=1e-5, out=out, codes=c8, scales=sc)
    torch.cuda.synchronize()
    s, y = layer8.add_rmsnorm(x, r, w, 1e-5)
    assert (np.abs(host(ro) - s) <= (F32 if rt == "f32" else F32 + BF16) * np.abs(s)).all()
    assert (np.abs(host(out) - y) <= (NORM + BF16) * np.abs(y) + 1e-38).all()
    assert_codes(host(c8), host(sc), y, NORM, f"{m}x{n}")
    for t in (xd, rd, ro, out, c8):
        assert padding_kept(t)
    # one output alone is the same
    only, c2, s2 = blank(m, n, torch.bfloat16), blank(m, n, torch.int8), torch.zeros(m, device="cuda")
    binding.add_rmsnorm(xd, rd, None, torch.from_numpy(w).cuda(), m, n, eps=1e-5, out=only)
    binding.add_rmsnorm(xd, rd, None, torch.from_numpy(w).cuda(), m, n, eps=1e-5, codes=c2, scales=s2)
    assert torch.equal(only, out) and torch.equal(c2, c8) and torch.equal(s2, sc)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_norm_parts_may_be_left_out_and_sums_stored_in_place(kind):
    import torch
    rng, m, n, dt = np.random.default_rng(3), 9, 300, _types(kind)
    x, r = _values(rng, m, n, kind), _values(rng, m, n, kind)
    xd, rd, out = rows(x, dt), rows(r, dt), blank(m, n, torch.bfloat16)
    for a, b in ((x, None), (None, r)):
        y = layer8.add_rmsnorm(a, b, None, 0.0)[1]
        keep = blank(m, n, dt)
        binding.add_rmsnorm(None if a is None else xd, None if b is None else rd, keep, None, m, n, eps=0.0, out=out)
        assert (np.abs(host(out) - y) <= (NORM + BF16) * np.abs(y)).all()
        assert np.array_equal(host(keep), x if b is None else r)
    want = blank(m, n, dt)
    binding.add_rmsnorm(xd, rd, want, None, m, n, out=out)
    for at in (xd, rd):                             # the sum over either of its parts
        a, b = xd.clone(), rd.clone()
        a, b = rows(x, dt), rows(r, dt)
        place = a if at is xd else b
        other = blank(m, n, torch.bfloat16)
        binding.add_rmsnorm(a, b, place, None, m, n, out=other)
        assert torch.equal(place, want) and torch.equal(other, out) and padding_kept(place)


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_activation(m, n, kind):
    import torch
    rng = np.random.default_rng(n)
    g, u = _values(rng, m, n, kind, 2.0), _values(rng, m, n, kind)
    out, c8, sc = blank(m, n, torch.bfloat16), blank(m, n, torch.int8, 1), torch.zeros(m, device="cuda")
    binding.silu_mul(rows(g, _types(kind)), rows(u, _types(kind), 1), m, n, out=out, codes=c8, scales=sc)
    y = layer8.silu_mul(g, u)
    assert (np.abs(host(out) - y) <= (SILU + BF16) * np.abs(y) + far_below(g, u) + 1e-38).all()
    assert_codes(host(c8), host(sc), y, SILU, f"{m}x{n}")
    assert padding_kept(out) and padding_kept(c8)


def test_activation_of_two_ranges_of_one_array_and_of_far_values():
    import torch
    f = 136
    both = torch.empty(3, 2 * f, dtype=torch.bfloat16, device="cuda").normal_()
    both[0, :4] = torch.tensor([-200.0, 200.0, -3e38, 3e38])
    both[0, f:f + 4] = 1.0
    out = blank(3, f, torch.bfloat16)
    binding.silu_mul(both[:, :f], both[:, f:], 3, f, out=out)
    g, u = host(both[:, :f]), host(both[:, f:])
    y = layer8.silu_mul(g, u)
    assert (np.abs(host(out) - y) <= (SILU + BF16) * np.abs(y) + far_below(g, u) + 1e-38).all()


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_rows_to_codes_and_back(m, n, kind):
    """The codes are the rule's in fp32, bit for bit, and what is read is scale * code."""
    import torch
    x = _values(np.random.default_rng(n + m), m, n, kind)
    c8, sc = blank(m, n, torch.int8, 1), torch.zeros(m, device="cuda")
    binding.i8_quantize(rows(x, _types(kind), 1), m, n, c8, sc)
    code, scale = oa.quantise_rows(x)
    assert np.array_equal(host(c8), code) and np.array_equal(host(sc), scale) and padding_kept(c8)
    value = scale[:, None] * code.astype(np.float32)
    for t in ("f32", "bf16"):
        y = blank(m, n, _types(t), 1)
        binding.i8_read(c8, sc, m, n, y)
        assert np.array_equal(host(y), value if t == "f32" else bf16(value)) and padding_kept(y)


@pytest.mark.parametrize("n", [40, 2100])
def test_rows_that_are_not_numbers_or_too_small(n):
    import torch
    x = np.random.default_rng(1).normal(0, 1, (6, n)).astype(np.float32)
    x[0, 3], x[1, n - 1], x[2, 0] = np.nan, np.inf, -np.inf
    x[3], x[4] = 0, 1e-38
    xd = rows(x, torch.float32)
    c8, sc, y = blank(6, n, torch.int8), torch.zeros(6, device="cuda"), blank(6, n, torch.float32)
    binding.i8_quantize(xd, 6, n, c8, sc)
    binding.i8_read(c8, sc, 6, n, y)
    y = host(y)
    assert np.isnan(y[:3]).all() and (y[3:5] == 0).all() and np.isfinite(y[5]).all()
    # the norm: a row that is not finite is NaN in 8 bits, the others are not touched by it
    out = blank(6, n, torch.bfloat16)
    binding.add_rmsnorm(xd, None, None, None, 6, n, eps=1e-6, out=out, codes=c8, scales=sc)
    sc = host(sc)
    assert np.isnan(sc[:3]).all() and np.isfinite(sc[3:]).all() and (host(c8)[:4] == 0).all()
    assert (host(out)[3] == 0).all() and np.isfinite(host(out)[5]).all()
    binding.silu_mul(xd, xd, 6, n, codes=c8, scales=torch.zeros(6, device="cuda"))


def test_no_rows():
    import torch
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    c8, sc = torch.zeros(0, 64, dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda")
    binding.add_rmsnorm(x, x, x, None, 0, 64, out=x)
    binding.silu_mul(x, x, 0, 64, codes=c8, scales=sc)
    binding.i8_quantize(x, 0, 64, c8, sc)
    binding.i8_read(c8, sc, 0, 64, x)


def test_more_rows_than_workgroups_and_rows_past_m():
    """A row's result is the same alone and among 20000; rows past m are left."""
    import torch
    n = 72
    x = torch.empty(20000, n, device="cuda").normal_()
    c8, sc = torch.full((20000, 80), 9, dtype=torch.int8, device="cuda")[:, :n], torch.full((20000,), 5.0, device="cuda")
    binding.add_rmsnorm(x, None, None, None, 19999, n, codes=c8, scales=sc)
    assert (c8[19999] == 9).all() and sc[19999] == 5
    for r in (0, 4097, 19998):
        a, b = torch.zeros(1, 80, dtype=torch.int8, device="cuda")[:, :n], torch.zeros(1, device="cuda")
        binding.add_rmsnorm(x[r:r + 1], None, None, None, 1, n, codes=a, scales=b)
        assert torch.equal(a[0], c8[r]) and torch.equal(b[0], sc[r])
