"""Helpers of the 8-bit integer side's tests: seeded rows and codes in padded
arrays whose padding is poison, and the roundings that tolerances count."""
from __future__ import annotations

import numpy as np

F32, BF16 = 2.0 ** -24, 2.0 ** -8              # half a step of a value


def bf16(x):
    """Values rounded to bf16, as fp32."""
    import torch
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def rows(x, dtype, pad=0, poison=7.0):
    """Host values [m][n] as device rows whose leading dimension is n rounded up to
    16, plus 16 * pad; the columns past n hold `poison`."""
    import torch
    x = torch.from_numpy(np.ascontiguousarray(x))
    m, n = x.shape
    out = torch.full((m, -(-n // 16) * 16 + 16 * pad), poison, dtype=dtype, device="cuda")
    out[:, :n] = x.to(dtype).cuda()
    return out[:, :n]


def blank(m, n, dtype, pad=0, poison=7):
    import torch
    return torch.full((m, -(-n // 16) * 16 + 16 * pad), poison, dtype=dtype, device="cuda")[:, :n]


def padding_kept(t, poison=7):
    """Whether the columns past a row's length hold what they held."""
    whole = t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1))
    return bool((whole[:, t.shape[1]:] == poison).all())


def host(t):
    import torch
    return (t.float() if t.dtype == torch.bfloat16 else t).cpu().numpy()


def codes(rng, *shape):
    """Codes of normal values with the extremes among them."""
    c = np.clip(np.rint(rng.normal(0, 40, shape)), -127, 127).astype(np.int8)
    c.reshape(-1)[::97] = 127
    c.reshape(-1)[5::89] = -128
    return c


def scales(rng, *shape):
    return rng.uniform(0.001, 0.02, shape).astype(np.float32)


def dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def assert_codes(got, got_scale, y, rel, what=""):
    """8-bit rows of y (fp64 [m][n]) computed with a relative error of at most `rel`: a
    code is off its place by half a step, by the error of the value and of the scale
    (each at most 127 steps times rel) and by the roundings of the factor 127 / top and
    of the product."""
    from oracle import layer8
    place, step = layer8.in_codes(y)
    assert (np.abs(got - place) <= 0.5 + 127 * (2 * rel + 3 * F32)).all(), \
        f"{what}: {np.abs(got - place).max()} steps off"
    assert (np.abs(got_scale - step) <= (rel + 2 * F32) * step).all(), f"{what}: scales"
