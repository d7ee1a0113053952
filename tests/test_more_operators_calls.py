"""The dense MLP's calls of perf/more_operators.py where gate and up are products of their
own (rows of an odd length): the workspace they share serves each of them."""
import importlib.util
import os

import pytest
import torch

from speculative_decoding_verify_dspk_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CASES = [dict(op="mlp", m=23, n=4352, f=873), dict(op="mlp", m=109, n=2878, f=1977), dict(op="mlp", m=23, n=4352, f=872)]


@pytest.fixture
def more():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


class OnHost:
    """torch, with the tensors that are asked for on the GPU on the host."""

    def __getattr__(self, name):
        return getattr(torch, name)

    def empty(self, *size, device=None, **options):
        return torch.empty(*size, **options)

    def zeros(self, *size, device=None, **options):
        return torch.zeros(*size, **options)


@pytest.mark.parametrize("case", CASES)
def test_the_workspace_serves_every_product(more, case, monkeypatch):
    """The sizes alone, with recorders in place of the calls."""
    m, n, f = case["m"], case["n"], case["f"]
    products, given = [], []

    class Weight:
        def __init__(self, codes, scales):
            self.n, self.k = codes.shape

    monkeypatch.setattr(more, "torch", OnHost())
    monkeypatch.setattr(binding, "Int8Weight", Weight)
    monkeypatch.setattr(binding, "alloc_workspace", lambda need: given.append(need) or need)
    monkeypatch.setattr(binding, "prepare_i8_gemm", lambda w, x, s, m, y, ws: products.append((w.n, w.k, m)))
    for name in ("prepare_add_rmsnorm", "prepare_silu_mul"):
        monkeypatch.setattr(binding, name, lambda *a, **k: None)
    codes = lambda *z: torch.zeros(z, dtype=torch.int8)
    rows, scales = torch.zeros(m, n), torch.zeros(2 * f)
    more._calls(dict(case=case, x=rows, res=rows, res_out=rows, w=rows[0], y=rows, gu8=codes(2 * f, n), gus=scales,
                     dn8=codes(n, f), dns=torch.zeros(n)))
    assert products == ([(2 * f, n, m)] if f % 8 == 0 else [(f, n, m)] * 2) + [(n, f, m)]
    assert len(given) == 1 and given[0] >= max(binding.i8_workspace_bytes(*p) for p in products)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_the_calls_run_and_give_what_calls_without_a_workspace_give(more, case):
    more.own = True
    s = more.prepare(case, 3)
    got = [t.clone() for t in more.run(s)]
    m, n, f = case["m"], case["n"], case["f"]
    blank = lambda k, dt: torch.zeros(m, -(-k // 16) * 16, dtype=dt, device="cuda")[:, :k]
    c8, h8, sums, y = blank(n, torch.int8), blank(f, torch.int8), blank(n, s["res"].dtype), blank(n, torch.bfloat16)
    cs, hs = torch.zeros(m, device="cuda"), torch.zeros(m, device="cuda")
    binding.add_rmsnorm(s["x"], s["res"], sums, s["w"], m, n, eps=1e-6, codes=c8, scales=cs)
    halves = []
    for lo in (0, f):
        halves.append(blank(f, torch.bfloat16))
        binding.i8_gemm(binding.Int8Weight(s["gu8"][lo:lo + f], s["gus"][lo:lo + f].contiguous()), c8, cs, m, halves[-1])
    binding.silu_mul(*halves, m, f, codes=h8, scales=hs)
    binding.i8_gemm(binding.Int8Weight(s["dn8"], s["dns"]), h8, hs, m, y)
    torch.cuda.synchronize()
    assert torch.equal(got[0], sums) and torch.equal(got[1], y)
