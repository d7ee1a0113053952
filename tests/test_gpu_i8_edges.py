"""Calls of the 8-bit integer side at the edges of its variants: few slots of an expert
layer, two streams at once, replays of captured calls."""
import numpy as np
import pytest

from i8util import blank, dev, host, rows
from speculative_decoding_verify_dspk_amd import binding
from test_gpu_moe import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden,inter,experts,m,top", [
    (48, 1030, 4, 3, 2),            # rows of h longer than a wave holds
    (2048, 2048, 9, 16, 1),         # the longest such rows, 16 slots, two parts
    (64, 2049, 3, 2, 3),            # one value more
    (100, 37, 40, 1, 16), (80, 513, 40, 1, 17), (16, 1, 2, 8, 2), (33, 129, 1, 16, 1)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_few_slots(hidden, inter, experts, m, top, kind):
    import torch
    L = Layer(hidden, inter, experts, m, seed=hidden + inter)
    L.check(*L.choice(top), dtype=torch.float32 if kind == "f32" else torch.bfloat16)


@pytest.mark.parametrize("hidden,inter,experts,m,top", [
    (33, 48, 40, 64, 32), (48, 31, 33, 64, 9),       # slots past what LDS holds at a time
    (16, 16, 1024, 20, 32), (8200, 40, 6, 9, 2)])    # the most experts; more columns than parts are numbered for
def test_many_slots_experts_and_columns(hidden, inter, experts, m, top):
    L = Layer(hidden, inter, experts, m, seed=hidden + inter)
    L.check(*L.choice(top))


def test_few_slots_unused_twice_or_no_expert():
    L = Layer(80, 300, 5, 4, seed=2)
    ids = np.array([[2, 2, 2, 2], [-1, 0, -1, 3], [4, 5, 0, 1], [-1, -1, -1, -1]], dtype=np.int32)
    wt = L.rng.uniform(0.1, 1, (4, 4)).astype(np.float32)
    wt[1, 0] = wt[3, 1] = np.nan                     # weights of slots that are not used
    got = L.check(ids, np.where(ids == -1, 0, wt).astype(np.float32))
    assert np.isnan(got[2]).all() and (got[3] == 0).all() and np.isfinite(got[:2]).all()
    assert np.array_equal(L.run(ids, wt), got, equal_nan=True)
    ids[:] = [-1, 5, 1 << 30, -2]                    # nothing to multiply
    assert np.isnan(L.run(ids, wt)).all()
    ids[:] = -1
    assert (L.run(ids, wt) == 0).all()


@pytest.mark.parametrize("inter", [48, 1030, 2048])
def test_a_tokens_bits_do_not_depend_on_how_its_codes_are_made(inter):
    """Up to 16 slots and more of them."""
    L = Layer(128, inter, 6, 40, seed=inter)
    ids, wt = L.choice(4)
    whole, x, xs = L.run(ids, wt), L.x, L.xs
    for a, b in ((0, 1), (7, 11), (20, 24), (12, 17)):
        L.m, L.x, L.xs = b - a, x[a:b], xs[a:b]
        assert np.array_equal(L.run(ids[a:b], wt[a:b]), whole[a:b])


def test_rows_and_layers_on_two_streams_and_in_graphs():
    """Norm, activation, router and experts, each stream with its own workspace and
    outputs; then captured, with eager calls between the replays."""
    import torch
    m, hidden, inter, experts, top = 6, 256, 512, 8, 2
    L = Layer(hidden, inter, experts, m, seed=5)
    rng = np.random.default_rng(1)
    residual = rows(rng.normal(0, 1, (m, hidden)).astype(np.float32), torch.bfloat16)
    router = rows(rng.normal(0, 1, (experts, hidden)).astype(np.float32), torch.bfloat16)

    class Side:
        def __init__(self):
            self.x = rows(rng.normal(0, 1, (m, hidden)).astype(np.float32), torch.float32)
            self.sums, self.out = blank(m, hidden, torch.bfloat16), blank(m, hidden, torch.bfloat16)
            self.codes, self.scales = blank(m, hidden, torch.int8), torch.zeros(m, device="cuda")
            self.ids = torch.zeros(m, top, dtype=torch.int32, device="cuda")
            self.wt, self.y = torch.zeros(m, top, device="cuda"), torch.zeros(m, hidden, device="cuda")
            self.acts, self.act_scales = blank(m, hidden // 2, torch.int8), torch.zeros(m, device="cuda")
            self.ws = binding.alloc_workspace(binding.moe_workspace_bytes(hidden, inter, experts, m, top))

        def step(self):
            binding.add_rmsnorm(self.x, residual, self.sums, None, m, hidden, eps=1e-6, out=self.out,
                                codes=self.codes, scales=self.scales)
            binding.moe_route(self.out, router, m, self.ids, self.wt, self.ws)
            binding.moe_mlp(L.moe, self.codes, self.scales, m, self.ids, self.wt, self.y, self.ws)
            binding.silu_mul(self.y[:, :hidden // 2], self.y[:, hidden // 2:], m, hidden // 2, codes=self.acts,
                             scales=self.act_scales)

        def results(self):
            return [host(t).copy() for t in (self.sums, self.out, self.codes, self.scales, self.ids, self.wt, self.y,
                                             self.acts, self.act_scales)]

    sides, streams = [Side(), Side()], [torch.cuda.Stream(), torch.cuda.Stream()]
    wants = []
    for s in sides:
        s.step()
        torch.cuda.synchronize()
        wants.append(s.results())
        s.y.zero_(), s.codes.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for s, st in zip(sides, streams):
            with torch.cuda.stream(st):
                s.step()
    torch.cuda.synchronize()
    for s, want in zip(sides, wants):
        assert all(np.array_equal(a, b) for a, b in zip(s.results(), want))
    graphs = []
    for s in sides:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.step()
    for turn in range(4):
        for s, g in zip(sides, graphs):
            s.x.mul_(0.5)
            s.step()
            torch.cuda.synchronize()
            want = s.results()
            s.y.zero_(), s.codes.zero_(), s.ids.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(np.array_equal(a, b) for a, b in zip(s.results(), want))
            s.step()
