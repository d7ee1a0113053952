"""The router and the experts of a mixture layer, against fp64 on the same inputs."""
import numpy as np
import pytest

from i8util import BF16, F32, bf16, codes, dev, host, rows, scales
from oracle import layer8
from speculative_decoding_verify_dspk_amd import binding

pytestmark = pytest.mark.gpu


def _ws(hidden, inter, experts, m, top):
    return binding.alloc_workspace(binding.moe_workspace_bytes(hidden, inter, experts, m, top))


def _route(x, r, top, normalize, scores=False, ws=None):
    import torch
    m, e = x.shape[0], r.shape[0]
    ids = torch.full((m, top), -9, dtype=torch.int32, device="cuda")
    wt = torch.full((m, top), -9.0, device="cuda")
    z = torch.full((m, e + 3), 7.0, device="cuda") if scores else None
    binding.moe_route(x, r, m, ids, wt, _ws(x.shape[1], 16, e, m, top) if ws is None else ws, normalize, z)
    return host(ids), host(wt), None if z is None else host(z)


@pytest.mark.parametrize("m,k,experts,top", [(1, 1, 1, 1), (1, 64, 8, 2), (3, 70, 5, 5), (16, 256, 16, 4), (17, 257, 17, 3),
                                             (33, 2048, 128, 8), (64, 100, 200, 6), (5, 512, 257, 32),
                                             (9, 96, 1024, 9)])
@pytest.mark.parametrize("normalize", [False, True])
def test_choice_over_exact_scores(m, k, experts, top, normalize):
    """Rows of small whole numbers, whose scores fp32 holds exactly, with many ties:
    the choice is the definition's.  Weights: exp off by 2 ulp (4 half steps) of
    arguments that are exact, at most `experts` terms, the quotient."""
    import torch
    rng = np.random.default_rng(m + experts)
    x, r = rng.integers(-3, 4, (m, k)), rng.integers(-1, 2, (experts, k))
    x[0], z = 0, None
    ids, wt, z = _route(rows(x.astype(np.float32), torch.bfloat16, 1, float("nan")),
                        rows(r.astype(np.float32), torch.bfloat16, 2, float("nan")), top, normalize, True)
    assert np.array_equal(z[:, :experts], x @ r.T) and (z[:, experts:] == 7).all()
    want, wts = layer8.route(x @ r.T, top, normalize)
    assert np.array_equal(ids, want) and ids[0].tolist() == list(range(top))
    assert (np.abs(wt - wts) <= (9 + experts) * F32 * wts + 1e-38).all()


def test_scores_of_ordinary_rows():
    """A score is a sum of k products in fp32: off by at most (k + 1) half steps of the sum of magnitudes."""
    import torch
    rng = np.random.default_rng(5)
    for m, k, experts, top in ((6, 2048, 128, 8), (40, 777, 60, 4)):
        x, r = bf16(rng.normal(0, 1, (m, k))), bf16(rng.normal(0, k ** -0.5, (experts, k)))
        ids, wt, z = _route(rows(x, torch.bfloat16), rows(r, torch.bfloat16), top, True, True)
        exact, most = x.astype(np.float64) @ r.astype(np.float64).T, np.abs(x) @ np.abs(r).T
        assert (np.abs(z[:, :experts] - exact) <= (k + 1) * F32 * most).all()
        want, wts = layer8.route(z[:, :experts], top, True)
        assert np.array_equal(ids, want)
        # the largest score's and the own one's difference is rounded too: half a step of at most 16
        assert (np.abs(wt - wts) <= (9 + top + 2 * 16) * F32 * wts).all()


def test_scores_that_are_not_numbers():
    import torch
    k, experts = 32, 10
    x, r = np.ones((5, k), np.float32), np.zeros((experts, k), np.float32)
    r[:, 0] = np.arange(experts)
    r[3, 0], r[4, 0], r[7, 1] = np.nan, -np.inf, 1
    x[1, 0] = 0                                      # 0 * inf: NaN too
    x[2, :] = np.inf
    rd = rows(r, torch.bfloat16)
    ids, wt, z = _route(rows(x, torch.bfloat16), rd, 4, True, True)
    for i in range(5):
        assert sorted(set(ids[i])) == sorted(ids[i]) and (ids[i] >= 0).all() and (ids[i] < experts).all()
    assert np.isnan(wt).all()                        # expert 3's score is NaN in every row
    assert ids[0].tolist() == [9, 7, 8, 6]
    r[3, 0] = 3
    ids, wt, z = _route(rows(x, torch.bfloat16), rows(r, torch.bfloat16), 10, False, True)
    want, wts = layer8.route(z[:, :experts], 10, False)
    assert np.array_equal(ids, want)
    assert np.array_equal(np.isnan(wt), np.isnan(wts)) and wt[0, 9] == 0 and ids[0, 9] == 4
    # every score minus infinity; plus infinity
    for sign in (-1, 1):
        r[:] = 0
        r[:, 0] = -np.inf
        if sign > 0:
            r[2, 0] = np.inf
        ids, wt, _ = _route(rows(np.ones((1, k), np.float32), torch.bfloat16), rows(r, torch.bfloat16), 3, True)
        assert np.isnan(wt).all() and ids[0].tolist() == ([0, 1, 2] if sign < 0 else [2, 0, 1])


class Layer:
    """Random experts and rows."""

    def __init__(self, hidden, inter, experts, m, seed=0):
        import torch
        rng = self.rng = np.random.default_rng(seed)
        self.hidden, self.inter, self.experts, self.m = hidden, inter, experts, m
        self.gate, self.up = ((codes(rng, experts, inter, hidden), scales(rng, experts, inter)) for _ in range(2))
        self.down = codes(rng, experts, hidden, inter), scales(rng, experts, hidden)
        self.moe = binding.MoEWeights(*(binding.Int8Weight(dev(c), dev(s)) for c, s in (self.gate, self.up, self.down)))
        self.c, self.s = codes(rng, m, hidden), scales(rng, m) * np.float32(3 / hidden ** 0.5)
        t = torch.full((m, -(-hidden // 16) * 16 + 16), -77, dtype=torch.int8, device="cuda")
        t[:, :hidden] = dev(self.c)
        self.x, self.xs = t[:, :hidden], dev(self.s)

    def choice(self, top):
        ids = np.stack([self.rng.permutation(self.experts)[:top] for _ in range(self.m)]).astype(np.int32)
        return ids, self.rng.uniform(0.05, 1, (self.m, top)).astype(np.float32)

    def run(self, ids, wt, dtype=None, ws=None, y=None):
        import torch
        if y is None:
            y = torch.full((self.m, self.hidden + 3), 7.0, dtype=dtype or torch.float32, device="cuda")
        if ws is None:
            ws = _ws(self.hidden, self.inter, self.experts, self.m, ids.shape[1])
        binding.moe_mlp(self.moe, self.x, self.xs, self.m, dev(ids), dev(wt), y, ws)
        torch.cuda.synchronize()
        assert not ws[:256 + 4 * 1024 + 4 * 512].any(), "counters left"
        assert (y[:, self.hidden:] == 7).all()
        return host(y)[:, :self.hidden]

    def check(self, ids, wt, dtype=None, ws=None):
        """h is off by at most 14 half steps (3 of each product, 8 of the activation), its
        step as much, so a code's place by 127 * 2 * 14 and the roundings of the factor
        and the product; y's terms by the step's 15, 3 of a product, the weight's product
        and top sums, besides the border codes' whole steps and the final rounding."""
        import torch
        got = self.run(ids, wt, dtype, ws)
        y, slack = layer8.experts(self.c, self.s, self.gate, self.up, self.down, ids, wt, 127 * 31 * F32)
        mag = self._magnitude(ids, wt)
        tol = slack + (20 + ids.shape[1]) * F32 * mag
        if dtype == torch.bfloat16:
            tol = tol + BF16 * (np.abs(y) + tol)
        bad = np.isnan(y)
        assert np.array_equal(np.isnan(got), bad)
        worst = (np.abs(got - y)[~bad] / (tol[~bad] + 1e-30)).max() if (~bad).any() else 0.0
        assert worst <= 1, f"{worst:.2f} of the tolerance"
        return got

    def _magnitude(self, ids, wt):
        """sum over slots of |weight * product|, as the sums' roundings count it."""
        mag = np.zeros((self.m, self.hidden))
        for i in range(self.m):
            for e, w in zip(ids[i], wt[i]):
                if 0 <= e < self.experts:
                    one, _ = layer8.experts(self.c[i:i + 1], self.s[i:i + 1], self.gate, self.up, self.down, [[e]], [[w]], 0)
                    mag[i] += np.abs(one[0])
        return mag


LAYERS = [(16, 16, 1, 1, 1), (64, 64, 4, 1, 2), (100, 37, 3, 5, 2), (256, 128, 8, 6, 2), (130, 1030, 4, 7, 3),
          (512, 96, 32, 17, 8), (2048, 768, 16, 3, 8), (80, 48, 6, 64, 6), (300, 2100, 2, 40, 1), (33, 16, 200, 64, 8)]


@pytest.mark.parametrize("hidden,inter,experts,m,top", LAYERS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_experts(hidden, inter, experts, m, top, kind):
    import torch
    L = Layer(hidden, inter, experts, m, seed=hidden + m)
    L.check(*L.choice(top), dtype=torch.float32 if kind == "f32" else torch.bfloat16)


@pytest.mark.parametrize("m", [16, 17, 33, 64])
def test_all_tokens_to_one_expert(m):
    """More rows of an expert than a pass takes, and an expert chosen twice by a token."""
    L = Layer(128, 80, 4, m, seed=m)
    ids = np.full((m, 3), 2, dtype=np.int32)
    wt = L.rng.uniform(0.1, 1, (m, 3)).astype(np.float32)
    L.check(ids, wt)
    ids[:, 1] = 0
    L.check(ids, wt)


def test_unused_slots_and_ids_that_are_no_expert():
    L = Layer(96, 64, 5, 6, seed=1)
    ids, wt = L.choice(3)
    ids[0] = -1                                       # a token without experts: zeros
    ids[1, 1] = -1
    ids[2, 0], ids[3, 2], ids[4, 1] = 5, -2, 2 ** 30  # faults: their rows alone are NaN
    got = L.check(ids, wt)
    assert (got[0] == 0).all() and np.isnan(got[2:5]).all() and np.isfinite(got[[0, 1, 5]]).all()
    assert (L.run(np.full((6, 3), -1, np.int32), wt) == 0).all()
    assert np.isnan(L.run(np.full((6, 3), 77, np.int32), wt)).all()


def test_rows_and_weights_that_are_not_numbers_stay_alone():
    L = Layer(96, 64, 5, 6, seed=2)
    ids, wt = L.choice(2)
    clean = L.run(ids, wt)
    L.xs[1] = float("nan")
    L.xs[2] = float("inf")
    wt2 = wt.copy()
    wt2[4, 1] = np.nan
    got = L.run(ids, wt2)
    assert np.isnan(got[[1, 2, 4]]).all() and np.array_equal(got[[0, 3, 5]], clean[[0, 3, 5]])
    L.xs[:] = dev(L.s)
    assert np.array_equal(L.run(ids, wt), clean)      # nothing of it stays in the weights or the workspace


def test_a_tokens_bits_do_not_depend_on_the_tokens_beside_it():
    import torch
    L = Layer(512, 320, 12, 24, seed=3)
    ids, wt = L.choice(4)
    whole = L.run(ids, wt)
    x, xs = L.x, L.xs
    for a, b in ((0, 1), (3, 8), (5, 22)):
        L.m, L.x, L.xs = b - a, x[a:b], xs[a:b]
        assert np.array_equal(L.run(ids[a:b], wt[a:b]), whole[a:b])
    del torch


def test_one_workspace_serves_router_and_layers_of_all_sizes():
    import torch
    sizes = [(512, 96, 32, 17, 8), (64, 64, 4, 1, 2), (130, 1030, 4, 7, 3), (33, 16, 200, 64, 8)]
    ws = binding.alloc_workspace(max(binding.moe_workspace_bytes(*s) for s in sizes))
    for turn in range(2):
        for hidden, inter, experts, m, top in sizes:
            L = Layer(hidden, inter, experts, m, seed=turn)
            x, r = L.rng.integers(-3, 4, (m, hidden)), L.rng.integers(-1, 2, (experts, hidden))
            ids, wt, _ = _route(rows(x.astype(np.float32), torch.bfloat16), rows(r.astype(np.float32), torch.bfloat16), top,
                                True, ws=ws)
            assert np.array_equal(ids, layer8.route(x @ r.T, top, True)[0])
            L.check(ids, wt, ws=ws)


def test_layer_in_a_graph():
    """Router and experts captured once: replays with new rows and eager calls between."""
    import torch
    L = Layer(256, 128, 16, 5, seed=9)
    top, ws = 4, _ws(256, 128, 16, 5, 4)
    x = torch.zeros(5, 256, dtype=torch.bfloat16, device="cuda")
    router = torch.empty(16, 256, dtype=torch.bfloat16, device="cuda").normal_()
    ids, wt = torch.zeros(5, top, dtype=torch.int32, device="cuda"), torch.zeros(5, top, device="cuda")
    y = torch.zeros(5, 256, device="cuda")

    def layer(out):
        binding.moe_route(x, router, 5, ids, wt, ws)
        binding.moe_mlp(L.moe, L.x, L.xs, 5, ids, wt, out, ws)

    layer(y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(y)
    for turn in range(4):
        x.normal_()
        want = torch.empty_like(y)
        layer(want)
        torch.cuda.synchronize()
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_no_rows():
    import torch
    L = Layer(64, 32, 2, 1)
    ws, e = _ws(64, 32, 2, 1, 1), lambda *z, t=torch.float32: torch.zeros(z, dtype=t, device="cuda")
    binding.moe_route(e(0, 64, t=torch.bfloat16), e(2, 64, t=torch.bfloat16), 0, e(0, 1, t=torch.int32), e(0, 1), ws)
    binding.moe_mlp(L.moe, e(0, 64, t=torch.int8), e(0), 0, e(0, 1, t=torch.int32), e(0, 1), e(0, 64), ws)
