"""Calls of the 8-bit integer side at the largest sizes that they take: row calls whose last
rows' numbers are within a launch's workgroups of 2^31, the router over rows as long."""
import numpy as np
import pytest

from i8util import host
from oracle import attention as oa
from speculative_decoding_verify_dspk_amd import binding

pytestmark = pytest.mark.gpu

MOST, TAIL = 2 ** 31 - 1, 40000                      # rows; more than a launch has workgroups


@pytest.fixture(autouse=True)
def _give_back():
    import torch
    yield
    torch.cuda.empty_cache()


def _room(gib):
    import torch
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of free device memory")


def _ends(rng, n):
    """Rows for the front and the back of an array."""
    import torch
    return [torch.from_numpy(rng.normal(0, 1, (TAIL, n)).astype(np.float32)).bfloat16().cuda() for _ in range(2)]


def test_the_most_rows_to_codes():
    import torch
    _room(96)
    n = 5
    x = torch.zeros(MOST, 8, dtype=torch.bfloat16, device="cuda")
    c8, sc = torch.full((MOST + 1, 16), 9, dtype=torch.int8, device="cuda"), torch.full((MOST + 1,), 5.0, device="cuda")
    front, back = _ends(np.random.default_rng(0), n)
    x[:TAIL, :n], x[-TAIL:, :n] = front, back
    binding.i8_quantize(x, MOST, n, c8, sc)
    torch.cuda.synchronize()
    for rows, at in ((front, slice(0, TAIL)), (back, slice(MOST - TAIL, MOST))):
        code, scale = oa.quantise_rows(host(rows))
        assert np.array_equal(host(c8[at, :n]), code) and np.array_equal(host(sc[at]), scale)
    assert (c8[MOST] == 9).all() and sc[MOST] == 5 and (c8[::1 << 20, n:] == 9).all()
    middle = slice(MOST // 2, MOST // 2 + TAIL)
    assert not c8[middle, :n].any() and not sc[middle].any()


def test_the_most_rows_through_norm_and_activation():
    """Results are those of the same rows in a call of their own."""
    import torch
    _room(96)
    n = 8
    x = torch.zeros(MOST, n, dtype=torch.bfloat16, device="cuda")
    out = torch.full((MOST + 1, n), 9.0, dtype=torch.bfloat16, device="cuda")
    front, back = _ends(np.random.default_rng(1), n)
    x[:TAIL], x[-TAIL:] = front, back
    calls = (lambda x, m, out: binding.add_rmsnorm(x, None, None, None, m, n, eps=1e-6, out=out),
             lambda x, m, out: binding.silu_mul(x, x, m, n, out=out),
             lambda x, m, out: binding.add_rmsnorm(x, x, x, None, m, n, eps=1e-6, out=out))      # the sum in place
    for call in calls:
        wants = [torch.zeros_like(rows) for rows in (front, back)]
        alone = [rows.clone() for rows in (front, back)]
        for rows, want in zip(alone, wants):
            call(rows, TAIL, want)
        call(x, MOST, out)
        torch.cuda.synchronize()
        assert torch.equal(out[:TAIL], wants[0]) and torch.equal(out[MOST - TAIL:MOST], wants[1])
        assert torch.equal(x[:TAIL], alone[0]) and torch.equal(x[-TAIL:], alone[1]) and (out[MOST] == 9).all()


@pytest.mark.parametrize("k", [2 ** 31 - 1, 2 ** 31 - 2049, 2 ** 31 - 8])
def test_router_over_the_longest_rows(k):
    """Scores of a few whole numbers at the front, in the middle and up to the last column."""
    import torch
    _room(24)
    x = torch.zeros(1, 2 ** 31, dtype=torch.bfloat16, device="cuda")
    router = torch.zeros(2, 2 ** 31, dtype=torch.bfloat16, device="cuda")
    x[:, k:], router[:, k:] = float("nan"), float("nan")
    rng, want = np.random.default_rng(k % 1000), np.zeros(2)
    for at in (0, 2 ** 30 - 700, k - 3000):
        a, r = rng.integers(-3, 4, (1, 3000)), rng.integers(-3, 4, (2, 3000))
        x[:, at:at + 3000] = torch.from_numpy(a).bfloat16().cuda()
        router[:, at:at + 3000] = torch.from_numpy(r).bfloat16().cuda()
        want += (a @ r.T)[0]
    ids, wt = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, device="cuda")
    z, ws = torch.zeros(1, 2, device="cuda"), binding.alloc_workspace(binding.moe_workspace_bytes(16, 16, 2, 1, 1))
    binding.moe_route(x[:, :k], router[:, :k], 1, ids, wt, ws, scores=z)
    torch.cuda.synchronize()
    assert z[0].tolist() == want.tolist() and ids.tolist() == [[int(want[1] > want[0])]] and wt.tolist() == [[1.0]]
