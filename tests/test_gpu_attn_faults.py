"""Attention-side calls on data that holds faults or values that are not finite,
and under page tables wider than the lengths."""
import numpy as np
import pytest

from attnutil import Round, assert_attention, bf16, chain_masks, dev, i32, pools_host, run_attention
from oracle import attention as oa
from speculative_decoding_verify_dspk_amd import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit_keeps_requests_whose_path_meets_a_bad_page(bits, in_place):
    """A path is taken whole or not at all: where an entry lies, or would go, on
    a page that is none of the cache's, nothing moves in any layer and the
    length stays.  Bad pages that the path does not meet do not matter."""
    import torch
    lens, m = [60, 60, 63, 62, 60, 130], 8
    A, B = (Round(lens, [m] * 6, 2, 64, bits, 64, seed=s) for s in (51, 52))
    table = A.table.clone()
    pages = A.cache.pages
    table[0, 1] = pages                 # node 5 alone is on it: a source
    table[1, 1] = -1                    # not met
    table[2, 0] = pages + 7             # node 0 alone is on it
    table[3, 1] = -1                    # a source and a destination
    table[4, 0] = -2                    # the only node
    batch = binding.AttnBatch(A.len_dev, table, m)
    paths = [[0, 2, 5], [0, 2, 3], [0, 4], [0, 3, 5], [0], [0, 1, 6]]
    kept = [False, True, False, False, False, True]
    path = np.full((6, m), -1, np.int32)
    for r, p in enumerate(paths):
        path[r, :len(p)] = p
    before = [pools_host(R.cache) for R in (A, B)]
    new = A.len_dev if in_place else torch.full_like(A.len_dev, -7)
    binding.kv_commit([A.cache, B.cache], batch, i32(path.tolist()), i32([len(p) for p in paths]), new)
    assert new.tolist() == [n + (len(p) if ok else 0) for n, p, ok in zip(lens, paths, kept)]
    for R, was in zip((A, B), before):
        for got, x in zip(pools_host(R.cache), was):
            want = x.copy()
            for r, p in enumerate(paths):
                for to, node in enumerate(p if kept[r] else []):
                    a, b = lens[r] + node, lens[r] + to
                    # both rounds have shuffled pages of their own; the call's are A's
                    want[A.table_np[r, b // 64], b % 64] = x[A.table_np[r, a // 64], a % 64]
            assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("n,m,hq,hkv,d", [(100, 1, 4, 1, 128), (3000, 17, 8, 1, 128), (700, 6, 8, 2, 64), (500, 3, 2, 1, 256),
                                          (9000, 40, 16, 2, 128)])
@pytest.mark.parametrize("even", [True, False])
def test_cached_v_that_is_not_finite(n, m, hq, hkv, d, even):
    """Infinities and NaN of cached v, with probabilities of any number of bits
    (even: all the same, a power of two): an infinity comes out as one, opposite
    ones and NaN as NaN, and other dimensions keep their bits."""
    import torch
    R = Round([n], [m], hkv, d, 16, 64, seed=n + m)
    q = bf16(R.rng.normal(0, 0 if even else 1, (m, hq, d)))
    clean, odd = R.v[0].copy(), R.v[0].copy()
    inf = np.float32("inf")
    # (position, dimension, value); the last two positions are among the call's rows
    spots = [(3, 5, inf), (n - 1, 9, -inf), (n // 2, 17, inf), (n // 2 + 1, 17, -inf), (40, 33, np.nan), (7, 40, inf),
             (n, 40, -inf), (n + m - 1, 41, inf)]
    for t, i, x in spots:
        clean[t, 0, i], odd[t, 0, i] = 0, x
    out = []
    every = binding.AttnBatch(i32([0]), R.table, n + m)
    for v in (clean, odd):
        binding.kv_append(R.cache, every, *(dev(x.reshape(n + m, -1), torch.bfloat16) for x in (R.k[0], v)))
        out.append(run_attention(R, q, hq))
    want = out[0].copy()
    rep = hq // hkv                                       # the first k/v head alone holds them
    want[:, :rep, 5], want[:, :rep, 9] = inf, -inf
    want[:, :rep, [17, 33]] = np.nan
    want[:, :rep, 40] = np.nan                            # every row sees row 0 of the call
    want[m - 1, :rep, 41] = inf
    assert np.array_equal(out[1], want, equal_nan=True)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("lens,rows,hq,hkv,d", [([1021], [1], 32, 8, 128), ([1000], [16], 32, 8, 128),
                                                ([400, 30, 0], [6, 2, 1], 8, 2, 64), ([700], [3], 8, 1, 256)])
def test_page_tables_wider_than_the_lengths(lens, rows, hq, hkv, d, bits):
    """A table with room for 1, 8 and 128 times the positions (the plan goes by
    its width); its unused entries are no pages."""
    R = Round(lens, rows, hkv, d, bits, 64, seed=61, max_rows=max(rows))
    q = bf16(R.rng.normal(0, 1, (R.total, hq, d)))
    tight = R.table_np
    for wide in (1, 8, 128):
        table = np.full((len(lens), tight.shape[1] * wide), -1, np.int32)
        table[:, :tight.shape[1]] = tight
        R.batch = binding.AttnBatch(R.len_dev, dev(table), R.max_rows, R.total, R.start_dev)
        got = run_attention(R, q, hq)
        for r, (n, m) in enumerate(zip(lens, rows)):
            a, e = R.starts[r], R.starts[r + 1]
            ref, mag = oa.attention(q[a:e], R.k[r], R.v[r], n, chain_masks(m), d ** -0.5)
            assert_attention(got[a:e], ref, mag, f"{wide}x, request {r}")


@pytest.mark.parametrize("bits", [16, 8])
def test_a_prompt_in_calls_of_64_rows(bits):
    """A prompt's rows attend in calls of up to 64, cache_len advanced by each,
    over entries that one append has stored."""
    import torch
    n, m, hq, hkv, d = 37, 150, 8, 2, 64
    R = Round([n], [m], hkv, d, bits, 64, seed=62)
    q = bf16(R.rng.normal(0, 1, (m, hq, d)))
    qd = dev(q.reshape(m, -1), torch.bfloat16)
    out = torch.zeros_like(qd)
    ws = binding.alloc_workspace(binding.attn_workspace_bytes(hq, hkv, d, 1, 64))
    for a in range(0, m, 64):
        e = min(a + 64, m)
        binding.tree_attention(R.cache, binding.AttnBatch(i32([n + a]), R.table, e - a), qd[a:e], hq, out[a:e], ws)
    got = out.float().cpu().numpy().reshape(m, hq, d)
    for a in range(0, m, 64):
        e = min(a + 64, m)
        ref, mag = oa.attention(q[a:e], R.k[0][:n + e], R.v[0][:n + e], n + a, chain_masks(e - a), d ** -0.5)
        assert_attention(got[a:e], ref, mag, f"rows {a}..")
