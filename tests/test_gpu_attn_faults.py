"""Attention-side calls on data that holds faults or values that are not finite."""
import numpy as np
import pytest

from attnutil import Round, i32, pools_host
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
