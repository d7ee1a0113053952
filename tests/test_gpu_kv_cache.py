"""Rows into the paged cache and back: layout, 8-bit codes, norm and rotation,
ragged and padded batches, faults, and the accepted path's move."""
import numpy as np
import pytest

from attnutil import Round, bf16, dev, i32, make_cache, page_table, pools_host
from oracle import attention as oa
from speculative_decoding_verify_dspk_amd import binding

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _append_case(lens, rows, heads, d, bits, page, f32, seed=1):
    import torch
    rng = np.random.default_rng(seed)
    pages = sum(-(-(n + m) // page) for n, m in zip(lens, rows)) + 2
    cache = make_cache(pages, heads, d, page, bits)
    table = page_table([n + m for n, m in zip(lens, rows)], page, pages, seed)
    total = sum(rows)
    k, v = (rng.normal(0, 2, (total, heads, d)).astype(np.float32) for _ in range(2))
    if not f32:
        k, v = bf16(k), bf16(v)
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    batch = binding.AttnBatch(i32(lens), dev(table), max(rows), total, dev(start))
    dt = torch.float32 if f32 else torch.bfloat16
    kd, vd = (dev(x.reshape(total, -1), dt) for x in (k, v))
    return cache, table, batch, k, v, kd, vd, start


CASES = [
    # lens, rows, heads, d, bits, page, fp32 rows
    ([0], [1], 8, 128, 16, 64, False),
    ([63], [1], 8, 128, 8, 64, True),
    ([61], [6], 2, 128, 16, 64, True),           # across a page
    ([64, 0, 127], [5, 5, 5], 1, 256, 8, 128, False),
    ([3, 130, 40], [17, 1, 64], 3, 64, 16, 64, False),
    ([3, 130, 40], [17, 1, 64], 3, 64, 8, 64, True),
    ([10], [300], 2, 128, 8, 256, False),        # a prompt over several pages and blocks
    ([0, 500], [200, 77], 2, 128, 16, 1024, True),
    ([31], [33], 1, 256, 16, 64, False),
    ([5, 7], [0, 3], 2, 64, 16, 64, False),      # a request without rows
]


@pytest.mark.parametrize("lens,rows,heads,d,bits,page,f32", CASES)
def test_append_layout_and_read_back(lens, rows, heads, d, bits, page, f32):
    import torch
    cache, table, batch, k, v, kd, vd, start = _append_case(lens, rows, heads, d, bits, page, f32)
    binding.kv_append(cache, batch, kd, vd)
    pk, pv = pools_host(cache)
    if bits == 8:
        (ck, sk), (cv, sv) = oa.quantise_rows(k), oa.quantise_rows(v)
        want_k, want_v = ck.astype(np.float32), cv.astype(np.float32)
        ks, vs = cache.k_scales.cpu().numpy(), cache.v_scales.cpu().numpy()
        held_k, held_v = ck * sk[..., None].astype(np.float64), cv * sv[..., None].astype(np.float64)
    else:
        want_k, want_v = bf16(k), bf16(v)
        held_k, held_v = want_k, want_v
    written = np.zeros(pk.shape[:2], dtype=bool)
    for r, (n, m) in enumerate(zip(lens, rows)):
        for i in range(m):
            page_id, t = table[r, (n + i) // page], (n + i) % page
            row = start[r] + i
            assert np.array_equal(pk[page_id, t], want_k[row]), (r, i)
            assert np.array_equal(pv[page_id, t], want_v[row]), (r, i)
            if bits == 8:
                assert np.array_equal(ks[page_id, :, t], sk[row]) and np.array_equal(vs[page_id, :, t], sv[row])
            written[page_id, t] = True
    # everything else is as it was: NaN, or code -1
    for p in (pk, pv):
        rest = p[~written]
        assert (rest == -1).all() if bits == 8 else np.isnan(rest).all()
    for out32 in (True, False):
        dt = torch.float32 if out32 else torch.bfloat16
        ko, vo = (torch.full((sum(rows) + 1, heads * d + 8), 7.0, dtype=dt, device="cuda") for _ in range(2))
        binding.kv_read(cache, batch, ko, vo)
        for o, held in ((ko, held_k), (vo, held_v)):
            o = o.float().cpu().numpy()
            assert (o[-1] == 7).all() and (o[:, heads * d:] == 7).all()     # rows and columns of no request
            want = held.reshape(sum(rows), -1).astype(np.float32)           # one rounding of scale * code
            assert np.array_equal(o[:-1, :heads * d], want if out32 else bf16(want))


def test_8bit_extreme_rows():
    """Rows of zeros, of one huge value, of values too small to scale, and rows
    with NaN or infinity: held as the rule says, without touching others."""
    import torch
    d, rows = 128, 6
    x = np.random.default_rng(0).normal(0, 1, (rows, 1, d)).astype(np.float32)
    x[0] = 0
    x[1, 0, 5] = 3e38
    x[2] *= 1e-39
    x[3, 0, 7] = NAN
    x[4, 0, 9] = -np.inf
    cache = make_cache(1, 1, d, 64, 8)
    batch = binding.AttnBatch(i32([2]), i32([[0]]), rows)
    binding.kv_append(cache, batch, dev(x.reshape(rows, d)), dev(x.reshape(rows, d)))
    ko, vo = (torch.empty((rows, d), device="cuda") for _ in range(2))
    binding.kv_read(cache, batch, ko, vo)
    code, scale = oa.quantise_rows(x)
    with np.errstate(invalid="ignore"):
        want = (code * scale[..., None]).reshape(rows, d).astype(np.float32)
    for o in (ko, vo):
        assert np.array_equal(o.cpu().numpy(), want, equal_nan=True)
    assert (want[0] == 0).all() and (want[2] == 0).all() and np.isnan(want[3:5]).all() and np.isfinite(want[5]).all()


PREP = [
    # lens, rows, hq, hkv, d, bits, fp32, rotary_dim, interleaved, norm, positions
    ([0], [1], 32, 8, 128, 16, True, 128, False, True, False),
    ([1021], [1], 32, 8, 128, 8, True, 128, False, True, True),
    ([50, 9], [6, 6], 40, 8, 128, 16, True, 128, False, True, True),
    ([7], [70], 5, 1, 64, 16, False, 32, False, False, False),
    ([100], [9], 14, 2, 64, 16, False, 64, True, True, False),
    ([30, 0, 200], [3, 90, 1], 8, 1, 256, 16, False, 256, False, True, False),
    ([30], [20], 8, 1, 256, 8, True, 96, False, True, True),
    ([5], [1100], 3, 1, 128, 16, False, 128, False, True, False),       # many rows: one workgroup per row
    ([5], [10], 4, 4, 128, 16, True, 0, False, True, False),            # norm alone
    ([5], [10], 4, 4, 128, 16, True, 48, True, False, True),
]


@pytest.mark.parametrize("lens,rows,hq,hkv,d,bits,f32,rot,inter,norm,given", PREP)
def test_norm_rope_append(lens, rows, hq, hkv, d, bits, f32, rot, inter, norm, given):
    import torch
    cache, table, batch, k, v, kd, vd, start = _append_case(lens, rows, hkv, d, bits, 64, f32, seed=3)
    rng, total = np.random.default_rng(5), sum(rows)
    q = rng.normal(0, 2, (total, hq, d)).astype(np.float32)
    q = q if f32 else bf16(q)
    dt = torch.float32 if f32 else torch.bfloat16
    qd = torch.zeros((total, hq * d + 16), dtype=dt, device="cuda")[:, :hq * d]
    qd.copy_(dev(q.reshape(total, -1), dt))
    qw, kw = ((1 + 0.3 * rng.normal(size=d)).astype(np.float32) for _ in range(2))
    freq = (1e6 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32) if rot else None
    at = np.concatenate([np.arange(n, n + m) for n, m in zip(lens, rows)])
    pos = rng.integers(0, 1 << 20, total).astype(np.int32) if given else at     # far positions too
    out = torch.full((total + 1, hq * d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    binding.qkv_norm_rope_append(cache, batch, qd, kd, vd, hq, out, q_weight=dev(qw) if norm else None,
                                 k_weight=dev(kw) if norm else None, eps=1e-6, inv_freq=dev(freq) if rot else None,
                                 interleaved=inter, positions=dev(pos) if given else None)
    got = out.float().cpu().numpy()
    assert (got[-1] == 7).all() and (got[:, hq * d:] == 7).all()
    want = oa.norm_rotate(q, qw if norm else None, 1e-6, freq, pos, inter)
    # fp32: the norm's factor is off by about 2^-22, cosines and sines by 2^-21 (the
    # fraction of a turn is rounded to 2^-25, times 2 pi), the rotation adds a few
    # 2^-24 of the pair; 2^-19 of the row's largest value covers them.  Then the rounding to bf16
    size = np.abs(want).max(-1, keepdims=True)
    err = np.abs(got[:-1, :hq * d].reshape(want.shape) - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size).all(), err.max()
    wk = oa.norm_rotate(k, kw if norm else None, 1e-6, freq, pos, inter)
    ko, vo = (torch.empty((total, hkv * d), device="cuda") for _ in range(2))
    binding.kv_read(cache, batch, ko, vo)
    for o, w in ((ko, wk), (vo, v.astype(np.float64))):
        err, size = np.abs(o.cpu().numpy().reshape(w.shape) - w), np.abs(w).max(-1, keepdims=True)
        half = size / 254 if bits == 8 else 2.0 ** -8 * np.abs(w)
        assert (err <= half * (1 + 2.0 ** -10) + 2.0 ** -19 * size).all()


def test_norm_rope_in_place_and_repeatable():
    import torch
    rng = np.random.default_rng(1)
    cache, table, batch, k, v, kd, vd, start = _append_case([9], [40], 2, 128, 16, 64, False)
    q = dev(rng.normal(size=(40, 4 * 128)).astype(np.float32), torch.bfloat16)
    w, f = dev(np.ones(128, np.float32)), dev((0.5 ** np.arange(64)).astype(np.float32))
    a = torch.empty_like(q)
    binding.qkv_norm_rope_append(cache, batch, q, kd, vd, 4, a, q_weight=w, k_weight=w, inv_freq=f)
    pools = cache.k.clone(), cache.v.clone()
    binding.qkv_norm_rope_append(cache, batch, q, kd, vd, 4, q, q_weight=w, k_weight=w, inv_freq=f)
    assert torch.equal(a, q) and torch.equal(pools[0], cache.k) and torch.equal(pools[1], cache.v)


def test_bad_lengths_and_pages_store_nothing():
    """Requests whose length or page number is a fault leave the cache as it
    is and read back as NaN; their neighbours are stored."""
    import torch
    heads, d, m = 2, 64, 4
    for bits in (16, 8):
        cache = make_cache(4, heads, d, 64, bits)
        # request 0: fine; 1: negative length; 2: past its page table; 3: page 4 of 0..3; 4: page -1
        table = i32([[0, 1], [1, 2], [1, 2], [4, 0], [-1, 0]])
        batch = binding.AttnBatch(i32([0, -1, 125, 0, 60]), table, m)
        x = dev(np.random.default_rng(0).normal(size=(5 * m, heads * d)).astype(np.float32))
        binding.kv_append(cache, batch, x, x)
        pk, pv = pools_host(cache)
        for p in (pk, pv):
            p = p[1:]
            assert (p == -1).all() if bits == 8 else np.isnan(p).all()
        ko, vo = (torch.zeros((5 * m, heads * d), device="cuda") for _ in range(2))
        binding.kv_read(cache, batch, ko, vo)
        assert np.isfinite(ko[:m].cpu().numpy()).all() and np.isfinite(vo[:m].cpu().numpy()).all()
        assert torch.isnan(ko[m:]).all() and torch.isnan(vo[m:]).all()
    # row ranges that do not fit hold no rows
    cache = make_cache(4, heads, d)
    batch = binding.AttnBatch(i32([0, 0, 0]), i32([[0], [1], [2]]), m, 5 * m, i32([-1, 8, 6, 8]))
    binding.kv_append(cache, batch, x, x)
    pk, _ = pools_host(cache)
    assert np.isnan(pk[[0, 1, 3]]).all() and np.isfinite(pk[2, :2]).all() and np.isnan(pk[2, 2:]).all()


@pytest.mark.parametrize("bits,d,heads,page,layers", [(16, 128, 3, 64, 2), (8, 64, 2, 128, 1), (16, 256, 1, 64, 70),
                                                      (8, 256, 2, 64, 3), (8, 128, 8, 64, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit_moves_the_path(bits, d, heads, page, layers, in_place):
    import torch
    rng = np.random.default_rng(bits + d)
    lens, m = [60, 3, 30, 10, 0], 64
    paths = [[0, 2, 3, 7, 9, 63], [0], [0, 1, 2, 40], [0, 5, 4], list(range(64))]      # the fourth is no path
    rounds = [Round(lens, [m] * 5, heads, d, bits, page, seed=s) for s in range(min(layers, 2))]
    base = rounds[0]
    caches = [base.cache] if layers == 1 else [rounds[i % 2].cache if i < 2 else
                                               make_cache(base.cache.pages, heads, d, page, bits) for i in range(layers)]
    before = [pools_host(c) for c in caches[:2]]
    path = np.full((5, m), -1, np.int32)
    for r, p in enumerate(paths):
        path[r, :len(p)] = p
    alen = i32([len(p) for p in paths])
    new = base.len_dev if in_place else torch.empty_like(base.len_dev)
    binding.kv_commit(caches, base.batch, dev(path), alen, new)
    want_len = [n + (0 if r == 3 else len(p)) for r, (n, p) in enumerate(zip(lens, paths))]
    assert new.tolist() == want_len
    for i, c in enumerate(caches[:2]):
        k, v = (x.copy() for x in before[i])
        for got, x in zip((k, v), before[i]):
            for r, p in enumerate(paths):
                if r == 3:
                    continue
                for to, node in enumerate(p):
                    a, b = lens[r] + node, lens[r] + to
                    got[base.table_np[r, b // page], b % page] = x[base.table_np[r, a // page], a % page]
        after = pools_host(c)
        assert np.array_equal(after[0], k, equal_nan=True) and np.array_equal(after[1], v, equal_nan=True)
    if bits == 8:
        r, (a, b) = 0, (lens[0] + 7, lens[0] + 3)
        t = base.table_np
        got = base.cache.k_scales[int(t[r, b // page]), :, b % page].cpu().numpy()
        assert np.allclose(got * 127, np.abs(base.k[0][a]).max(-1), rtol=1e-6)


def test_commit_without_lengths_and_with_bad_pages():
    R = Round([10, 20], [8, 8], 2, 64, 16, 64, seed=2)
    before = pools_host(R.cache)
    table = R.table.clone()
    table[0, 0] = 99
    batch = binding.AttnBatch(R.len_dev, table, 8)
    path = i32([[0, 3, 5, -1, -1, -1, -1, -1]] * 2)
    binding.kv_commit([R.cache], batch, path, i32([3, -1]))
    after = pools_host(R.cache)
    assert np.array_equal(before[0], after[0], equal_nan=True) and np.array_equal(before[1], after[1], equal_nan=True)
