"""Attention-side calls at the edges of what they take: batches without rows,
calls side by side, pages of several requests, faults beside whole requests."""
import numpy as np
import pytest

from attnutil import Round, assert_attention, bf16, chain_masks, dev, i32, run_attention
from oracle import attention as oa
from speculative_decoding_verify_dspk_amd import binding

pytestmark = pytest.mark.gpu


def _q(R, hq):
    return bf16(R.rng.normal(0, 1, (R.total, hq, R.d)))


def _reference(R, q, r=0):
    a, e = R.starts[r], R.starts[r + 1]
    return oa.attention(q[a:e], R.k[r], R.v[r], R.lens[r], chain_masks(R.rows[r]), R.d ** -0.5)


@pytest.mark.parametrize("b", [1, 3, 70])
@pytest.mark.parametrize("pages", [1, 8, 64])
def test_batches_without_rows(b, pages):
    """Requests of no rows alone (page tables of one, two and many units): nothing
    is written, and the workspace serves the next call."""
    import torch
    R = Round([90], [2], 2, 64, 16, 64, seed=b)
    q = _q(R, 4)
    qd = dev(q.reshape(2, -1), torch.bfloat16)
    ws = binding.alloc_workspace(binding.attn_workspace_bytes(4, 2, 64, b, 8))
    table = torch.zeros((b, pages), dtype=torch.int32, device="cuda")
    empty = binding.AttnBatch(i32([0] * b), table, 8, 2, i32([0] * (b + 1)))
    out = torch.full((2, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    binding.tree_attention(R.cache, empty, qd, 4, out, ws)
    k = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    before = R.cache.k.clone()
    binding.kv_append(R.cache, empty, k, k)
    binding.qkv_norm_rope_append(R.cache, empty, qd, k, k, 4, out)
    back = torch.full((2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    binding.kv_read(R.cache, empty, back, back)
    torch.cuda.synchronize()
    assert (out == 7).all() and (back == 7).all() and torch.equal(R.cache.k, before)
    assert_attention(run_attention(R, q, 4, ws=ws), *_reference(R, q))


@pytest.mark.parametrize("bits", [16, 8])
def test_calls_on_two_streams_at_once(bits):
    """Calls that overlap, each with a workspace of its own, over one cache."""
    import torch
    R = Round([5000], [6], 2, 128, bits, 64, seed=21)
    q = _q(R, 8)
    want = run_attention(R, q, 8)
    qd = dev(q.reshape(R.total, -1), torch.bfloat16)
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(qd) for _ in sides]
    spaces = [binding.alloc_workspace(binding.attn_workspace_bytes(8, 2, 128, 1, 6)) for _ in sides]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, ws in zip(sides, outs, spaces):
            binding.tree_attention(R.cache, R.batch, qd, 8, o, ws, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert np.array_equal(o.float().cpu().numpy().reshape(want.shape), want)


@pytest.mark.parametrize("bits", [16, 8])
def test_requests_that_share_pages(bits):
    """Requests over one prefix: full pages in common, the rest their own; and
    the same request twice gives the same bits."""
    R = Round([128 + 9], [4], 2, 64, bits, 64, seed=22, pages=16)
    q = _q(R, 4)
    alone = run_attention(R, q, 4)
    table = np.repeat(R.table_np, 3, axis=0)
    lens = [137, 137, 60]
    batch = binding.AttnBatch(i32(lens), dev(table), 4)
    three = np.concatenate([q, q, q])
    T = Round([0], [1], 2, 64, bits, 64, seed=23)
    T.cache, T.batch, T.lens, T.max_rows = R.cache, batch, lens, 4
    got = run_attention(T, three, 4)
    assert np.array_equal(got[:4], got[4:8])
    assert_attention(got[:4], *_reference(R, q))
    # 60 cached positions and the four after them
    ref, mag = oa.attention(q, R.k[0][:64], R.v[0][:64], 60, chain_masks(4), R.d ** -0.5)
    assert_attention(got[8:], ref, mag)
    assert np.array_equal(alone, run_attention(R, q, 4))


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("lens,rows,hq,hkv,d", [
    ([700, 3, 0, 2500, 260], [9, 0, 1, 33, 4], 12, 2, 128),         # additions by a launch of their own, two row tiles
    ([8000, 11, 900], [1, 5, 2], 16, 1, 128),                       # few pieces, many groups
    ([6000, 500], [3, 7], 4, 1, 256),
    ([257, 511, 255, 300], [1, 1, 1, 0], 8, 2, 128),                # segments of one and two units
    ([33 * i for i in range(150)], [i % 4 for i in range(150)], 8, 2, 64),
])
def test_ragged_batches_split_over_workgroups(lens, rows, hq, hkv, d, bits):
    R = Round(lens, rows, hkv, d, bits, 64, seed=len(lens), max_rows=max(rows) + 1)
    q = _q(R, hq)
    got = run_attention(R, q, hq)
    for r in range(len(lens)):
        if rows[r]:
            assert_attention(got[R.starts[r]:R.starts[r + 1]], *_reference(R, q, r), f"request {r}")
    assert np.array_equal(got, run_attention(R, q, hq))


@pytest.mark.parametrize("bits", [16, 8])
def test_rows_that_are_not_finite_stay_alone(bits):
    """NaN and infinities in a row of q reach no other row."""
    R = Round([300], [12], 2, 128, bits, 64, seed=24)
    q = _q(R, 8)
    clean = run_attention(R, q, 8)
    q[3, 5], q[7, 0, 9] = np.nan, np.inf
    got = run_attention(R, q, 8)
    assert np.isnan(got[3, 5]).all()
    keep = np.ones(got.shape[:2], bool)
    keep[3, 5] = keep[7, 0] = False
    assert np.array_equal(got[keep], clean[keep])


def test_workspace_of_the_largest_serves_calls_of_every_shape():
    """One workspace, calls of different heads, dimensions and formats in turn."""
    import torch
    shapes = [([900], [1], 32, 8, 128, 16), ([2000], [17], 40, 8, 128, 8), ([3000, 40], [4, 4], 4, 1, 256, 16),
              ([600], [64], 64, 1, 64, 8)]
    size = max(binding.attn_workspace_bytes(hq, hkv, d, len(lens), max(rows)) for lens, rows, hq, hkv, d, _ in shapes)
    ws = binding.alloc_workspace(size)
    made = [(R, _q(R, hq), hq) for R, hq in ((Round(lens, rows, hkv, d, bits, 64, seed=hq), hq)
                                             for lens, rows, hq, hkv, d, bits in shapes)]
    want = [run_attention(R, q, hq) for R, q, hq in made]
    for i in (0, 2, 1, 3, 3, 0, 1, 2):
        R, q, hq = made[i]
        assert np.array_equal(run_attention(R, q, hq, ws=ws), want[i]), i
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits,d,f32", [(16, 128, True), (8, 128, False), (8, 64, True), (16, 256, False)])
def test_many_blocks_at_once_equal_few_at_a_time(bits, d, f32):
    """Rows of many requests in one call and request by request, in two parts,
    give the same cache and the same q to the bit."""
    import torch
    from attnutil import make_cache, page_table
    lens, rows, heads, hq = [0, 37, 64, 130, 5], [600, 411, 512, 64, 1], 16, 16
    assert sum(rows) >= 1024 and 5 * 10 * heads > 512
    g = torch.Generator(device="cuda").manual_seed(31)
    dt = torch.float32 if f32 else torch.bfloat16
    q, k, v = (torch.empty((sum(rows), heads * d), dtype=dt, device="cuda").normal_(generator=g) for _ in range(3))
    full = [n + m for n, m in zip(lens, rows)]
    pages = sum(-(-n // 64) for n in full)
    table = dev(page_table(full, 64, pages, 3))
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    w = torch.rand((2, d), device="cuda", generator=g) + 0.5
    freq = 1e4 ** (-torch.arange(0, d, 2, device="cuda") / d)
    how = dict(q_weight=w[0].contiguous(), k_weight=w[1].contiguous(), inv_freq=freq)
    got = []
    for parts in (False, True):
        c = make_cache(pages, heads, d, 64, bits)
        out = torch.zeros((sum(rows), hq * d), dtype=torch.bfloat16, device="cuda")
        if parts:
            for r, (n, m) in enumerate(zip(lens, rows)):
                for a, e in ((0, m // 3), (m // 3, m)):
                    if a < e:
                        s = slice(int(start[r]) + a, int(start[r]) + e)
                        batch = binding.AttnBatch(i32([n + a]), table[r:r + 1], e - a)
                        binding.qkv_norm_rope_append(c, batch, q[s], k[s], v[s], hq, out[s], **how)
        else:
            batch = binding.AttnBatch(i32(lens), table, max(rows), sum(rows), dev(start))
            binding.qkv_norm_rope_append(c, batch, q, k, v, hq, out, **how)
        got.append([out, c.k, c.v] + ([c.k_scales, c.v_scales] if bits == 8 else []))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("m", [1, 17])
def test_large_v_under_scores_that_rise(m):
    """v of 2^75 while a wave's scores rise by up to 2^56 of its first ones: sums
    of unscaled products stay in fp32's range."""
    import torch
    n, d = 3000, 128
    R = Round([n], [m], 1, d, 16, 64, seed=41)
    # scores of 3 |k| along one direction that q shares: from 0 to 39 nats
    q = np.zeros((m, 4, d), np.float32)
    q[:, :, 0] = 4 * d ** 0.5
    q = bf16(q)
    k = np.zeros((n + m, 1, d), np.float32)
    k[:, 0, 0] = np.linspace(0, 9.75, n + m)
    v = R.rng.normal(0, 1, (n + m, 1, d)) * 2.0 ** 75
    k, v = bf16(k), bf16(v)
    binding.kv_append(R.cache, binding.AttnBatch(i32([0]), R.table, n + m),
                      *(dev(x.reshape(n + m, -1), torch.bfloat16) for x in (k, v)))
    got = run_attention(R, q, 4)
    for i in (0, m - 1):
        ref, mag = oa.attention(q[i:i + 1], k[:n + i + 1], v[:n + i + 1], n + i, [1], d ** -0.5)
        # one product per score, of up to 39 nats: off by 2^-24 * 39 * log2(e) in the exponent, below the usual allowance
        assert_attention(got[i:i + 1], ref, mag, f"row {i}")
