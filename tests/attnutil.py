"""Helpers of the attention tests: a paged cache of poisoned memory, host-side
views of its layout, and the tolerances."""
from __future__ import annotations

import numpy as np

from speculative_decoding_verify_dspk_amd import binding

# Tolerance of an attention output (bf16) against fp64 on the same inputs, per
# element: the final rounding, half a step = 2^-8 |o|; plus, times sum p|v|:
# probabilities held to 16 significant bits (2^-16), the exponential and the
# sums in fp32 (below 2^-20), and the score's own error.  A score is a sum of at
# most 256 products in fp32, off by at most 256 * 2^-24 * scale * sum|q k| in
# the worst case; with sum|q k| * scale <= 12 for the inputs used here, 2^-12.5
# at 256 dimensions, half that at 128, as a relative error of p.
REL, ABS = 2.0 ** -8, 2.0 ** -11.5


def assert_attention(got, ref, mag, what=""):
    err, tol = np.abs(got - ref), REL * np.abs(ref) + ABS * mag + 1e-30
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    assert (err <= tol).all(), f"{what}: error {err.max():.3e}, {(err / tol).max():.2f} of the tolerance"


def bf16(x: np.ndarray) -> np.ndarray:
    """Values rounded to bf16, as fp32."""
    import torch
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def dev(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_cache(pages, heads, d, page=64, bits=16):
    """A cache whose every byte is 0xff: bf16 and fp32 NaN, code -1."""
    c = binding.KVCache.alloc(pages, heads, d, page, bits)
    for t in (c.k, c.v):
        t.fill_(255)
    if bits == 8:
        c.k_scales.fill_(float("nan"))
        c.v_scales.fill_(float("nan"))
    return c


def page_table(lens, page, pages, seed=0, spare=1):
    """Shuffled pages for the requests' total lengths; unused entries are -1."""
    need = [-(-n // page) for n in lens]
    assert sum(need) <= pages
    ids = np.random.default_rng(seed).permutation(pages)
    t = np.full((len(lens), max(max(need), 1) + spare), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        t[r, :n] = ids[at:at + n]
        at += n
    return t


def pools_host(c):
    """The pools as [page][position][head][d] (bf16 values as fp32, or codes) by the documented index."""
    import torch
    w = 8 if c.bits == 16 else 16
    dt = torch.bfloat16 if c.bits == 16 else torch.int8
    P, H, T, D = c.pages, c.kv_heads, c.page_tokens, c.head_dim
    k = c.k.view(dt).float().cpu().numpy().reshape(P, H, T // 16, D // (4 * w), 4, 16, w)
    v = c.v.view(dt).float().cpu().numpy().reshape(P, H, T // (4 * w), D // 16, 4, 16, w // 4, 4)
    out_k, out_v = np.empty((P, T, H, D), np.float32), np.empty((P, T, H, D), np.float32)
    for t in range(T):
        for d in range(D):
            out_k[:, t, :, d] = k[:, :, t // 16, d // (4 * w), d % (4 * w) // w, t % 16, d % w]
            out_v[:, t, :, d] = v[:, :, t // (4 * w), d // 16, t % 16 // 4, d % 16, t % (4 * w) // 16, t % 4]
    return out_k, out_v


class Round:
    """Requests with cached entries and a call's rows: random k/v appended
    to a poisoned cache, their values as the cache holds them on the host."""

    def __init__(self, lens, rows, heads, d, bits=16, page=64, seed=0, std=1.0, max_rows=None, pages=None):
        rng = np.random.default_rng(seed)
        self.lens, self.rows, self.heads, self.d = lens, rows, heads, d
        ragged = len(set(rows)) > 1 or (max_rows is not None and max_rows != rows[0])
        self.max_rows = max_rows or max(rows)
        full = [n + m for n, m in zip(lens, rows)]
        pages = pages or sum(-(-n // page) for n in full) + 2
        self.cache = make_cache(pages, heads, d, page, bits)
        self.table_np = page_table(full, page, pages, seed)
        self.table = dev(self.table_np)
        self.k = [bf16(rng.normal(0, std, (n, heads, d))) for n in full]
        self.v = [bf16(rng.normal(0, std, (n, heads, d))) for n in full]
        # everything in one append, as a prompt
        start = np.concatenate([[0], np.cumsum(full)]).astype(np.int32)
        import torch
        flat = lambda xs: dev(np.concatenate(xs).reshape(-1, heads * d), torch.bfloat16)
        every = binding.AttnBatch(i32([0] * len(lens)), self.table, max(full), int(start[-1]), dev(start))
        binding.kv_append(self.cache, every, flat(self.k), flat(self.v))
        if bits == 8:
            from oracle import attention as oa
            held = lambda x: (lambda c, s: c.astype(np.float64) * s[..., None])(*oa.quantise_rows(x))
            self.k, self.v = [held(x) for x in self.k], [held(x) for x in self.v]
        self.starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.total = int(self.starts[-1])
        self.len_dev = i32(lens)
        self.start_dev = dev(self.starts) if ragged else None
        self.batch = binding.AttnBatch(self.len_dev, self.table, self.max_rows, self.total, self.start_dev)
        self.rng = rng
        torch.cuda.synchronize()


def chain_masks(m):
    return [(2 << i) - 1 for i in range(m)]


def masks_dev(masks):
    return dev(np.array([x & (1 << 64) - 1 for x in masks], dtype=np.uint64).view(np.int64))


def run_attention(R: Round, q, hq, masks=None, scale=None, out=None, ws=None):
    """q fp32 values [total][hq][d] -> fp32 output [total][hq][d]."""
    import torch
    qd = dev(q.reshape(q.shape[0], -1), torch.bfloat16)
    if out is None:
        out = torch.full((q.shape[0], hq * R.d), 7.0, dtype=torch.bfloat16, device="cuda")
    if ws is None:
        ws = binding.alloc_workspace(binding.attn_workspace_bytes(hq, R.heads, R.d, len(R.lens), R.max_rows))
    binding.tree_attention(R.cache, R.batch, qd, hq, out, ws, scale, None if masks is None else masks_dev(masks))
    torch.cuda.synchronize()
    return out.float().cpu().numpy().reshape(q.shape[0], -1, R.d)
