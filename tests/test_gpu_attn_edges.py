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
