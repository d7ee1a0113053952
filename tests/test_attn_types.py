"""Element types that the attention side's calls do not read are refused (no GPU:
every call fails before its arguments are handed on)."""
import pytest
import torch

from speculative_decoding_verify_dspk_amd import binding

HEADS, D, ROWS = 2, 64, 3
BAD_ROWS = [torch.float16, torch.float64, torch.int32, torch.int64, torch.int8, torch.bool]


def _rows(dtype, columns=HEADS * D):
    return torch.zeros((ROWS, columns), dtype=dtype)


@pytest.fixture(scope="module")
def cache():
    return binding.KVCache.alloc(2, HEADS, D, device="cpu")


@pytest.fixture(scope="module")
def batch():
    return binding.AttnBatch(torch.zeros(1, dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int32), ROWS)


@pytest.mark.parametrize("dtype", BAD_ROWS)
def test_rows_of_other_types_are_refused(cache, batch, dtype):
    good, bad = _rows(torch.bfloat16), _rows(dtype)
    f32 = _rows(torch.float32)
    ws = torch.zeros(256, dtype=torch.uint8)
    for name, call in (
        ("k", lambda: binding.kv_append(cache, batch, bad, bad)),
        ("v", lambda: binding.kv_append(cache, batch, good, bad)),
        ("k", lambda: binding.kv_read(cache, batch, bad, good)),
        ("v", lambda: binding.kv_read(cache, batch, f32, bad)),
        ("k", lambda: binding.qkv_norm_rope_append(cache, batch, good, bad, bad, HEADS, good)),
        ("q", lambda: binding.qkv_norm_rope_append(cache, batch, bad, good, good, HEADS, good)),
        ("q_out", lambda: binding.qkv_norm_rope_append(cache, batch, f32, f32, f32, HEADS, bad)),
        ("q", lambda: binding.tree_attention(cache, batch, bad, HEADS, good, ws)),
        ("out", lambda: binding.tree_attention(cache, batch, good, HEADS, bad, ws)),
    ):
        with pytest.raises(ValueError, match=f"^{name}: expected float32 or bf16 rows, got {dtype}"):
            call()


@pytest.mark.parametrize("dtype", [torch.int32, torch.float16, torch.float64])
def test_scales_of_other_types_are_refused(dtype):
    pool = torch.zeros(binding.kv_cache_bytes(2, HEADS, D, 64, 8), dtype=torch.uint8)
    good, bad = (torch.zeros((4, HEADS, 64), dtype=t) for t in (torch.float32, dtype))
    binding.KVCache(pool, pool, 2, HEADS, D, 64, 8, good, good)
    for name, scales in (("k_scales", (bad, good)), ("v_scales", (good, bad))):
        with pytest.raises(ValueError, match=f"{name}: expected float32"):
            binding.KVCache(pool, pool, 2, HEADS, D, 64, 8, *scales)


@pytest.mark.parametrize("dtype", [torch.float64, torch.complex64, torch.int32])
def test_masks_of_other_types_are_refused(cache, batch, dtype):
    q, ws = _rows(torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    with pytest.raises(ValueError, match="tree_mask"):
        binding.tree_attention(cache, batch, q, HEADS, q.clone(), ws, tree_mask=torch.zeros(8, dtype=dtype))
    with pytest.raises(ValueError, match="tree_mask"):
        binding.tree_layout(i(2), 1, 3, i(1), torch.zeros(8, dtype=dtype), i(3))
