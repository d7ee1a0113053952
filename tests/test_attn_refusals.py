"""Refusals of the attention side's calls, each a call that differs from an
accepted one in one thing alone and names it (no GPU: nothing is launched)."""
import ctypes

import pytest

from speculative_decoding_verify_dspk_amd import binding

EINVAL, EUNSUPPORTED = -1, -2
P = 0x100000           # aligned addresses that are never dereferenced


@pytest.fixture(scope="module")
def lib():
    return binding.lib()


def _cache(**kw):
    a = dict(kv_heads=8, head_dim=128, page_tokens=64, bits=16, pages=100, k=P, v=2 * P, k_scales=None, v_scales=None)
    a.update(kw)
    return binding.KVCacheDesc(*[a[n] for n, _ in binding.KVCacheDesc._fields_])


def _batch(**kw):
    a = dict(b=2, max_rows=4, total_rows=8, max_pages=9, row_start=None, cache_len=3 * P, page_table=4 * P)
    a.update(kw)
    return binding.AttnBatchDesc(*[a[n] for n, _ in binding.AttnBatchDesc._fields_])


def _refused(lib, code, expect, text):
    assert code == expect and text in lib.dspk_last_error().decode(), lib.dspk_last_error().decode()


@pytest.mark.parametrize("new_len,text", [
    (3 * P + 4, "cache_len without being it"), (3 * P - 4, "cache_len without being it"),
    (5 * P, "path or the page table"), (5 * P + 28, "path or the page table"), (6 * P, "accept_len, path"),
    (6 * P + 4, "accept_len, path"), (4 * P + 68, "the page table"), (4 * P - 4, "the page table"),
])
def test_new_lengths_over_what_a_commit_reads_are_refused(lib, new_len, text):
    """Every workgroup reads the path and its length, the first one writes new_len."""
    c, b = _cache(), _batch()
    _refused(lib, lib.dspk_kv_commit(1, ctypes.byref(c), ctypes.byref(b), 5 * P, 6 * P, new_len, None), EINVAL, text)


def _attend(lib, cache=None, batch=None, q=8 * P, ldq=4096, hq=32, scale=0.1, mask=None, out=9 * P, ldo=4096, ws=10 * P,
            wsb=1 << 30):
    c, b = cache or _cache(), batch or _batch()
    return lib.dspk_tree_attention(ctypes.byref(c), ctypes.byref(b), q, ldq, hq, scale, mask, out, ldo, ws, wsb, None)


ATTEND = [
    (dict(q=None), EINVAL, "q must be"), (dict(q=8 * P + 8), EINVAL, "q must be"),
    (dict(ldq=4088), EINVAL, "leading dimension 4088 of q"), (dict(ldq=4100), EINVAL, "leading dimension 4100 of q"),
    (dict(out=None), EINVAL, "out must be"), (dict(out=9 * P + 2), EINVAL, "out must be"),
    (dict(ldo=4088), EINVAL, "leading dimension 4088 of out"), (dict(out=8 * P), EINVAL, "out must not be q"),
    (dict(hq=12), EINVAL, "q_heads=12"), (dict(hq=4), EINVAL, "q_heads=4"), (dict(hq=0), EINVAL, "q_heads=0"),
    (dict(hq=8 * 257, ldq=1 << 20, ldo=1 << 20), EUNSUPPORTED, "at most 256 per k/v head"),
    (dict(scale=0.0), EINVAL, "scale must be"), (dict(scale=-1.0), EINVAL, "scale must be"),
    (dict(scale=float("nan")), EINVAL, "scale must be"), (dict(scale=float("inf")), EINVAL, "scale must be"),
    (dict(mask=P + 4), EINVAL, "tree_mask misaligned"),
    (dict(ws=None), EINVAL, "workspace of"), (dict(ws=10 * P + 128), EINVAL, "workspace of"),
    (dict(wsb=0), EINVAL, "workspace of"), (dict(wsb=1000), EINVAL, "workspace of"),
    (dict(batch=_batch(max_rows=65, total_rows=130)), EUNSUPPORTED, "max_rows=65"),
    (dict(batch=_batch(b=60000, total_rows=1 << 30, max_pages=1 << 20)), EUNSUPPORTED, "too large for one launch"),
    (dict(cache=_cache(bits=4)), EUNSUPPORTED, "cache bits=4"), (dict(cache=_cache(head_dim=96)), EUNSUPPORTED, "head_dim=96"),
    (dict(cache=_cache(page_tokens=96)), EUNSUPPORTED, "page_tokens=96"), (dict(cache=_cache(kv_heads=0)), EINVAL, "kv_heads=0"),
    (dict(cache=_cache(pages=0)), EINVAL, "pages=0"), (dict(cache=_cache(k=None)), EINVAL, "cache k and v"),
    (dict(cache=_cache(v=P + 16)), EINVAL, "cache k and v"), (dict(cache=_cache(k_scales=P)), EINVAL, "takes no scales"),
    (dict(cache=_cache(bits=8)), EINVAL, "needs 16-byte aligned"),
    (dict(cache=_cache(bits=8, k_scales=P, v_scales=P + 4)), EINVAL, "needs 16-byte aligned"),
    (dict(batch=_batch(b=0)), EINVAL, "b=0"), (dict(batch=_batch(max_rows=0)), EINVAL, "max_rows=0"),
    (dict(batch=_batch(total_rows=7)), EINVAL, "total_rows=7"), (dict(batch=_batch(max_pages=0)), EINVAL, "max_pages=0"),
    (dict(batch=_batch(max_pages=(1 << 24) + 1)), EUNSUPPORTED, "2^30 positions"),
    (dict(batch=_batch(cache_len=None)), EINVAL, "cache_len or page_table"),
    (dict(batch=_batch(page_table=4 * P + 2)), EINVAL, "cache_len or page_table"),
    (dict(batch=_batch(row_start=P + 1)), EINVAL, "an array misaligned"),
]


@pytest.mark.parametrize("bad,code,text", ATTEND)
def test_attention_says_what_it_refuses(lib, bad, code, text):
    _refused(lib, _attend(lib, **bad), code, text)
    assert lib.dspk_last_error().decode().startswith("dspk_tree_attention")


def test_the_workspace_asked_for_is_the_one_that_is_checked(lib):
    need = lib.dspk_attn_workspace_bytes(32, 8, 128, 2, 4)
    for size in (need - 256, need - 1):
        _refused(lib, _attend(lib, wsb=size), EINVAL, f"workspace of {need} bytes")
