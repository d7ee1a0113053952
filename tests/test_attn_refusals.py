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
