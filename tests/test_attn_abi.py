"""Argument checks of the attention, cache and tree calls (no GPU: every call
fails before a kernel would be launched)."""
import ctypes

import pytest

from speculative_decoding_verify_dspk_amd import binding

EINVAL, EUNSUPPORTED = -1, -2
P = 0x100000           # an aligned address that is never dereferenced


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


def _attend(lib, cache=None, batch=None, q=P, ldq=4096, hq=32, scale=0.1, mask=None, out=P, ldo=4096, ws=P, wsb=None):
    if wsb is None:
        wsb = 1 << 30
    c, b = cache or _cache(), batch or _batch()
    return lib.dspk_tree_attention(ctypes.byref(c), ctypes.byref(b), q, ldq, hq, scale, mask, out, ldo, ws, wsb, None)


def _append(lib, cache=None, batch=None, k=P, ldk=1024, v=P, ldv=1024, dt=1):
    c, b = cache or _cache(), batch or _batch()
    return lib.dspk_kv_append(ctypes.byref(c), ctypes.byref(b), k, ldk, v, ldv, dt, None)


CACHE = [
    (dict(bits=4), EUNSUPPORTED), (dict(head_dim=96), EUNSUPPORTED), (dict(page_tokens=32), EUNSUPPORTED),
    (dict(page_tokens=96), EUNSUPPORTED), (dict(page_tokens=1 << 17), EUNSUPPORTED), (dict(kv_heads=0), EINVAL),
    (dict(pages=0), EINVAL), (dict(pages=1 << 31), EINVAL), (dict(k=None), EINVAL), (dict(v=P + 16), EINVAL),
    (dict(k_scales=P), EINVAL), (dict(bits=8), EINVAL), (dict(bits=8, k_scales=P, v_scales=P + 4), EINVAL),
]
BATCH = [
    (dict(b=0), EINVAL), (dict(b=65536), EINVAL), (dict(max_rows=0), EINVAL), (dict(total_rows=7), EINVAL),
    (dict(total_rows=-1, row_start=P), EINVAL), (dict(max_pages=0), EINVAL), (dict(cache_len=None), EINVAL),
    (dict(page_table=None), EINVAL), (dict(page_table=P + 2), EINVAL), (dict(row_start=P + 1), EINVAL),
]


@pytest.mark.parametrize("bad,code", CACHE)
def test_cache_is_checked(lib, bad, code):
    c = _cache(**bad)
    assert _attend(lib, cache=c) == code
    assert lib.dspk_last_error().decode().startswith("dspk_tree_attention")
    assert _append(lib, cache=c) == code
    b = _batch()
    assert lib.dspk_kv_read(ctypes.byref(c), ctypes.byref(b), P, 1024, P, 1024, 1, None) == code
    assert lib.dspk_kv_commit(1, ctypes.byref(c), ctypes.byref(b), P, P, None, None) == code
    prep = binding.QKPrepDesc(1e-6, None, None, None, 0, 0, None)
    assert lib.dspk_qkv_norm_rope_append(ctypes.byref(c), ctypes.byref(b), ctypes.byref(prep), P, 4096, P, 1024, P, 1024,
                                         1, 8, P, 4096, None) == code


@pytest.mark.parametrize("bad,code", BATCH)
def test_batch_is_checked(lib, bad, code):
    c, b = _cache(), _batch(**bad)
    assert _attend(lib, batch=b) == code
    assert _append(lib, batch=b) == code
    assert lib.dspk_kv_read(ctypes.byref(c), ctypes.byref(b), P, 1024, P, 1024, 1, None) == code
    assert lib.dspk_kv_commit(1, ctypes.byref(c), ctypes.byref(b), P, P, None, None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), EINVAL), (dict(q=P + 8), EINVAL), (dict(ldq=4090), EINVAL), (dict(ldq=4100), EINVAL),
    (dict(out=None), EINVAL), (dict(ldo=4088), EINVAL), (dict(hq=12), EINVAL), (dict(hq=4), EINVAL), (dict(hq=0), EINVAL),
    (dict(scale=0.0), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(mask=P + 4), EINVAL), (dict(ws=None), EINVAL), (dict(ws=P + 128), EINVAL), (dict(wsb=1000), EINVAL),
    (dict(batch=_batch(max_rows=65, total_rows=130)), EUNSUPPORTED),
    (dict(batch=_batch(b=60000, total_rows=1 << 30, max_pages=1 << 20)), EUNSUPPORTED),
])
def test_attention_is_checked(lib, bad, code):
    assert _attend(lib, **bad) == code
    assert lib.dspk_last_error().decode().startswith("dspk_tree_attention")


@pytest.mark.parametrize("bad,code", [
    (dict(k=None), EINVAL), (dict(v=P + 4), EINVAL), (dict(ldk=1000), EINVAL), (dict(ldv=1028), EINVAL),
    (dict(dt=2), EINVAL), (dict(ldk=1026, dt=0), EINVAL),
    (dict(batch=_batch(b=1000, row_start=P, max_rows=1 << 30, total_rows=(1 << 31) - 1)), EUNSUPPORTED),
])
def test_append_is_checked(lib, bad, code):
    assert _append(lib, **bad) == code


@pytest.mark.parametrize("prep,args,code", [
    (None, {}, EINVAL), (dict(q_weight=P + 4), {}, EINVAL), (dict(q_weight=P, eps=-1.0), {}, EINVAL),
    (dict(k_weight=P, eps=float("nan")), {}, EINVAL), (dict(inv_freq=P + 2, rotary_dim=64), {}, EINVAL),
    (dict(inv_freq=P, rotary_dim=0), {}, EINVAL), (dict(inv_freq=P, rotary_dim=130), {}, EINVAL),
    (dict(inv_freq=P, rotary_dim=63), {}, EINVAL), (dict(inv_freq=P, rotary_dim=40), {}, EUNSUPPORTED),
    (dict(inv_freq=P, rotary_dim=64, interleaved=2), {}, EINVAL),
    (dict(inv_freq=P, rotary_dim=64, positions=P + 2), {}, EINVAL),
    ({}, dict(q=None), EINVAL), ({}, dict(ldq=4000), EINVAL), ({}, dict(hq=0), EINVAL), ({}, dict(qo=P + 8), EINVAL),
    ({}, dict(ldo=1024), EINVAL),
])
def test_norm_rope_append_is_checked(lib, prep, args, code):
    c, b = _cache(), _batch()
    a = dict(eps=1e-6, q_weight=None, k_weight=None, inv_freq=None, rotary_dim=0, interleaved=0, positions=None)
    a.update(prep or {})
    d = binding.QKPrepDesc(*[a[n] for n, _ in binding.QKPrepDesc._fields_])
    v = dict(q=P, ldq=4096, hq=32, qo=P, ldo=4096)
    v.update(args)
    assert lib.dspk_qkv_norm_rope_append(ctypes.byref(c), ctypes.byref(b), None if prep is None else ctypes.byref(d),
                                         v["q"], v["ldq"], P, 1024, P, 1024, 1, v["hq"], v["qo"], v["ldo"], None) == code
    assert lib.dspk_last_error().decode().startswith("dspk_qkv_norm_rope_append")


def test_tree_calls_are_checked(lib):
    lay, acc = lib.dspk_tree_layout, lib.dspk_accept_tree_greedy
    for args in ((P, 0, 4, P, P, P), (P, 1, 0, P, P, P), (P, 1, 65, P, P, P), (None, 1, 4, P, P, P), (P, 1, 4, None, P, P),
                 (P, 1, 4, P, P + 4, P), (P, 1, 4, P, P, None)):
        assert lay(*args, None) == EINVAL
    for args in ((None, P, P, 1, 4, P, P, P), (P, None, P, 1, 4, P, P, P), (P, P, None, 1, 4, P, P, P),
                 (P, P, P, 0, 4, P, P, P), (P, P, P, 1, 65, P, P, P), (P, P, P, 1, 4, None, P, P),
                 (P, P, P, 1, 4, P, P, None), (P + 2, P, P, 1, 4, P, P, P)):
        assert acc(*args, None) == EINVAL


def test_commit_is_checked(lib):
    two = (binding.KVCacheDesc * 2)(_cache(), _cache(kv_heads=4))
    b = _batch()
    f = lib.dspk_kv_commit
    assert f(2, two, ctypes.byref(b), P, P, None, None) == EINVAL                # not one shape
    assert f(0, two, ctypes.byref(b), P, P, None, None) == EINVAL
    assert f(1, None, ctypes.byref(b), P, P, None, None) == EINVAL
    assert f(1, two, ctypes.byref(b), None, P, None, None) == EINVAL
    assert f(1, two, ctypes.byref(b), P, None, None, None) == EINVAL
    assert f(1, two, ctypes.byref(b), P, P, 3 * P + 4, None) == EINVAL           # overlaps cache_len
    assert f(1, two, ctypes.byref(_batch(row_start=P)), P, P, None, None) == EUNSUPPORTED
    assert f(1, two, ctypes.byref(_batch(max_rows=65, total_rows=130)), P, P, None, None) == EUNSUPPORTED


def test_sizes(lib):
    assert lib.dspk_kv_cache_bytes(10, 8, 128, 64, 16) == 10 * 8 * 128 * 64 * 2
    assert lib.dspk_kv_cache_bytes(10, 8, 128, 64, 8) == 10 * 8 * 128 * 64
    assert lib.dspk_kv_cache_bytes(10, 8, 100, 64, 8) == 0 and lib.dspk_kv_cache_bytes(0, 8, 128, 64, 8) == 0
    f = lib.dspk_attn_workspace_bytes
    assert f(32, 8, 128, 1, 17) > 0 and f(32, 8, 128, 1, 17) % 256 == 0
    assert f(32, 5, 128, 1, 1) == 0 and f(32, 8, 100, 1, 1) == 0 and f(32, 8, 128, 1, 65) == 0 and f(4, 8, 128, 1, 1) == 0
    # fewer rows never need more than the most
    for d, hq, hkv in ((128, 40, 8), (256, 8, 1), (64, 8, 8)):
        for m in range(1, 65):
            assert all(f(hq, hkv, d, 1, x) <= f(hq, hkv, d, 1, m) for x in range(1, m))


def test_binding_checks_tensors():
    import torch
    e = torch.empty
    with pytest.raises(binding.DspkError):
        binding.KVCache.alloc(4, 8, 100, device="cpu")
    with pytest.raises(ValueError):
        binding.KVCache(e(10), e(10), 4, 8, 128)
    c = binding.KVCache.alloc(4, 2, 64, bits=8, device="cpu")
    lens, table = e(3, dtype=torch.int32), e((3, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.AttnBatch(lens, table[:2], 4)
    with pytest.raises(ValueError):
        binding.AttnBatch(lens.long(), table, 4)
    with pytest.raises(ValueError):
        binding.AttnBatch(lens, table, 4, row_start=lens)
    b = binding.AttnBatch(lens, table, 4)
    row = lambda n, m, t=torch.bfloat16: e((n, m), dtype=t)
    with pytest.raises(ValueError):
        binding.kv_append(c, b, row(11, 128), row(12, 128))           # too few rows
    with pytest.raises(ValueError):
        binding.kv_append(c, b, row(12, 120), row(12, 128))           # too few columns
    with pytest.raises(ValueError):
        binding.kv_append(c, b, row(12, 128), row(12, 128, torch.float32))
    with pytest.raises(ValueError):
        binding.tree_attention(c, b, row(12, 256), 4, row(12, 256), e(256, dtype=torch.uint8),
                               tree_mask=e(12, dtype=torch.int32))


def test_page_tables_past_2_to_the_30_positions_are_refused(lib):
    """A length near 2^31 would pass 32 bits in position arithmetic."""
    c = _cache(page_tokens=65536)
    for pages, code in ((16385, EUNSUPPORTED), (32768, EUNSUPPORTED), ((1 << 31) - 1, EUNSUPPORTED)):
        b = _batch(max_pages=pages)
        assert _attend(lib, cache=c, batch=b) == code and _append(lib, cache=c, batch=b) == code
        assert lib.dspk_kv_read(ctypes.byref(c), ctypes.byref(b), P, 1024, P, 1024, 1, None) == code
        assert lib.dspk_kv_commit(1, ctypes.byref(c), ctypes.byref(b), P, P, None, None) == code
    b = _batch(max_pages=16384)                                              # the most: refused for what follows it
    assert _append(lib, cache=c, batch=b, k=None) == EINVAL


def test_outputs_over_inputs_are_refused(lib):
    """Workgroups read q rows that others would have overwritten."""
    assert _attend(lib, q=P, out=P) == EINVAL
    assert "out must not be q" in lib.dspk_last_error().decode()
    c, b, d = _cache(), _batch(), binding.QKPrepDesc(1e-6, None, None, None, 0, 0, None)
    for dt, ldq, ldo in ((0, 4096, 4096), (1, 4096, 4608)):
        assert lib.dspk_qkv_norm_rope_append(ctypes.byref(c), ctypes.byref(b), ctypes.byref(d), P, ldq, 2 * P, 1024,
                                             3 * P, 1024, dt, 32, P, ldo, None) == EINVAL
        assert "q_out may be q only" in lib.dspk_last_error().decode()


def test_binding_checks_sizes_of_trees():
    import torch
    i = lambda *z: torch.zeros(z, dtype=torch.int32)
    b, m = 2, 5
    good = dict(target_ids=i(b, m), draft_ids=i(b, m - 1), parents=i(b, m - 1), accept_len=i(b), committed=i(b, m),
                path=i(b, m))
    for name, t in good.items():
        for bad in (t.view(-1)[:-1], t.long()):
            with pytest.raises(ValueError, match=name):
                binding.prepare_accept_tree_greedy(**{**good, name: bad}, b=b, m_rows=m)
    good = dict(parents=i(b, m - 1), cache_len=i(b), tree_mask=i(b, m).long(), positions=i(b, m))
    for name, t in good.items():
        with pytest.raises(ValueError, match=name):
            binding.prepare_tree_layout(**{**good, name: t.view(-1)[:-1]}, b=b, m_rows=m)
    c = binding.KVCache.alloc(4, 2, 64, device="cpu")
    batch = binding.AttnBatch(i(b), i(b, 2), m)
    good = dict(path=i(b, m), accept_len=i(b), new_len=i(b))
    for name, t in good.items():
        with pytest.raises(ValueError, match=name):
            binding.prepare_kv_commit([c], batch, **{**good, name: t.view(-1)[:-1]})
