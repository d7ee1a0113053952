"""Refusals of the 8-bit integer side's calls, each a call that differs from an
accepted one in one thing alone and names it (no GPU: nothing is launched; the
accepted calls themselves have no rows)."""
import ctypes

import pytest
import torch

from speculative_decoding_verify_dspk_amd import binding

EINVAL, EUNSUPPORTED = -1, -2
P = 0x100000           # aligned addresses that are never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return binding.lib()


def _refused(lib, who, got, expect, text):
    said = lib.dspk_last_error().decode()
    assert got == expect and said.startswith(who) and text in said, (got, said)


def _out(**kw):
    a = dict(rows=P, ld=264, codes=2 * P, ldc=272, scales=3 * P)
    a.update(kw)
    return ctypes.byref(binding.RowsOutDesc(*[a[n] for n, _ in binding.RowsOutDesc._fields_]))


def _norm(lib, x=4 * P, ldx=264, xt=1, r=5 * P, ldr=264, rt=1, ro=6 * P, ldro=264, w=7 * P, eps=1e-6, m=3, n=260,
          out=None):
    return lib.dspk_add_rmsnorm(x, ldx, xt, r, ldr, rt, ro, ldro, w, eps, m, n, _out() if out is None else out, None)


OUT = [
    (dict(rows=P + 8), "out.rows must be"), (dict(ld=256), "leading dimension 256 of out.rows"),
    (dict(ld=260), "leading dimension 260 of out.rows"), (dict(codes=2 * P + 8), "out.codes must be"),
    (dict(ldc=264), "leading dimension 264 of out.codes"), (dict(ldc=256), "leading dimension 256 of out.codes"),
    (dict(scales=None), "the scales of out.codes"), (dict(scales=3 * P + 2), "the scales of out.codes"),
    (dict(codes=None), "out.scales without"), (dict(rows=None, codes=None, scales=None), "neither rows nor codes"),
]


@pytest.mark.parametrize("bad,code,text", [
    (dict(m=-1), EINVAL, "m=-1"), (dict(n=0), EINVAL, "n=0"), (dict(n=32769), EUNSUPPORTED, "n=32769"),
    (dict(xt=2), EINVAL, "element type 2 of x"), (dict(rt=-1), EINVAL, "element type -1 of residual"),
    (dict(eps=-1.0), EINVAL, "eps"), (dict(eps=NAN), EINVAL, "eps"), (dict(eps=INF), EINVAL, "eps"),
    (dict(w=7 * P + 4), EINVAL, "weight must be"), (dict(x=None, r=None), EINVAL, "both NULL"),
    (dict(x=4 * P + 4), EINVAL, "x must be"), (dict(ldx=256), EINVAL, "leading dimension 256 of x"),
    (dict(ldx=268), EINVAL, "leading dimension 268 of x"), (dict(xt=0, ldx=262), EINVAL, "leading dimension 262 of x"),
    (dict(r=5 * P + 2), EINVAL, "residual must be"), (dict(ldr=268), EINVAL, "leading dimension 268 of residual"),
    (dict(ro=6 * P + 2), EINVAL, "residual_out must be"), (dict(ldro=1), EINVAL, "of residual_out"),
    (dict(ro=5 * P, ldro=272), EINVAL, "residual_out may be"), (dict(ro=4 * P, ldro=272), EINVAL, "residual_out may be"),
    (dict(ro=4 * P, xt=0), EINVAL, "residual_out may be"),
])
def test_norm_says_what_it_refuses(lib, bad, code, text):
    assert _norm(lib, m=0) == 0
    _refused(lib, "dspk_add_rmsnorm", _norm(lib, **bad), code, text)


@pytest.mark.parametrize("bad,text", OUT)
def test_outputs_of_row_calls_are_checked(lib, bad, text):
    _refused(lib, "dspk_add_rmsnorm", _norm(lib, out=_out(**bad)), EINVAL, text)
    got = lib.dspk_silu_mul(P, 264, 2 * P, 264, 1, 3, 260, _out(**bad), None)
    _refused(lib, "dspk_silu_mul", got, EINVAL, text)
    _refused(lib, "dspk_silu_mul", lib.dspk_silu_mul(P, 264, 2 * P, 264, 1, 3, 260, None, None), EINVAL, "out is NULL")


@pytest.mark.parametrize("bad,code,text", [
    (dict(g=None), EINVAL, "gate must be"), (dict(ldg=262), EINVAL, "of gate"), (dict(u=P + 2), EINVAL, "up must be"),
    (dict(ldu=200), EINVAL, "of up"), (dict(dt=3), EINVAL, "element type 3"), (dict(m=-2), EINVAL, "m=-2"),
    (dict(n=1 << 16), EUNSUPPORTED, "n=65536"),
])
def test_activation_says_what_it_refuses(lib, bad, code, text):
    a = dict(g=P, ldg=264, u=2 * P, ldu=264, dt=1, m=3, n=260)
    call = lambda a: lib.dspk_silu_mul(a["g"], a["ldg"], a["u"], a["ldu"], a["dt"], a["m"], a["n"], _out(), None)
    assert call(dict(a, m=0)) == 0
    _refused(lib, "dspk_silu_mul", call(dict(a, **bad)), code, text)


@pytest.mark.parametrize("bad,code,text", [
    (dict(x=None), EINVAL, " must be"), (dict(ldx=260), EINVAL, "leading dimension 260 of"), (dict(dt=2), EINVAL, "element type 2"),
    (dict(c=2 * P + 4), EINVAL, "codes must be"), (dict(ldc=264), EINVAL, "leading dimension 264 of codes"),
    (dict(s=None), EINVAL, "the scales of codes"), (dict(m=-1), EINVAL, "m=-1"), (dict(n=0), EINVAL, "n=0"),
    (dict(n=40000), EUNSUPPORTED, "n=40000"),
])
def test_quantising_and_reading_say_what_they_refuse(lib, bad, code, text):
    a = dict(x=P, ldx=264, dt=1, m=3, n=260, c=2 * P, ldc=272, s=3 * P)
    there = lambda a: lib.dspk_i8_quantize(a["x"], a["ldx"], a["dt"], a["m"], a["n"], a["c"], a["ldc"], a["s"], None)
    back = lambda a: lib.dspk_i8_read(a["c"], a["ldc"], a["s"], a["m"], a["n"], a["x"], a["ldx"], a["dt"], None)
    for who, call in (("dspk_i8_quantize", there), ("dspk_i8_read", back)):
        assert call(dict(a, m=0)) == 0
        _refused(lib, who, call(dict(a, **bad)), code, text)


def _weight(**kw):
    a = dict(n=100, k=130, count=1, tiles=P, scales=2 * P)
    a.update(kw)
    return binding.Int8WeightDesc(*[a[n] for n, _ in binding.Int8WeightDesc._fields_])


def _gemm(lib, w=None, x=3 * P, ldx=144, xs=4 * P, m=3, y=5 * P, dt=0, ldy=100, ws=None, wsb=0, **weight):
    w = ctypes.byref(_weight(**weight)) if w is None else None
    return lib.dspk_i8_gemm(w, x, ldx, xs, m, y, dt, ldy, ws, wsb, None)


WEIGHT = [
    (dict(n=0), EINVAL, "n=0"), (dict(k=0), EINVAL, "k=0"), (dict(count=0), EINVAL, "count=0"),
    (dict(k=131072), EUNSUPPORTED, "k=131072"), (dict(tiles=None), EINVAL, "tiles of"), (dict(tiles=P + 128), EINVAL, "tiles of"),
    (dict(scales=None), EINVAL, "tiles of"), (dict(scales=P + 1), EINVAL, "tiles of"),
]


@pytest.mark.parametrize("bad,code,text", WEIGHT + [
    (dict(w="none"), EINVAL, "w is NULL"), (dict(count=2), EINVAL, "count=2"), (dict(m=-1), EINVAL, "m=-1"),
    (dict(x=None), EINVAL, "x must be"), (dict(x=P + 8), EINVAL, "x must be"), (dict(ldx=128), EINVAL, "of x"),
    (dict(ldx=136), EINVAL, "leading dimension 136 of x"), (dict(ldx=(1 << 24) + 16), EUNSUPPORTED, "ldx=16777232"), (dict(xs=None), EINVAL, "the scales of x"),
    (dict(y=None), EINVAL, "y NULL"), (dict(y=5 * P + 2), EINVAL, "y NULL or misaligned"), (dict(ldy=99), EINVAL, "ldy=99"),
    (dict(dt=2), EINVAL, "element type 2 of y"), (dict(ws=P + 64, wsb=1 << 30), EINVAL, "workspace of"),
    (dict(n=(1 << 31) - 1, m=1 << 20, ldy=1 << 31), EUNSUPPORTED, "too many tiles"),
])
def test_product_says_what_it_refuses(lib, bad, code, text):
    assert _gemm(lib, m=0) == 0
    _refused(lib, "dspk_i8_gemm", _gemm(lib, **bad), code, text)


def test_the_product_workspace_asked_for_is_the_one_that_is_checked(lib):
    for m, n, k in ((300, 640, 4000), (128, 128, 8192), (1, 100, 130)):
        need = lib.dspk_i8_workspace_bytes(n, k, m)
        if need:
            _refused(lib, "dspk_i8_gemm", _gemm(lib, n=n, k=k, m=m, ldx=8192, ldy=n, ws=P, wsb=need - 1), EINVAL,
                     f"workspace of {need} bytes")
    assert lib.dspk_i8_workspace_bytes(0, 64, 1) == lib.dspk_i8_workspace_bytes(64, 64, 0) == 0
    assert lib.dspk_i8_workspace_bytes(64, 131072, 1) == 0


@pytest.mark.parametrize("bad,code,text", [
    (dict(c=None), EINVAL, "codes NULL"), (dict(ldc=129), EINVAL, "ldc=129"), (dict(t=None), EINVAL, "tiles of"),
    (dict(t=P + 16), EINVAL, "tiles of"), (dict(b=-1), EINVAL, "tiles of"), (dict(n=0), EINVAL, "n=0"),
    (dict(k=131072, ldc=1 << 20), EUNSUPPORTED, "k=131072"), (dict(count=-1), EINVAL, "count=-1"),
])
def test_packing_says_what_it_refuses(lib, bad, code, text):
    need = lib.dspk_i8_tiled_bytes(100, 130, 2)
    assert need == 2 * 7 * 4 * 1024 and lib.dspk_i8_tiled_bytes(1, 1, 1) == 2048
    a = dict(c=P + 1, ldc=130, n=100, k=130, count=2, t=2 * P, b=0)
    a.update(bad)
    got = lib.dspk_i8_pack(a["c"], a["ldc"], a["n"], a["k"], a["count"], a["t"], need + a["b"], None)
    _refused(lib, "dspk_i8_pack", got, code, text)


@pytest.mark.parametrize("n,k,count", [(0, 1, 1), (1, 0, 1), (1, 1, 0), (-5, 64, 1), (64, 131072, 1)])
def test_sizes_without_a_layout(lib, n, k, count):
    assert lib.dspk_i8_tiled_bytes(n, k, count) == 0


@pytest.mark.parametrize("bad,code,text", [
    (dict(m=65), EINVAL, "m=65"), (dict(m=-1), EINVAL, "m=-1"), (dict(experts=0), EINVAL, "experts=0"),
    (dict(experts=1025), EINVAL, "experts=1025"), (dict(top=0), EINVAL, "top_k=0"), (dict(top=33), EINVAL, "top_k=33"),
    (dict(top=9), EINVAL, "top_k=9 of 8"), (dict(k=0), EINVAL, "k=0"), (dict(norm=2), EINVAL, "normalize=2"),
    (dict(x=None), EINVAL, "x must be"), (dict(ldx=100), EINVAL, "of x"), (dict(r=P + 2), EINVAL, "router must be"),
    (dict(ldr=60), EINVAL, "of router"), (dict(ids=None), EINVAL, "ids or weights"), (dict(wt=P + 2), EINVAL, "ids or weights"),
    (dict(z=P + 1), EINVAL, "scores misaligned"), (dict(lds=7), EINVAL, "lds=7"), (dict(ws=None), EINVAL, "workspace of"),
    (dict(ws=P + 16), EINVAL, "workspace of"), (dict(wsb=1000), EINVAL, "workspace of"),
])
def test_router_says_what_it_refuses(lib, bad, code, text):
    a = dict(x=P, ldx=104, r=2 * P, ldr=104, m=3, k=100, experts=8, top=2, norm=1, ids=3 * P, wt=4 * P, z=5 * P, lds=8,
             ws=6 * P, wsb=1 << 20)
    call = lambda a: lib.dspk_moe_route(a["x"], a["ldx"], a["r"], a["ldr"], a["m"], a["k"], a["experts"], a["top"], a["norm"],
                                        a["ids"], a["wt"], a["z"], a["lds"], a["ws"], a["wsb"], None)
    assert call(dict(a, m=0)) == 0
    _refused(lib, "dspk_moe_route", call(dict(a, **bad)), code, text)


def _moe(lib, gate=None, up=None, down=None, x=3 * P, ldx=144, xs=4 * P, m=3, ids=5 * P, wt=6 * P, top=2, y=7 * P, dt=0,
         ldy=130, ws=8 * P, wsb=1 << 28):
    big = dict(n=100, k=130, count=8)
    w = [None if b == "none" else ctypes.byref(_weight(**dict(a, **(b or {}))))
         for a, b in ((big, gate), (big, up), (dict(n=130, k=100, count=8), down))]
    return lib.dspk_moe_mlp(*w, x, ldx, xs, m, ids, wt, top, y, dt, ldy, ws, wsb, None)


@pytest.mark.parametrize("bad,code,text", [(dict([(w, b)]), c, t) for w in ("gate", "up", "down") for b, c, t in WEIGHT] + [
    (dict(gate="none"), EINVAL, "gate is NULL"), (dict(up="none"), EINVAL, "up is NULL"),
    (dict(down="none"), EINVAL, "down is NULL"), (dict(up=dict(n=101)), EINVAL, "different sizes"),
    (dict(up=dict(k=131)), EINVAL, "different sizes"), (dict(up=dict(count=7)), EINVAL, "different sizes"),
    (dict(down=dict(n=100)), EINVAL, "different sizes"), (dict(down=dict(k=130)), EINVAL, "different sizes"),
    (dict(down=dict(count=9)), EINVAL, "different sizes"), (dict(m=65), EINVAL, "m=65"), (dict(top=33), EINVAL, "top_k=33"),
    (dict(gate=dict(count=1025), up=dict(count=1025), down=dict(count=1025)), EINVAL, "experts=1025"),
    (dict(x=None), EINVAL, "x must be"), (dict(ldx=130), EINVAL, "of x"), (dict(xs=None), EINVAL, "the scales of x"),
    (dict(ids=None), EINVAL, "ids or weights"), (dict(wt=None), EINVAL, "ids or weights"), (dict(y=None), EINVAL, "y NULL"),
    (dict(ldy=129), EINVAL, "ldy=129"), (dict(dt=7), EINVAL, "element type 7"), (dict(ws=None), EINVAL, "workspace of"),
    (dict(ws=8 * P + 8), EINVAL, "workspace of"), (dict(wsb=4096), EINVAL, "workspace of"),
])
def test_experts_say_what_they_refuse(lib, bad, code, text):
    assert _moe(lib, m=0) == 0
    _refused(lib, "dspk_moe_mlp", _moe(lib, **bad), code, text)


def test_the_expert_workspace_asked_for_is_the_one_that_is_checked(lib):
    need = lib.dspk_moe_workspace_bytes(130, 100, 8, 3, 2)
    _refused(lib, "dspk_moe_mlp", _moe(lib, wsb=need - 1), EINVAL, f"workspace of {need} bytes")
    for bad in ((0, 100, 8, 3, 2), (130, 0, 8, 3, 2), (130, 100, 0, 3, 2), (130, 100, 1025, 3, 2), (130, 100, 8, 0, 2),
                (130, 100, 8, 65, 2), (130, 100, 8, 3, 0), (130, 100, 8, 3, 33), (131072, 100, 8, 3, 2), (130, 131072, 8, 3, 2)):
        assert lib.dspk_moe_workspace_bytes(*bad) == 0


# ------------------------------------------------------ the binding's own checks
def _t(*z, dtype=torch.bfloat16):
    return torch.zeros(z, dtype=dtype)


I8, F32 = torch.int8, torch.float32


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int32, torch.int8])
def test_rows_of_other_types_are_refused(dtype):
    good, bad, c, s = _t(3, 64), _t(3, 64, dtype=dtype), _t(3, 64, dtype=I8), _t(3, dtype=F32)
    for name, call in (
        ("x", lambda: binding.add_rmsnorm(bad, good, good, None, 3, 64, out=good)),
        ("residual", lambda: binding.add_rmsnorm(good, bad, None, None, 3, 64, out=good)),
        ("residual_out", lambda: binding.add_rmsnorm(good, good, bad, None, 3, 64, out=good)),
        ("out", lambda: binding.add_rmsnorm(good, good, good, None, 3, 64, out=bad)),
        ("gate", lambda: binding.silu_mul(bad, good, 3, 64, out=good)),
        ("up", lambda: binding.silu_mul(good, bad, 3, 64, out=good)),
        ("x", lambda: binding.i8_quantize(bad, 3, 64, c, s)),
        ("y", lambda: binding.i8_read(c, s, 3, 64, bad)),
    ):
        with pytest.raises(ValueError, match=f"^{name}: expected float32 or bf16 rows"):
            call()


@pytest.mark.parametrize("name,call", [
    ("out", lambda: binding.add_rmsnorm(_t(3, 64), None, None, None, 3, 64, out=_t(3, 64, dtype=F32))),
    ("residual and residual_out", lambda: binding.add_rmsnorm(None, _t(3, 64), _t(3, 64, dtype=F32), None, 3, 64, out=_t(3, 64))),
    ("gate and up", lambda: binding.silu_mul(_t(3, 64), _t(3, 64, dtype=F32), 3, 64, out=_t(3, 64))),
    ("codes", lambda: binding.i8_quantize(_t(3, 64), 3, 64, _t(3, 64, dtype=torch.uint8), _t(3, dtype=F32))),
    ("codes", lambda: binding.i8_quantize(_t(3, 64), 3, 64, _t(3, 64, dtype=I8), None)),
    ("codes", lambda: binding.i8_quantize(_t(3, 64), 3, 64, _t(2, 64, dtype=I8), _t(3, dtype=F32))),
    ("codes", lambda: binding.i8_quantize(_t(3, 64), 3, 64, _t(3, 48, dtype=I8), _t(3, dtype=F32))),
    ("the scales of codes", lambda: binding.i8_quantize(_t(3, 64), 3, 64, _t(3, 64, dtype=I8), _t(2, dtype=F32))),
    ("the scales of codes", lambda: binding.i8_quantize(_t(3, 64), 3, 64, _t(3, 64, dtype=I8), _t(3, dtype=torch.float64))),
    ("scales", lambda: binding.silu_mul(_t(3, 64), _t(3, 64), 3, 64, out=_t(3, 64), scales=_t(3, dtype=F32))),
    ("x", lambda: binding.i8_quantize(_t(2, 64), 3, 64, _t(3, 64, dtype=I8), _t(3, dtype=F32))),
    ("x", lambda: binding.i8_quantize(_t(3, 32), 3, 64, _t(3, 64, dtype=I8), _t(3, dtype=F32))),
    ("weight", lambda: binding.add_rmsnorm(_t(3, 64), None, None, _t(64), 3, 64, out=_t(3, 64))),
    ("weight", lambda: binding.add_rmsnorm(_t(3, 64), None, None, _t(63, dtype=F32), 3, 64, out=_t(3, 64))),
    ("codes", lambda: binding.Int8Weight(_t(4, 64), _t(4, dtype=F32))),
    ("codes", lambda: binding.Int8Weight(_t(4, dtype=I8), _t(4, dtype=F32))),
    ("codes", lambda: binding.Int8Weight(_t(64, 4, dtype=I8).t(), _t(4, dtype=F32))),
    ("codes", lambda: binding.Int8Weight(_t(4, 5, 64, dtype=I8)[:, :4], _t(4, 4, dtype=F32))),
    ("scales", lambda: binding.Int8Weight(_t(4, 64, dtype=I8), _t(5, dtype=F32))),
    ("scales", lambda: binding.Int8Weight(_t(4, 64, dtype=I8), _t(4, dtype=torch.float64))),
    ("x and router", lambda: binding.moe_route(_t(3, 64, dtype=F32), _t(8, 64), 3, _t(3, 2, dtype=torch.int32), _t(3, 2, dtype=F32), _t(9, dtype=torch.uint8))),
    ("ids", lambda: binding.moe_route(_t(3, 64), _t(8, 64), 3, _t(2, 2, dtype=torch.int32), _t(3, 2, dtype=F32), _t(9, dtype=torch.uint8))),
    ("ids", lambda: binding.moe_route(_t(3, 64), _t(8, 64), 3, _t(3, 2, dtype=torch.int64), _t(3, 2, dtype=F32), _t(9, dtype=torch.uint8))),
    ("weights", lambda: binding.moe_route(_t(3, 64), _t(8, 64), 3, _t(3, 2, dtype=torch.int32), _t(3, 1, dtype=F32), _t(9, dtype=torch.uint8))),
    ("scores", lambda: binding.moe_route(_t(3, 64), _t(8, 64), 3, _t(3, 2, dtype=torch.int32), _t(3, 2, dtype=F32), _t(9, dtype=torch.uint8), scores=_t(3, 8))),
])
def test_the_binding_says_what_it_refuses(name, call):
    with pytest.raises(ValueError, match=f"^{name}: "):
        call()
