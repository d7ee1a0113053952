"""Rounds over 8-bit integer layers: every step of a layer against the oracle on
what the step before it wrote, captured rounds, trees, and rows that do not depend on
the rows verified with them."""
import numpy as np
import pytest

from attnutil import i32
from i8util import BF16, F32, assert_codes, bf16, host
from oracle import attention as oa
from oracle import layer8
from speculative_decoding_verify_dspk_amd import binding
from speculative_decoding_verify_dspk_amd.verify_round import Int8VerifyStack

pytestmark = pytest.mark.gpu

MODEL, NORM, SILU = "qwen3-4b", 32 * F32, 8 * F32        # the row kernels' tolerances
MIXTURE = dict(experts=16, top_k=4, expert_inter=768)


def _stack(layers=1, m=6, **options):
    return Int8VerifyStack(MODEL, layers, 8, m, seed="int8-stack", **options)


def _codes_of(w, g=0):
    """Codes [n][k] of a packed weight, by the documented index."""
    n, k = w.n, w.k
    t = w.tiles.cpu().numpy().view(np.int8).reshape(w.count, -(-n // 16), -(-k // 128) * 2, 4, 16, 16)[g]
    return t.transpose(0, 3, 1, 2, 4).reshape(t.shape[0] * 16, -1)[:n, :k]


def _product(rows8, w, g=0):
    """float(sum) * x_scale * w_scale in fp32: the definition's bits."""
    c, s = host(rows8[0]), host(rows8[1])
    sums = c.astype(np.float64) @ _codes_of(w, g).astype(np.float64).T       # exact: below 2^53
    return sums.astype(np.float32) * s[:, None] * host(w.scales).reshape(w.count, -1)[g][None]


def _take(rows8, m):
    return rows8[0][:m].clone(), rows8[1][:m].clone()


@pytest.mark.parametrize("options", [{}, MIXTURE])
@pytest.mark.parametrize("context", [None, 300])
def test_a_layer_step_by_step(options, context):
    """Each call's outputs from the inputs it was given, which are kept after each call."""
    import torch
    m = 5
    st = _stack(m=m, **options)
    if context is not None:
        st.attach_cache(context)
    L, keep = st.layers[0][0], []
    names = ("residual", "x8", "qkv", "o8", "y_o", "normed", "h8", "gate_up", "y_down")

    def snap():
        torch.cuda.synchronize()
        out = {}
        for n in names:
            v = getattr(st, n)
            out[n] = None if v is None else _take(v, m) if isinstance(v, tuple) else v[:m].clone()
        return out

    for call in st.layer_calls(0, m):
        call()
        keep.append((call.name, snap()))
    by = {}
    for name, v in keep:
        by.setdefault(name, []).append(v)
    # residual and first norm
    first = by["dspk_add_rmsnorm"][0]
    x = host(st.x_in[:m])
    assert np.array_equal(host(first["residual"]), x)
    y = layer8.add_rmsnorm(None, x, host(L.attn_norm), st.norm_eps)[1]
    assert_codes(host(first["x8"][0]), host(first["x8"][1]), y, NORM, "attention norm")
    assert np.array_equal(host(by["dspk_i8_gemm"][0]["qkv"]), _product(first["x8"], L.qkv))
    # the rows that o reads, its product, the residual's sum
    o_in = host((st.attn_out if context is not None else st.x_o)[:m])
    code, scale = oa.quantise_rows(o_in)
    got = by["dspk_i8_quantize"][0]["o8"]
    assert np.array_equal(host(got[0]), code) and np.array_equal(host(got[1]), scale)
    y_o = host(by["dspk_i8_gemm"][1]["y_o"])
    assert np.array_equal(y_o, _product(got, L.o))
    second = by["dspk_add_rmsnorm"][1]
    s, y = layer8.add_rmsnorm(y_o, x, host(L.mlp_norm), st.norm_eps)
    assert (np.abs(host(second["residual"]) - s) <= (F32 + BF16) * np.abs(s)).all()
    assert_codes(host(second["x8"][0]), host(second["x8"][1]), y, NORM, "MLP norm")
    if not options:
        wide = host(by["dspk_i8_gemm"][2]["gate_up"])
        assert np.array_equal(wide, bf16(_product(second["x8"], L.gate_up)))
        h = layer8.silu_mul(*np.split(wide, 2, axis=1))
        h8 = by["dspk_silu_mul"][0]["h8"]
        assert_codes(host(h8[0]), host(h8[1]), h, SILU, "activation")
        assert np.array_equal(host(by["dspk_i8_gemm"][3]["y_down"]), _product(h8, L.down))
    else:
        normed = host(second["normed"])
        assert (np.abs(normed - y) <= (NORM + BF16) * np.abs(y)).all()
        z = normed.astype(np.float64) @ host(L.router).astype(np.float64).T
        ids, wt = host(st.ids[:m]), host(st.expert_weights[:m])
        # a score is off by at most (k + 1) half steps of the sum of its products' magnitudes
        off = (st.hidden + 1) * F32 * (np.abs(normed) @ np.abs(host(L.router)).T)
        for i in range(m):
            rest = np.delete(np.arange(st.experts), ids[i])
            assert (z[i, ids[i]].min() >= z[i, rest] - off[i].max() * 2).all()
        # the experts' own tolerance, as in their tests
        c, sc = host(second["x8"][0]), host(second["x8"][1])
        w = [([_codes_of(q, e) for e in range(st.experts)], host(q.scales).reshape(st.experts, -1))
             for q in (L.moe.gate, L.moe.up, L.moe.down)]
        w = [(np.stack(a), b) for a, b in w]
        ref, slack = layer8.experts(c, sc, *w, ids, wt, 127 * 31 * F32)
        mag = sum(np.abs(layer8.experts(c, sc, *w, ids[:, j:j + 1], wt[:, j:j + 1], 0)[0]) for j in range(st.top_k))
        got = host(by["dspk_moe_mlp"][0]["y_down"])
        assert (np.abs(got - ref) <= slack + (20 + st.top_k) * F32 * mag).all()
    # the head's rows
    st.final_call(m)()
    torch.cuda.synchronize()
    y = layer8.add_rmsnorm(host(keep[-1][1]["y_down"]), host(keep[-1][1]["residual"]), host(st.final_norm), st.norm_eps)[1]
    assert (np.abs(host(st.h[:m]) - y) <= (NORM + BF16) * np.abs(y)).all()


@pytest.mark.parametrize("options", [{}, MIXTURE])
def test_rows_do_not_depend_on_the_rows_beside_them(options):
    """Without attention, whose splits go by its rows: a row verified with others is, bit
    for bit, the row computed alone, through two layers, norms and experts."""
    import torch
    m = 6
    st = _stack(2, m, **options)
    st.launch_layers(m)
    torch.cuda.synchronize()
    want = st.h[:m].clone()
    for i in range(m):
        x, o = st.x_in.clone(), st.x_o.clone()
        st.x_in[0], st.x_o[0] = x[i], o[i]
        st.launch_layers(1)
        torch.cuda.synchronize()
        assert torch.equal(st.h[0], want[i]), i
        st.x_in.copy_(x)
        st.x_o.copy_(o)


@pytest.mark.parametrize("options", [{}, MIXTURE])
def test_captured_rounds_of_trees(options):
    """Graphs of a round over two layers with caches: replays give what eager rounds
    give, with eager work between, and the committed path is the oracle's."""
    import torch
    m = 6
    st = _stack(2, m, **options)
    st.attach_cache(100, room=64)
    new = lambda *z: torch.zeros(z, dtype=torch.int32, device="cuda")
    draft, al, com = new(1, m - 1), new(1), new(1, m)
    par = [0, 0, 1, 2, 2]
    st.set_tree(i32(par), m)
    graphs = st.capture_round(m, 0, draft, al, com)
    for turn in range(3):
        st.launch_layers(m)
        st.launch_head(m)
        torch.cuda.synchronize()
        want, t = st.h[:m].clone(), st.argmax[:m].tolist()
        st.h.zero_()
        st.argmax.fill_(-1)
        for g in graphs[:2]:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(st.h[:m], want) and st.argmax[:m].tolist() == t
        d = [t[p] if j in (2, 5) else t[p] + 1 for j, p in enumerate(par, 1)]
        draft.copy_(i32([d]))
        graphs[2].replay()
        torch.cuda.synchronize()
        n, toks, path = oa.accept_tree_greedy(t, d, par)
        assert al.tolist() == [n] and com[0].tolist() == toks + [-1] * (m - n)
        st.launch_commit(st.path, al, m)
        torch.cuda.synchronize()
        assert st.cache_len.tolist() == [100 + n * (turn + 1)]
        st.x_in.copy_(torch.randn_like(st.x_in, dtype=torch.float32).bfloat16())


def test_sizes_and_refusals():
    st = _stack(1, 4)
    L = st.layers[0][0]
    assert st.layer_weight_bytes() == sum((w.k + 4) * w.n for w in (L.qkv, L.o, L.gate_up, L.down))
    for bad in (dict(experts=4, top_k=5, expert_inter=64), dict(experts=4, top_k=0, expert_inter=64),
                dict(experts=4, top_k=2)):
        with pytest.raises(ValueError, match="experts: "):
            _stack(1, 4, **bad)
    with pytest.raises(binding.DspkError, match="workspace of"):
        small = binding.alloc_workspace(0)
        mix = _stack(1, 4, **MIXTURE)
        binding.moe_mlp(mix.layers[0][0].moe, *mix.x8, 4, mix.ids, mix.expert_weights, mix.y_down, small)
