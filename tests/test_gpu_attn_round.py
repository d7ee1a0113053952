"""Verify rounds with attention: projections, norm + rotation + store,
attention, o, head, acceptance along a tree and the commit, as one stack."""
import numpy as np
import pytest

import oracle
from attnutil import ABS, REL, chain_masks, i32
from gpuutil import assert_rows_close, oracle_columns
from oracle import attention as oa
from speculative_decoding_verify_dspk_amd import binding, inputs
from speculative_decoding_verify_dspk_amd.verify_round import HEAD_DIM, VerifyStack

pytestmark = pytest.mark.gpu


def _entries(st, li, n):
    """The first n cached k and v of a layer, as the library reads them back."""
    import torch
    k, v = (torch.empty((n, st.kvdim), device="cuda") for _ in range(2))
    binding.kv_read(st.caches[li], binding.AttnBatch(i32([0]), st.page_table, n), k, v)
    return (x.cpu().numpy().reshape(n, st.kv_heads, HEAD_DIM) for x in (k, v))


def _check_attention(st, m, n, masks, pos):
    """The last layer's q/k/v rows (on the device) against the reference."""
    q, k, v = (y[:m].cpu().numpy().reshape(m, -1, HEAD_DIM) for y in st.y_qkv)
    li, f = st.n_layers - 1, st.inv_freq.cpu().numpy()
    wq = oa.norm_rotate(q, st.q_norm[li].cpu().numpy(), st.eps, f, pos)
    got_q = st.q_rot[:m].float().cpu().numpy().reshape(q.shape)
    assert (np.abs(got_q - wq) <= REL * np.abs(wq) + 2.0 ** -18 * np.abs(wq).max(-1, keepdims=True)).all()
    wk = oa.norm_rotate(k, st.k_norm[li].cpu().numpy(), st.eps, f, pos)
    ks, vs = _entries(st, li, n + m)
    step = 254 if st.caches[li].bits == 8 else 2 / REL / 2
    for held, want in ((ks[n:], wk), (vs[n:], v)):
        assert (np.abs(held - want) <= np.abs(want).max(-1, keepdims=True) * (1 / step + 2.0 ** -17)).all()
    ref, mag = oa.attention(got_q, ks, vs, n, masks, HEAD_DIM ** -0.5)
    out = st.attn_out[:m].float().cpu().numpy().reshape(q.shape)
    assert (np.abs(out - ref) <= REL * np.abs(ref) + ABS * mag).all()


@pytest.mark.parametrize("kv_bits", [16, 8])
def test_rounds_of_a_chain_and_of_a_tree(kv_bits):
    """A chain's round, then two rounds of a tree whose accepted path is moved
    together: every part against its reference, and the second tree round sees
    the first one's accepted entries where the commit has put them."""
    import torch
    st = VerifyStack("qwen3-4b", 2, 8, 9, seed="attn")
    st.attach_cache(150, kv_bits, room=8)
    n, m = 150, 6
    st.launch_layers(m)
    torch.cuda.synchronize()
    _check_attention(st, m, n, chain_masks(m), np.arange(n, n + m))
    # o reads the attention's rows
    cols = np.arange(0, st.hidden, 97)
    o = inputs.make_qweight_device(st.hidden, st.qdim, 8, st.model, st.seed, 0, 1, "o")
    w = inputs.QWeight(st.hidden, st.qdim, 8, *(x.cpu().numpy().view(t) for x, t in
                                               zip(o, (np.uint32, np.uint16, np.uint16))), None)
    rows = st.attn_out[:m].view(torch.int16).cpu().numpy().view(np.uint16)
    assert_rows_close(st.y_o[:m].cpu().numpy()[:, cols], oracle_columns(w, rows, cols), what="o")

    m, par = 9, [0, 0, 1, 1, 2, 4, 4, 6]
    parents = i32(par)
    new = lambda *z: torch.empty(z, dtype=torch.int32, device="cuda")
    al, com, path = new(1), new(1, m), new(1, m)
    for rnd in range(2):
        st.set_tree(parents, m)
        st.launch_layers(m)
        st.launch_head(m)
        torch.cuda.synchronize()
        masks, pos = oa.tree_layout(par, n)
        _check_attention(st, m, n, masks, np.array(pos))
        before = [_entries(st, li, n + m) for li in range(2)]
        before = [[x.copy() for x in e] for e in before]
        # drafts that follow the head's tokens down to node 6, then part from them
        t = st.argmax[:m].tolist()
        draft = [t[p] if j in (1, 4, 6) else t[p] + 1 for j, p in enumerate(par, 1)]
        binding.accept_tree_greedy(st.argmax, i32(draft), parents, 1, m, al, com, path)
        st.launch_commit(path, al, m)
        torch.cuda.synchronize()
        want = oa.accept_tree_greedy(t, draft, par)
        assert want[2] == [0, 1, 4, 6]
        assert al.tolist() == [4] and path[0, :4].tolist() == want[2] and com[0, :4].tolist() == want[1]
        assert st.cache_len.tolist() == [n + 4]
        for li in range(2):
            for a, b in zip(_entries(st, li, n + 4), before[li]):
                assert np.array_equal(a[:n], b[:n]) and np.array_equal(a[n:], b[n + np.array(want[2])])
        n += 4


def test_captured_rounds_equal_eager_ones():
    """A round with attention captured into graphs and replayed with eager work
    in between gives the eager round's bits; prepared calls too."""
    import torch
    m = 8
    st = VerifyStack("qwen3-4b", 2, 8, m, seed="attn-graph")
    st.attach_cache(700, 8)
    st.set_tree(i32([0, 0, 1, 1, 2, 3, 3]), m)
    d = torch.zeros((1, m - 1), dtype=torch.int32, device="cuda")
    al, com = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty((1, m), dtype=torch.int32, device="cuda")
    st.launch_layers(m)
    st.launch_head(m)
    torch.cuda.synchronize()
    outs = lambda: [x.clone() for x in [st.q_rot, st.attn_out, st.y_o, st.argmax] + [c.k for c in st.caches]]
    want = outs()
    graphs = st.capture_round(m, 0, d, al, com)
    calls, head = st.prepare_round(m, 0)
    for rep in range(3):
        for x in (st.q_rot, st.attn_out, st.y_o):
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        if rep < 2:
            for g in graphs:
                g.replay()
        else:
            for c in calls:
                c()
            head()
        torch.cuda.synchronize()
        for a, b in zip(outs(), want):
            assert torch.equal(a, b), rep
        st.launch_layers(m)
        torch.cuda.synchronize()


def test_without_a_cache_the_stack_is_as_it_was():
    """A stack without a cache feeds o its own synthetic rows."""
    import torch
    st = VerifyStack("qwen3-4b", 1, 8, 4, seed="plain")
    st.launch_layers(4)
    torch.cuda.synchronize()
    y = st.y_o.clone()
    L = st.layers[0][0]
    binding.qgemm_verify(L.o, st.x_o, 4, st.y_o, st.ws_o)
    torch.cuda.synchronize()
    assert torch.equal(y, st.y_o)
