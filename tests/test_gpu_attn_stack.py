"""Stacks whose rounds are trees: rounds that follow one another without a new tree."""
import pytest

from attnutil import i32
from oracle import attention as oa
from speculative_decoding_verify_dspk_amd.verify_round import VerifyStack

pytestmark = pytest.mark.gpu


def _stack(context, m, room=0):
    st = VerifyStack("qwen3-4b", 1, 8, m, seed="attn-tree")
    st.attach_cache(context, room=room)
    return st


def test_rounds_of_one_tree_follow_the_cached_length():
    """One tree for several rounds: after a commit the next rows' positions count
    from the new length."""
    import torch
    m, par, n = 5, [0, 0, 1, 3], 90
    st = _stack(n, m, room=20)
    st.set_tree(i32(par), m)
    for kept in ([0, 1, 3], [0, 2], [0, 1, 3, 4]):
        masks, pos = oa.tree_layout(par, n)
        torch.cuda.synchronize()
        assert st.positions[0].tolist() == pos and st.tree_mask[0].tolist() == masks
        st.launch_layers(m)
        st.launch_commit(i32([kept + [-1] * (m - len(kept))]), i32([len(kept)]), m)
        n += len(kept)
    torch.cuda.synchronize()
    assert st.cache_len.tolist() == [n] and st.positions[0].tolist() == oa.tree_layout(par, n)[1]


def test_trees_that_do_not_fit_the_stack_are_refused():
    st = VerifyStack("qwen3-4b", 1, 8, 4, seed="attn-tree")
    with pytest.raises(ValueError, match="attach_cache"):
        st.set_tree(i32([0]), 2)
    st.attach_cache(10)
    with pytest.raises(ValueError, match="stack of 4 rows"):
        st.set_tree(i32([0, 1, 2, 3]), 5)
    with pytest.raises(ValueError, match="parents"):
        st.set_tree(i32([0]), 4)
    assert st.tree_mask is None
