"""The binding's check that weights lie as the ids of a choice do (no GPU)."""
import pytest
import torch

from speculative_decoding_verify_dspk_amd import binding


@pytest.fixture
def sent(monkeypatch):
    """The calls that pass the binding's checks, and their arguments."""
    calls = []

    class Recorder:
        def __init__(self, name, *args):
            calls.append((name, args))

        def __call__(self):
            pass

        def holding(self, *_):
            return self

    monkeypatch.setattr(binding, "Prepared", Recorder)
    monkeypatch.setattr(binding, "_stream", lambda s: None)
    return calls


def _calls(ids, wt):
    bf = lambda *z: torch.zeros(z, dtype=torch.bfloat16)
    ws = torch.zeros(9, dtype=torch.uint8)
    weight = type("W", (), dict(k=64, n=32, count=8, desc=binding.Int8WeightDesc()))
    moe = binding.MoEWeights(weight, weight, weight)
    x8 = torch.zeros(3, 64, dtype=torch.int8)
    return (lambda: binding.moe_route(bf(3, 64), bf(8, 64), 3, ids, wt, ws),
            lambda: binding.moe_mlp(moe, x8, torch.zeros(3), 3, ids, wt, torch.zeros(3, 64), ws))


@pytest.mark.parametrize("shape", [(3, 3), (2, 3), (3, 4), (1, 6), (3, 2, 3)])
def test_weights_of_another_width_are_refused(sent, shape):
    ids, wt = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(shape)
    for call in _calls(ids, wt):
        with pytest.raises(ValueError, match="^weights: "):
            call()
    assert not sent


@pytest.mark.parametrize("shape", [(3, 2), (5, 2), (6,), (7,), (6, 1), (3, 1, 2)])
def test_weights_like_the_ids_or_flat_are_taken(sent, shape):
    ids, wt = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(shape)
    for call in _calls(ids, wt):
        call()
    assert [name for name, _ in sent] == ["dspk_moe_route", "dspk_moe_mlp"]
    assert all(ids.data_ptr() in args and wt.data_ptr() in args and 2 in args for _, args in sent)
