"""A group-quantised weight packed on a stream other than the current one: neither stream's
memory is used before the other is done with it."""
import numpy as np
import pytest

from speculative_decoding_verify_dspk_amd import binding, inputs

pytestmark = pytest.mark.gpu


def _busy(stream):
    """Some tens of milliseconds of work."""
    import torch
    with torch.cuda.stream(stream):
        a = torch.ones(4096, 4096, device="cuda")
        b = torch.empty_like(a)
        for _ in range(20):
            torch.mm(a, a, out=b)


@pytest.mark.parametrize("bits", [4, 16])
def test_a_weight_packed_on_a_side_stream(bits):
    import torch
    n, k, side = 1000, 2048, torch.cuda.Stream()
    w = inputs.make_qweight(n, k, bits, "streams")
    want = binding.DeviceQWeight.upload(w)
    host = [w.codes.view(np.int32 if bits != 16 else np.int16)] + ([] if bits == 16 else
                                                                   [a.view(np.int16) for a in (w.scales, w.biases)])
    sources = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in host]
    torch.cuda.synchronize()
    for _ in range(3):
        late = [torch.zeros_like(t) for t in sources]
        _busy(torch.cuda.current_stream())
        old = torch.zeros_like(want.tiles)
        read = old.clone()
        for a, b in zip(late, sources):
            a.copy_(b)                               # still on their way
        del old                                      # the tiles may come to lie here
        _busy(side)
        got = binding.DeviceQWeight(n, k, bits, *late, stream=side)
        shapes = [(t.shape, t.dtype) for t in late]
        del late, a                                  # released while the packing waits
        junk = [torch.full(z, 7, dtype=t, device="cuda") for z, t in shapes]
        torch.cuda.synchronize()
        assert torch.equal(got.tiles, want.tiles) and not read.any()
        del got, junk
