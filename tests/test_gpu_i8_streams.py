"""8-bit weights made on a stream other than the current one: neither stream's memory is
used before the other is done with it."""
import pytest

from speculative_decoding_verify_dspk_amd import binding

pytestmark = pytest.mark.gpu

COUNT, N, K = 3, 700, 2048


def _busy(stream):
    """Some tens of milliseconds of work."""
    import torch
    with torch.cuda.stream(stream):
        a = torch.ones(4096, 4096, device="cuda")
        b = torch.empty_like(a)
        for _ in range(20):
            torch.mm(a, a, out=b)


def _weights(seed):
    """Rows that quantize has to copy: the weights do not follow each other."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(COUNT, N + 5, K + 8, device="cuda").normal_(generator=g)[:, :N, :K]


def _junk():
    """Memory of the sizes that quantize uses for a while, if the allocator gives it out again."""
    import torch
    return [torch.full((COUNT * N, K), 77, dtype=torch.int8, device="cuda"), torch.full((COUNT * N, K), 5.0, device="cuda"),
            torch.full((COUNT * N,), 5.0, device="cuda")]


def test_temporaries_are_kept_until_the_side_stream_is_done():
    import torch
    w, side = _weights(1), torch.cuda.Stream()
    want = binding.Int8Weight.quantize(w)
    torch.cuda.synchronize()
    for _ in range(3):
        _busy(side)
        got = binding.Int8Weight.quantize(w, stream=side)
        junk = _junk()
        side.synchronize()
        assert torch.equal(got.tiles, want.tiles) and torch.equal(got.scales, want.scales)
        del got, junk


def test_codes_may_be_released_at_once():
    import torch
    side = torch.cuda.Stream()
    codes = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    scales = torch.rand(N, device="cuda")
    want = binding.Int8Weight(codes, scales)
    torch.cuda.synchronize()
    for _ in range(3):
        _busy(side)
        mine = codes.clone()
        got = binding.Int8Weight(mine, scales, stream=side)
        del mine
        junk = torch.full((N, K), 77, dtype=torch.int8, device="cuda")
        side.synchronize()
        assert torch.equal(got.tiles, want.tiles)
        del got, junk


def test_the_side_stream_waits_for_the_current_one():
    """For rows that are still being written, and for readers of memory that it is given."""
    import torch
    w, side = _weights(2), torch.cuda.Stream()
    want = binding.Int8Weight.quantize(w)
    late = torch.zeros_like(w)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.zeros(want.tiles.numel(), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    _busy(torch.cuda.current_stream())
    late.copy_(w)
    read = old.clone()
    del old                                        # the tiles may come to lie here
    got = binding.Int8Weight.quantize(late, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got.tiles, want.tiles) and torch.equal(got.scales, want.scales)
    assert not read.any()
