"""A W4Weight laid out on one stream and used on another."""

import pytest

pytestmark = pytest.mark.gpu


def _lib():
    import torch
    from speculative_drafting_expand_gb300 import binding as B
    B.lib()
    return torch, B


@pytest.mark.parametrize("made", ["pack", "quantize", "pack under a stream"])
@pytest.mark.parametrize("given", [False, True])
def test_dropped_before_another_stream_has_read_it(made, given):
    """The product waits 50 ms, in which the weight's memory is freed and taken
    again on the stream that it was laid out on."""
    torch, B = _lib()
    n, k = 512, 1024
    g = torch.Generator(device="cuda").manual_seed(0)
    weight = torch.randn(n, k, generator=g, device="cuda")
    codes = torch.randint(256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand(n, k // 32, generator=g, device="cuda").bfloat16()
    x = torch.randn(3, k, generator=g, device="cuda")

    def make(stream):
        if made == "quantize":
            return B.W4Weight.quantize(weight, stream=stream)
        if made == "pack" or stream is None:
            return B.W4Weight(codes, scales, k, 32, stream=stream)
        with torch.cuda.stream(stream):
            return B.W4Weight(codes, scales, k, 32)

    want = B.pe_w4_linear(make(None), x)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w = make(side)
    nbytes = w.packed.numel()
    reader = other if given else torch.cuda.current_stream()
    reader.wait_stream(side)
    with torch.cuda.stream(reader):
        torch.cuda._sleep(100_000_000)
    y = B.pe_w4_linear(w, x, stream=other if given else None)
    del w
    with torch.cuda.stream(side):
        taken = [torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert all(bool((t == 7).all()) for t in taken)


def test_a_weight_used_where_it_was_made_is_reused_at_once():
    """Nothing waits for other streams: the memory of a dropped weight serves the
    next one of its size."""
    torch, B = _lib()
    weight = torch.randn(1024, 4096, device="cuda")
    x = torch.randn(2, 4096, device="cuda")
    places = set()
    for _ in range(4):
        w = B.W4Weight.quantize(weight)
        places.add(w.packed.data_ptr())
        B.pe_w4_linear(w, x)
        del w
    assert len(places) == 1
