"""Outputs that a call with stream= allocates itself: they come from that
stream's memory.  Memory of the current stream may still be written by work
queued there when the tensor that held it is already gone."""

import numpy as np
import pytest
import torch

from quantized_linear_gemm_b200 import inputs, lq

pytestmark = pytest.mark.gpu


def operands():
    M, N, K, E, k = 24, 512, 1024, 4, 2
    g = torch.Generator().manual_seed(1)
    x = inputs.activations(M, K, seed=1).cuda()
    w = inputs.weights(E * N, K, seed=2).cuda()
    B, s, _ = lq.quant_weight_int4(w, 128)
    q8, s8 = lq.quant_per_token("fp8_dynamic", w)
    a8, sa = lq.quant_per_token("fp8_dynamic", x)
    ids = torch.randint(0, E, (M, k), generator=g).cuda()
    off, order, slots = lq.moe_sort(ids, E)
    xs = lq.moe_permute(x, slots)
    xq, xsc = lq.moe_permute_quant("fp8_dynamic", x, slots)
    wt = torch.rand((M, k), generator=g).cuda()
    B3, s3 = B.view(E, N, -1), s.view(E, N, -1)
    return {
        "int4_mm": lambda **kw: lq.int4_mm(x, B, s, **kw),
        "grouped_int4_mm": lambda **kw: lq.grouped_int4_mm(xs, B3, s3, off, **kw),
        "quant_weight_int4": lambda **kw: lq.quant_weight_int4(w, 64, True, **kw),
        "moe_sort": lambda **kw: lq.moe_sort(ids, E, **kw),
        "moe_permute": lambda **kw: lq.moe_permute(x, slots, **kw),
        "moe_permute_quant": lambda **kw: lq.moe_permute_quant("w8a8_int8", x, slots, **kw),
        "moe_unpermute": lambda **kw: lq.moe_unpermute(xs, slots, wt, **kw),
        "moe_unpermute_backward": lambda **kw: lq.moe_unpermute_backward(x, xs, slots, wt, **kw),
        "scaled_mm": lambda **kw: lq.scaled_mm("fp8_dynamic", a8, sa, q8[:N], s8[:N], **kw),
        "grouped_scaled_mm": lambda **kw: lq.grouped_scaled_mm("fp8_dynamic", xq, xsc, q8.view(E, N, K),
                                                               s8.view(E, N), off, **kw),
        "quant_per_token": lambda **kw: lq.quant_per_token("fp8_dynamic", x, **kw),
        "silu_and_mul": lambda **kw: lq.silu_and_mul_dynamic_per_token_quant("fp8_dynamic", x, **kw),
    }


NAMES = ("int4_mm", "grouped_int4_mm", "quant_weight_int4", "moe_sort", "moe_permute", "moe_permute_quant",
         "moe_unpermute", "moe_unpermute_backward", "scaled_mm", "grouped_scaled_mm", "quant_per_token", "silu_and_mul")


def listed(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_do_not_take_memory_that_is_still_written(cuda_device, name):
    call = operands()[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in listed(call())]
    call(stream=side)                                            # loaded, and its memory known
    busy = torch.zeros(1 << 28, dtype=torch.bfloat16, device="cuda")
    sink = torch.empty_like(busy)
    sizes = sorted({t.numel() * t.element_size() for t in want} |
                   {sum(t.numel() * t.element_size() for t in want)})
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(60):
        sink.copy_(busy)                                         # the current stream is busy for about ten milliseconds
    left = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x55) for n in sizes for _ in range(4)]
    del left                                                     # free for the current stream, written after the copies
    out = listed(call(stream=side))
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert np.array_equal(a.view(torch.uint8).cpu().numpy(), b.view(torch.uint8).cpu().numpy())


@pytest.mark.parametrize("name", ["int4_mm", "moe_unpermute", "scaled_mm"])
def test_outputs_read_on_the_current_stream_are_not_handed_out_before(cuda_device, name):
    """An output is read on the current stream, behind other work there, and dropped: the next call's output on
    the side stream does not take its memory while that read is still to come."""
    call = operands()[name]
    side = torch.cuda.Stream()
    want = call().clone()
    call(stream=side)
    got = torch.zeros_like(want)
    junk = torch.full_like(want, 7.0)
    busy = torch.zeros(1 << 28, dtype=torch.bfloat16, device="cuda")
    sink = torch.empty_like(busy)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    out = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(60):
        sink.copy_(busy)
    got.copy_(out)
    del out
    with torch.cuda.stream(side):                                # as large as the output, written at once
        over = [torch.empty_like(want) for _ in range(4)]
        for t in over:
            t.copy_(junk)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("name", ["int4_mm", "moe_sort", "moe_unpermute_backward", "scaled_mm"])
def test_captured_on_a_forked_stream(cuda_device, name):
    """A call on a side stream that joins a capture, its outputs allocated inside it: replayed twice."""
    call = operands()[name]
    want = [t.clone() for t in listed(call())]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    call(stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        out = listed(call(stream=side))
        again = listed(call(stream=side))
        main.wait_stream(side)
    for _ in range(2):
        for t in out + again:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for got in (out, again):
            for a, b in zip(got, want):
                assert np.array_equal(a.view(torch.uint8).cpu().numpy(), b.view(torch.uint8).cpu().numpy())


def test_no_tokens_on_a_side_stream(cuda_device):
    """Empty outputs."""
    side = torch.cuda.Stream()
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    assert lq.moe_permute(x, slots, stream=side).shape == (0, 64)
    assert lq.moe_unpermute(x, slots, stream=side).shape == (0, 64)
    off, order, got = lq.moe_sort(slots, 3, stream=side)
    side.synchronize()
    assert torch.all(off == 0) and order.numel() == 0 and got.shape == (0, 2)
