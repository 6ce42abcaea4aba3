"""The gradient that moe_unpermute_backward allocates and clears itself, on a
stream other than the current one."""

import pytest
import torch

from oracle import moe_tokens_oracle as T
from quantized_linear_gemm_b200 import inputs, lq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", ["stream", "external"])
def test_cleared_on_the_stream_of_the_call(cuda_device, handle):
    """The current stream is busy: clearing there would come after the kernel and wipe its rows."""
    tokens, k, H = 40, 4, 256
    slots = torch.arange(tokens * k, dtype=torch.int32).view(tokens, k)
    slots[::3, 1] = -1
    x, y = inputs.activations(tokens, H, seed=1), inputs.activations(tokens * k, H, seed=2)
    w = torch.rand((tokens, k), generator=torch.Generator().manual_seed(3))
    xd, yd, sd, wd = x.cuda(), y.cuda(), slots.cuda(), w.cuda()
    side = torch.cuda.Stream()
    given = side if handle == "stream" else torch.cuda.ExternalStream(side.cuda_stream)
    src = torch.zeros(1 << 28, dtype=torch.bfloat16, device="cuda")
    dst = torch.empty_like(src)
    lq.moe_unpermute_backward(xd, yd, sd, wd, stream=given)      # the kernel is loaded
    torch.cuda.synchronize()
    for _ in range(60):
        dst.copy_(src)                                           # about ten milliseconds of work
    dy, dw = lq.moe_unpermute_backward(xd, yd, sd, wd, stream=given)
    torch.cuda.synchronize()
    rdy, _, _ = T.unpermute_backward(x.float().numpy(), y.float().numpy(), slots.numpy(), w.numpy(),
                                     torch.zeros((tokens * k, H)).numpy())
    got = dy.double().cpu()
    # one fp32 product (2^-24) rounded to bf16 (half a step, 2^-8); zero rows exactly
    assert torch.all((got - torch.from_numpy(rdy)).abs() <= torch.from_numpy(rdy).abs() * (2.0 ** -8 + 2.0 ** -23))
