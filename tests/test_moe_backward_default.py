"""The gradient that moe_unpermute_backward allocates itself: rows that no slot
names have gradient zero.  The memory that the allocator hands out is filled
with NaN here, so that leaving a row out shows."""

import numpy as np
import pytest
import torch

from oracle import moe_tokens_oracle as T
from quantized_linear_gemm_b200 import lq


@pytest.fixture
def nan_memory():
    """torch.empty fills with NaN (the largest whole number for integers)."""
    before = torch.are_deterministic_algorithms_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    torch.use_deterministic_algorithms(True, warn_only=True)
    torch.utils.deterministic.fill_uninitialized_memory = True
    assert torch.isnan(torch.empty(1)).all()
    yield
    torch.use_deterministic_algorithms(before[0])
    torch.utils.deterministic.fill_uninitialized_memory = before[1]


class _Nothing:
    """A library whose calls do nothing: what the binding hands over is what comes back."""

    def __getattr__(self, name):
        return lambda *args: 0


def test_rows_without_a_slot_are_zero_before_the_call(monkeypatch, nan_memory):
    monkeypatch.setattr(lq, "_DEVICE_TYPE", "cpu")
    monkeypatch.setattr(lq, "lib", lambda: _Nothing())
    stream = type("S", (), {"cuda_stream": 0})()
    slots = torch.full((3, 2), -1, dtype=torch.int32)
    y, dout, w = torch.ones((6, 16)).bfloat16(), torch.ones((3, 16)).bfloat16(), torch.ones((3, 2))
    dy, _ = lq.moe_unpermute_backward(dout, y, slots, w, stream=stream)
    assert dy.shape == (6, 16) and torch.all(dy == 0)
    mine = torch.full((6, 16), 3.0).bfloat16()
    dy, _ = lq.moe_unpermute_backward(dout, y, slots, w, dy=mine, stream=stream)
    assert dy is mine and torch.all(dy == 3.0)                   # the caller's buffer is the caller's


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,k,H,extra", [(1, 8, 2048, 0), (37, 8, 272, 0), (20, 9, 1040, 5), (3, 0, 64, 4)])
def test_default_gradient_against_the_oracle(cuda_device, nan_memory, tokens, k, H, extra):
    """dy of a batch with dropped ids, and of a y with rows beyond the slots."""
    E, g = 19, np.random.default_rng(tokens)
    ids = np.stack([g.choice(E, size=k, replace=False) for _ in range(tokens)]).astype(np.int64).reshape(tokens, k)
    ids[g.random(ids.shape) < 0.4] = -1
    _, _, slots = T.moe_sort(ids, E)
    n = tokens * k + extra
    t = torch.Generator().manual_seed(H)
    y, dout = torch.randn((n, H), generator=t).bfloat16(), torch.randn((tokens, H), generator=t).bfloat16()
    w = torch.randn((tokens, k), generator=t)
    dy, dw = lq.moe_unpermute_backward(dout.cuda(), y.cuda(), torch.from_numpy(slots).cuda(), w.cuda())
    torch.cuda.synchronize()
    rdy, rdw, mag = T.unpermute_backward(dout.float().numpy(), y.float().numpy(), slots, w.numpy(), np.zeros((n, H)))
    got = dy.double().cpu().numpy()
    # one fp32 product (2^-24) rounded to bf16 (half a step, 2^-8); zero rows exactly
    assert np.all(np.abs(got - rdy) <= np.abs(rdy) * (2.0 ** -8 + 2.0 ** -23))
    # a sum of H fp32 multiply-adds: H 2^-23 of the terms' magnitudes
    assert np.all(np.abs(dw.cpu().numpy() - rdw) <= H * 2.0 ** -23 * mag)
