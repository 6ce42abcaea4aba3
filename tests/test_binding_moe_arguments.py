"""Outputs of the token calls that are no tensors or have the wrong number of
dimensions: refused like every other argument (TypeError, ValueError), before
the C call."""

import types

import pytest
import torch

from quantized_linear_gemm_b200 import lq

S = types.SimpleNamespace(cuda_stream=0)


class _NoCall:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was called")


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    monkeypatch.setattr(lq, "_DEVICE_TYPE", "cpu")
    monkeypatch.setattr(lq, "lib", _NoCall)


X, SLOTS = torch.zeros((5, 64), dtype=torch.bfloat16), torch.zeros((5, 2), dtype=torch.int32)
NOT_TENSORS = ([[0.0] * 64], "rows", 3)


@pytest.mark.parametrize("bad", NOT_TENSORS)
def test_no_tensor(bad):
    for call in (lambda: lq.moe_permute(X, SLOTS, xs=bad, stream=S),
                 lambda: lq.moe_permute_quant("fp8_dynamic", X, SLOTS, q=bad, stream=S),
                 lambda: lq.grouped_int4_mm(X, bad, X, SLOTS, stream=S)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("shape", [(), (640,), (10, 64, 1)])
def test_wrong_dimensions(shape):
    for call in (lambda: lq.moe_permute(X, SLOTS, xs=torch.zeros(shape, dtype=torch.bfloat16), stream=S),
                 lambda: lq.moe_permute_quant("fp8_dynamic", X, SLOTS, q=torch.zeros(shape, dtype=torch.uint8), stream=S)):
        with pytest.raises(ValueError):
            call()
