"""Where the 4-bit product keeps its weights exact and where it rounds them, on
every branch of the choice between its kernels.

The streaming kernel (up to 8 tokens, 16 rows of a grouped call) multiplies
exact codes and applies the scales in fp32: with any scales its error is that
of fp32 sums and of C's rounding, without the allowance for weights rounded to
bf16 (limit() of test_gpu_int4.py).  The tensor-core kernel rounds a weight
once, which scales that are powers of two make exact."""

import numpy as np
import pytest
import torch

from oracle import int4_oracle as I
from quantized_linear_gemm_b200 import inputs, lq

from test_gpu_int4 import check, dev, weight

pytestmark = pytest.mark.gpu


def dense(M, N, K, group, zeros, pow2, rounded):
    x = inputs.activations(M, K, seed=M)
    B, s, z = weight(N, K, group, zeros, seed=N + K, pow2=pow2)
    C = lq.int4_mm(x.cuda(), dev(B), dev(s, torch.bfloat16), b_zeros=dev(z))
    torch.cuda.synchronize()
    assert lq.device_status(0) == 0
    r, mag = I.int4_mm_ref(x.float().numpy(), B, s, z)
    check(C, r, mag, K, rounded, what=(M, N, K, group, zeros))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M", [1, 5, 8])
def test_few_tokens_are_exact(cuda_device, M, group, zeros):
    dense(M, 264, 1152, group, zeros, pow2=False, rounded=False)


@pytest.mark.parametrize("group,zeros", [(128, False), (128, True), (32, False), (32, True)])
@pytest.mark.parametrize("M", [1, 8])
def test_wide_layers_are_exact(cuda_device, M, group, zeros):
    """32-row tiles, the last one ragged."""
    dense(M, 16384 + 8, 384, group, zeros, pow2=False, rounded=False)


@pytest.mark.parametrize("group,zeros", [(128, True), (64, False), (32, True)])
@pytest.mark.parametrize("M", [1, 8])
@pytest.mark.parametrize("N,K", [(72, 16384 + 128), (16384 + 8, 384)])
@pytest.mark.parametrize("pow2", [True, False])
def test_long_rows_and_wide_layers(cuda_device, M, group, zeros, N, K, pow2):
    """Few tokens on both sides of the limits on K and N: within the documented rounding of the weights, and
    exact where the scales make that rounding nothing."""
    dense(M, N, K, group, zeros, pow2=pow2, rounded=not pow2)


@pytest.mark.parametrize("group,zeros", [(128, False), (64, True), (32, True)])
@pytest.mark.parametrize("counts", [[0, 9, 1, 0, 6], [16, 0], [1] * 16])
def test_few_grouped_rows_are_exact(cuda_device, counts, group, zeros):
    E, N, K, T = len(counts), 72, 384, sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x = inputs.activations(T, K, seed=T)
    B, s, z = weight(E * N, K, group, zeros, seed=E)
    B, s = B.reshape(E, N, -1), s.reshape(E, N, -1)
    z = None if z is None else z.reshape(E, N, -1)
    C = lq.grouped_int4_mm(x.cuda(), dev(B), dev(s, torch.bfloat16), dev(off), b_zeros=dev(z))
    torch.cuda.synchronize()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            r, mag = I.int4_mm_ref(x[lo:hi].float().numpy(), B[e], s[e], None if z is None else z[e])
            check(C[lo:hi], r, mag, K, False, what=e)
