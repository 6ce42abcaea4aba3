"""Grouped 4-bit products with more experts than the tensor-core kernel keeps
(1024): the streaming kernel at any number of rows, with one and with two
8-token tiles per CTA.  Tolerances as in test_gpu_int4.py; scales are powers of
two and this kernel keeps the codes exact."""

import numpy as np
import pytest
import torch

from oracle import int4_oracle as I
from quantized_linear_gemm_b200 import inputs, lq

from test_gpu_int4 import check, dev, weight

pytestmark = pytest.mark.gpu


def run(E, N, K, group, zeros, counts, seed, sample=None):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T = int(off[-1])
    x = inputs.activations(T, K, seed=seed)
    B, s, z = weight(E * N, K, group, zeros, seed + 1, pow2=True)
    B, s = B.reshape(E, N, -1), s.reshape(E, N, -1)
    z = None if z is None else z.reshape(E, N, -1)
    C = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    lq.grouped_int4_mm(x.cuda(), dev(B), dev(s, torch.bfloat16), dev(off), b_zeros=dev(z), C=C[:T])
    torch.cuda.synchronize()
    assert torch.all(C[T:] == 7.0)
    for e in range(E) if sample is None else sample:
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            r, mag = I.int4_mm_ref(x[lo:hi].float().numpy(), B[e], s[e], None if z is None else z[e])
            check(C[lo:hi], r, mag, K, False, what=e)


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False)])
@pytest.mark.parametrize("rows", [3000, 10007])           # up to 8 and more than 8 rows per expert on average
def test_uneven_experts(cuda_device, rows, group, zeros):
    E = 1025
    g = np.random.default_rng(rows)
    share = g.gamma(0.5, 1.0, E)
    share[g.integers(0, E, 200)] = 0
    run(E, 40, 192, group, zeros, g.multinomial(rows, share / share.sum()), seed=rows)


def test_more_token_tiles_than_one_grid_axis(cuda_device):
    """1.1 million rows: 69,775 tiles of 16, past the 65,535 of a grid's second axis."""
    E = 1025
    counts = np.full(E, 1073)
    counts[::7] += 5
    counts[3] = 0
    run(E, 8, 32, 32, False, counts, seed=5, sample=[0, 1, 2, 3, 4, 500, 975, 976, 1000, E - 2, E - 1])
