"""GPU parity of the 128-token form of the 4-bit tensor-core kernel (dense
products of 65 to 128 tokens, grouped products of prompts), with K long enough
for its ring to wrap many times and beside a stream that keeps HBM busy, so
that copies arrive late and unevenly.  Tolerances as in test_gpu_int4.py;
repeats are compared bit for bit."""

import numpy as np
import pytest
import torch

from oracle import int4_oracle as I
from quantized_linear_gemm_b200 import inputs, lq

from test_gpu_int4 import check, dev, weight

pytestmark = pytest.mark.gpu


def repeats(call, first, n=12):
    """n more calls while another stream copies 512 MB buffers: the bits of the first."""
    src = torch.empty(1 << 28, dtype=torch.bfloat16, device="cuda").normal_()
    dst = torch.empty_like(src)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(2 * n):
            dst.copy_(src)
    outs = [call() for _ in range(n)]
    torch.cuda.synchronize()
    assert lq.device_status(0) == 0
    assert all(torch.equal(o, first) for o in outs)


@pytest.mark.parametrize("M,N,K,group,zeros", [
    (65, 264, 4096, 128, False), (100, 264, 4096, 64, True), (128, 264, 4096, 32, False),
    (65, 264, 25600, 64, True), (100, 264, 25600, 128, False), (128, 264, 25600, 32, True),
    (100, 19200, 4096, 128, False),                       # a tile and more for every SM: no Split-K
    (128, 19336, 2048, 64, True)])                        # two tiles for some, the last one ragged
def test_dense(cuda_device, M, N, K, group, zeros):
    x = inputs.activations(M, K, seed=M + K)
    B, s, z = weight(N, K, group, zeros, 3, pow2=True)
    xd, Bd, sd, zd = x.cuda(), dev(B), dev(s, torch.bfloat16), dev(z)
    C = lq.int4_mm(xd, Bd, sd, b_zeros=zd)
    torch.cuda.synchronize()
    assert lq.device_status(0) == 0
    cols = np.unique(np.r_[np.arange(min(N, 264)), np.arange(N - 40, N)])
    r, mag = I.int4_mm_ref(x.float().numpy(), B[cols], s[cols], None if z is None else z[cols])
    check(C[:, torch.from_numpy(cols).cuda()], r, mag, K, False)
    repeats(lambda: lq.int4_mm(xd, Bd, sd, b_zeros=zd), C)


@pytest.mark.parametrize("K,group,zeros", [(768, 32, True), (2048, 128, False)])
def test_grouped_prompt(cuda_device, K, group, zeros):
    """1001 tokens of 8 choices over 128 experts, unevenly: none to several tiles per expert."""
    E, N, T = 128, 136, 8008
    g = np.random.default_rng(K)
    share = g.gamma(1.0, 1.0, E)
    share[g.integers(0, E, 5)] = 0
    counts = g.multinomial(T, share / share.sum())
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x = inputs.activations(T, K, seed=K)
    B, s, z = weight(E * N, K, group, zeros, 4, pow2=True)
    B, s = B.reshape(E, N, -1), s.reshape(E, N, -1)
    z = None if z is None else z.reshape(E, N, -1)
    xd, Bd, sd, zd, od = x.cuda(), dev(B), dev(s, torch.bfloat16), dev(z), dev(off)
    C = lq.grouped_int4_mm(xd, Bd, sd, od, b_zeros=zd)
    torch.cuda.synchronize()
    assert lq.device_status(0) == 0
    xf = x.float().numpy()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            r, mag = I.int4_mm_ref(xf[lo:hi], B[e], s[e], None if z is None else z[e])
            check(C[lo:hi], r, mag, K, False, what=e)
    repeats(lambda: lq.grouped_int4_mm(xd, Bd, sd, od, b_zeros=zd), C)
