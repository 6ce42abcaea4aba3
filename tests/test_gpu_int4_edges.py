"""Edges of the 4-bit products on the GPU: waits that run out, arrays past 32
bits of offset, scale arrays at odd addresses, zero points with stray high
bits, scales far from one, padded batches, and calls that overlap.  Tolerances
as in test_gpu_int4.py."""

import numpy as np
import pytest
import torch

from oracle import int4_oracle as I
from quantized_linear_gemm_b200 import inputs, lq

from test_gpu_int4 import check, dev, weight

pytestmark = pytest.mark.gpu

TIMEOUT = 6


# tokens: one tile of 16, 32, 64, 128 and 256 tokens; K long enough for Split-K in the last two
@pytest.mark.parametrize("M,N,K", [(12, 256, 512), (24, 256, 512), (50, 256, 512), (100, 256, 512), (300, 256, 512),
                                   (24, 128, 8192), (200, 128, 8192)])
def test_bounded_wait_runs_out_and_is_reported(cuda_device, M, N, K):
    x = inputs.activations(M, K, seed=1)
    B, s, _ = weight(N, K, 128, False, 2, pow2=True)
    Bd, sd, xd = dev(B), dev(s, torch.bfloat16), x.cuda()
    lq.init_device(0)
    assert lq.device_status(0) == 0
    lq.test_inject_stall(1, 100_000_000)             # K block 1 never arrives; waits give up after 0.1 s
    try:
        lq.int4_mm(xd, Bd, sd)
        torch.cuda.synchronize()                     # the kernel returned: nothing hung
        assert lq.device_status(0) == TIMEOUT
    finally:
        lq.test_inject_stall(-1, 0)
    C = lq.int4_mm(xd, Bd, sd)                       # the context is intact
    torch.cuda.synchronize()
    assert lq.device_status(0) == 0
    r, mag = I.int4_mm_ref(x.float().numpy(), B, s, None)
    check(C, r, mag, K, False)


@pytest.mark.parametrize("M", [3, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_scales_at_odd_addresses(cuda_device, M, group):
    """Views that start one element into their storage: the aligned-word loads do not apply."""
    N, K = 136, 384
    x = inputs.activations(M, K, seed=1)
    B, s, z = weight(N, K, group, True, 3, pow2=True)
    sbuf = torch.empty(s.size + 1, dtype=torch.bfloat16, device="cuda")
    zbuf = torch.empty(z.size + 1, dtype=torch.uint8, device="cuda")
    sv, zv = sbuf[1:].view(s.shape), zbuf[1:].view(z.shape)
    sv.copy_(dev(s, torch.bfloat16))
    zv.copy_(dev(z))
    C = lq.int4_mm(x.cuda(), dev(B), sv, b_zeros=zv)
    torch.cuda.synchronize()
    r, mag = I.int4_mm_ref(x.float().numpy(), B, s, z)
    check(C, r, mag, K, False)


@pytest.mark.parametrize("M", [2, 70])
def test_zero_points_use_their_low_four_bits(cuda_device, M):
    x = inputs.activations(M, 256, seed=1)
    B, s, z = weight(64, 256, 64, True, 5, pow2=True)
    stray = (z | (np.random.default_rng(1).integers(0, 16, z.shape, dtype=np.uint8) << 4)).astype(np.uint8)
    a = lq.int4_mm(x.cuda(), dev(B), dev(s, torch.bfloat16), b_zeros=dev(stray))
    b = lq.int4_mm(x.cuda(), dev(B), dev(s, torch.bfloat16), b_zeros=dev(z))
    assert torch.equal(a, b)


@pytest.mark.parametrize("M", [2, 70])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("e", [-40, -20, 20, 33])
def test_scales_far_from_one(cuda_device, M, zeros, e):
    """Scales of 2^e times 1 or 1.5: C is that much larger or smaller, with the same relative error."""
    N, K = 64, 512
    x = inputs.activations(M, K, seed=1)
    B, _, z = weight(N, K, 128, zeros, 6)
    s = (np.float32(2.0 ** e) * np.random.default_rng(2).choice([1.0, 1.5], (N, K // 128))).astype(np.float32)
    C = lq.int4_mm(x.cuda(), dev(B), dev(s, torch.bfloat16), b_zeros=dev(z))
    torch.cuda.synchronize()
    r, mag = I.int4_mm_ref(x.float().numpy(), B, s, z)
    check(C, r, mag, K, True)


def test_more_than_2_31_outputs(cuda_device):
    """C past 2^31 elements (tensor-core kernel), checked on sampled rows."""
    M, N, K = 90112, 24576, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    B, s, _ = weight(N, K, 128, False, 2, pow2=True)
    C = lq.int4_mm(x, dev(B), dev(s, torch.bfloat16))
    torch.cuda.synchronize()
    assert C.numel() > 2 ** 31
    rows = [0, 1, 87381, 87382, M - 257, M - 1]
    r, mag = I.int4_mm_ref(x[rows].float().cpu().numpy(), B, s, None)
    check(C[rows], r, mag, K, False)


@pytest.mark.parametrize("rows", [4, 40])
def test_weights_past_2_31_bytes(cuda_device, rows):
    """The last of many experts: its codes lie past 2^31 bytes (streaming and tensor-core kernels)."""
    E, N, K = 530, 2048, 4096
    B = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.ones((E, N, K // 128), dtype=torch.bfloat16, device="cuda") * 2.0 ** -6
    assert B.numel() > 2 ** 31
    x = inputs.activations(rows, K, seed=3)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = rows
    C = lq.grouped_int4_mm(x.cuda(), B, s, off)
    torch.cuda.synchronize()
    cols = slice(N - 64, N)
    r, mag = I.int4_mm_ref(x.float().numpy(), B[E - 1, cols].cpu().numpy(), s[E - 1, cols].float().cpu().numpy(), None)
    check(C[:, cols], r, mag, K, False)


@pytest.mark.parametrize("counts", [[3, 2, 0, 4], [30, 0, 70, 5]])
def test_rows_behind_the_last_expert_do_not_matter(cuda_device, counts):
    """A padded batch: rows past the last offset hold NaN; the experts' rows are exact and the rest of C untouched."""
    N, K, E = 136, 256, len(counts)
    used = sum(counts)
    T = used + 37
    x = inputs.activations(T, K, seed=1).cuda()
    x[used:] = float("nan")
    B, s, _ = weight(E * N, K, 64, False, 2, pow2=True)
    B, s = B.reshape(E, N, -1), s.reshape(E, N, -1)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    C = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    lq.grouped_int4_mm(x, dev(B), dev(s, torch.bfloat16), off, C=C)
    torch.cuda.synchronize()
    assert torch.all(C[used:] == 7.0)
    lo = 0
    for e, c in enumerate(counts):
        if c:
            r, mag = I.int4_mm_ref(x[lo:lo + c].float().cpu().numpy(), B[e], s[e], None)
            check(C[lo:lo + c], r, mag, K, False, what=e)
        lo += c


@pytest.mark.parametrize("many", [True, False])
def test_more_experts_than_the_tensor_core_kernel_keeps(cuda_device, many):
    """1025 experts take the streaming kernel, 1024 the tensor-core one; most are empty."""
    E, N, K = (1025 if many else 1024), 16, 64
    counts = np.zeros(E, dtype=np.int64)
    counts[[0, 7, 500, E - 1]] = [5, 20, 1, 19]
    x = inputs.activations(45, K, seed=1)
    B, s, z = weight(E * N, K, 32, True, 2, pow2=True)
    B, s, z = B.reshape(E, N, -1), s.reshape(E, N, -1), z.reshape(E, N, -1)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    C = lq.grouped_int4_mm(x.cuda(), dev(B), dev(s, torch.bfloat16), dev(off), b_zeros=dev(z))
    torch.cuda.synchronize()
    for e in np.nonzero(counts)[0]:
        lo, hi = off[e], off[e + 1]
        r, mag = I.int4_mm_ref(x[lo:hi].float().numpy(), B[e], s[e], z[e])
        check(C[lo:hi], r, mag, K, False, what=e)


def test_two_graphs_at_once(cuda_device):
    """Two captured products (Split-K clusters, and many tiles) replayed side by side on two streams, again and again."""
    xa, xb = inputs.activations(40, 8192, seed=1).cuda(), inputs.activations(300, 1024, seed=2).cuda()
    Ba, sa, _ = weight(512, 8192, 128, False, 3)
    Bb, sb, _ = weight(2048, 1024, 64, False, 4)
    Ba, sa, Bb, sb = dev(Ba), dev(sa, torch.bfloat16), dev(Bb), dev(sb, torch.bfloat16)
    ra, rb = lq.int4_mm(xa, Ba, sa), lq.int4_mm(xb, Bb, sb)
    Ca, Cb = torch.zeros_like(ra), torch.zeros_like(rb)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=s1):
        for _ in range(5):
            lq.int4_mm(xa, Ba, sa, C=Ca)
    with torch.cuda.graph(g2, stream=s2):
        for _ in range(5):
            lq.int4_mm(xb, Bb, sb, C=Cb)
    for _ in range(10):
        Ca.zero_()
        Cb.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(Ca, ra) and torch.equal(Cb, rb)
    assert lq.device_status(0) == 0


@pytest.mark.parametrize("fmt", ["fp8_dynamic", "block_fp8"])
def test_beside_an_8_bit_product(cuda_device, fmt):
    """Split-K clusters of both kinds of product on two streams: neither waits for tensor memory of the other's
    cluster peers for good, and no result changes."""
    x = inputs.activations(64, 8192, seed=1).cuda()
    B, s, _ = weight(512, 8192, 128, False, 3)
    B, s = dev(B), dev(s, torch.bfloat16)
    w = inputs.weights(1024, 8192, seed=4).cuda()
    if fmt == "block_fp8":
        a, sa = lq.quant_per_token_group128(x)
        b, sb = lq.quant_weight_block128(w)
    else:
        a, sa = lq.quant_per_token(fmt, x)
        b, sb = lq.quant_per_token(fmt, w)
    r4, r8 = lq.int4_mm(x, B, s), lq.scaled_mm(fmt, a, sa, b, sb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(s1):
            c4 = [lq.int4_mm(x, B, s) for _ in range(5)]
        with torch.cuda.stream(s2):
            c8 = [lq.scaled_mm(fmt, a, sa, b, sb) for _ in range(5)]
        torch.cuda.synchronize()
        assert all(torch.equal(c, r4) for c in c4) and all(torch.equal(c, r8) for c in c8)
    assert lq.device_status(0) == 0


@pytest.mark.parametrize("M", [4, 40, 300])
def test_weight_written_just_before(cuda_device, M):
    """A weight quantized on the same stream right before the product is the one used, whatever was there."""
    N, K = 512, 2048
    w = [inputs.weights(N, K, seed=i).cuda() for i in range(2)]
    x = inputs.activations(M, K, seed=5).cuda()
    want = []
    for v in w:
        q, s, _ = lq.quant_weight_int4(v, 128)
        torch.cuda.synchronize()
        want.append(lq.int4_mm(x, q, s).clone())
    q, s, _ = lq.quant_weight_int4(w[0], 128)
    C = torch.empty_like(want[0])
    for i in range(20):
        lq.quant_weight_int4(w[i & 1], 128, q=q, scales=s)
        lq.int4_mm(x, q, s, C=C)
        torch.cuda.synchronize()
        assert torch.equal(C, want[i & 1])


def test_static_weights_give_the_same(cuda_device):
    """The weight stream that starts before the previous launch has finished changes no result."""
    N, K = 1024, 4096
    B, s, _ = weight(N, K, 128, False, 2)
    B, s = dev(B), dev(s, torch.bfloat16)
    for M in (4, 40, 300):
        x = inputs.activations(M, K, seed=M).cuda()
        ref = lq.int4_mm(x, B, s)
        prev = lq.declare_static_weights(True)
        try:
            outs = [lq.int4_mm(x, B, s) for _ in range(4)]
        finally:
            lq.declare_static_weights(prev)
        assert all(torch.equal(o, ref) for o in outs)
