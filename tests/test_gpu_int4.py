"""GPU parity of the 4-bit weight quantizer and products against the CPU
oracle (fp64): every group size, with and without zero points and bias, token
counts from one to several tiles, ragged N and K, grouped products with empty
and crowded experts, graph replay and other streams.

Tolerances, derived: the reference r is exact in fp64 and S = sum |x| |w|.
C is one rounding to bf16 of an fp32 sum, half a step 2^-8 |r| (plus the same
share of the sum's error), and a sum of K terms in fp32, truncation allowed,
is off by at most K 2^-23 S.  Where the weights are rounded to bf16 before the
product (many tokens), each term is off by at most 2^-8 of itself: 2^-8 S more
in the worst case, nothing for scales that are powers of two (then
(q - z) s has at most 5 significant bits)."""

import numpy as np
import pytest
import torch

from oracle import int4_oracle as I
from quantized_linear_gemm_b200 import inputs, lq

from _lqtest import bf16_to_f64

pytestmark = pytest.mark.gpu


def weight(N, K, group, zeros, seed, pow2=False):
    """(codes, bf16-valued float32 scales, zero points or None): every code value occurs."""
    g = np.random.default_rng(seed)
    q = g.integers(0, 16, (N, K), dtype=np.uint8)
    s = np.exp2(g.integers(-8, -3, (N, K // group))) if pow2 else g.uniform(0.001, 0.03, (N, K // group))
    s = I.bf16_round(s.astype(np.float32))
    z = g.integers(0, 16, (N, K // group), dtype=np.uint8) if zeros else None
    return I.pack(q), s, z


def dev(a, dtype=None):
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def limit(r, mag, K, rounded_weights):
    e = K * 2.0 ** -23 * mag + (2.0 ** -8 * mag if rounded_weights else 0.0)
    return e + 2.0 ** -8 * (np.abs(r) + e) + 2.0 ** -126


def check(C, r, mag, K, rounded_weights, what=""):
    c = bf16_to_f64(C)
    over = np.abs(c - r) / limit(r, mag, K, rounded_weights)
    assert np.all(np.isfinite(c)), what
    assert over.max(initial=0.0) <= 1.0, (what, over.max(), np.unravel_index(over.argmax(), over.shape))


def run_dense(M, N, K, group, zeros, bias, seed=0, pow2=False):
    x = inputs.activations(M, K, seed=seed + 1)
    B, s, z = weight(N, K, group, zeros, seed + 2, pow2)
    b = torch.randn(N, generator=torch.Generator().manual_seed(seed)).bfloat16() if bias else None
    C = lq.int4_mm(x.cuda(), dev(B), dev(s, torch.bfloat16), b_zeros=dev(z), bias=b.cuda() if bias else None)
    torch.cuda.synchronize()
    assert lq.device_status(0) == 0
    r, mag = I.int4_mm_ref(x.float().numpy(), B, s, z, b.float().numpy() if bias else None)
    check(C, r, mag, K, rounded_weights=not pow2, what=(M, N, K, group, zeros, bias))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("shape", [(2, 128), (5, 384), (300, 1024)])
def test_quantizer_bit_exact(cuda_device, group, zeros, shape):
    N, K = shape
    w = inputs.weights(N, K, seed=N + group)
    w[0, :group] = 0                                             # an all-zero group
    w[1, :group] = torch.linspace(-1, 2, group).bfloat16()       # ties and one-sided groups
    w[1, group:2 * group if K >= 2 * group else group] = 0.25
    q, s, z = lq.quant_weight_int4(w.cuda(), group, zeros)
    torch.cuda.synchronize()
    rq, rs, rz = I.quant_weight_int4(w.float().numpy(), group, zeros)
    assert np.array_equal(s.float().cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert (z is None) == (rz is None) and (z is None or np.array_equal(z.cpu().numpy(), rz))


@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("group,zeros,bias", [(128, False, False), (128, True, True), (64, True, False),
                                              (64, False, True), (32, False, False), (32, True, True)])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 130, 257])
def test_dense(cuda_device, M, group, zeros, bias, pow2):
    run_dense(M, 264, 1152, group, zeros, bias, seed=M, pow2=pow2)


@pytest.mark.parametrize("M", [1, 8, 12, 40, 200])
@pytest.mark.parametrize("N", [8, 16, 120, 136])
@pytest.mark.parametrize("K,group", [(32, 32), (96, 32), (64, 64), (128, 128), (192, 64), (160, 32), (4096, 128)])
def test_ragged(cuda_device, M, N, K, group):
    run_dense(M, N, K, group, True, False, seed=N + K, pow2=True)


@pytest.mark.parametrize("layer", ["qkv", "down"])
@pytest.mark.parametrize("M", [1, 24])
def test_qwen3_8b(cuda_device, layer, M):
    K, N = inputs.QWEN3_8B[layer]
    run_dense(M, N, K, 128, False, False, seed=5)


def test_quantized_weight_through_the_product(cuda_device):
    """The path as used: quantize a bf16 weight, multiply; against fp64 over
    the dequantized weight, and near the unquantized product."""
    N, K, M = 512, 2048, 5
    w, x = inputs.weights(N, K, seed=3), inputs.activations(M, K, seed=4)
    for zp in (False, True):
        q, s, z = lq.quant_weight_int4(w.cuda(), 64, zp)
        C = lq.int4_mm(x.cuda(), q, s, b_zeros=z)
        torch.cuda.synchronize()
        r, mag = I.int4_mm_ref(x.float().numpy(), q.cpu().numpy(), s.float().cpu().numpy(),
                               None if z is None else z.cpu().numpy())
        check(C, r, mag, K, False)


def test_masked_tokens_do_not_mix(cuda_device):
    """NaN or infinity in one token's activations stays in its row."""
    for M in (3, 20, 150):
        x = inputs.activations(M, 256, seed=1)
        x[1, 7], x[2, 9] = float("nan"), float("inf")
        B, s, z = weight(128, 256, 128, False, 2, pow2=True)
        C = lq.int4_mm(x.cuda(), dev(B), dev(s, torch.bfloat16))
        torch.cuda.synchronize()
        c = bf16_to_f64(C)
        assert np.all(np.isnan(c[1])) and not np.any(np.isfinite(c[2]))
        keep = [m for m in range(M) if m not in (1, 2)]
        r, mag = I.int4_mm_ref(x[keep].float().numpy(), B, s, z)
        check(C[keep], r, mag, 256, False)


def run_grouped(counts, N, K, group, zeros, seed, pow2=True, offsets=None, T=None):
    E = len(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) if offsets is None else np.asarray(offsets, np.int32)
    T = int(off[-1]) if T is None else T
    x = inputs.activations(max(T, 1), K, seed=seed)[:T]
    B, s, z = weight(E * N, K, group, zeros, seed + 1, pow2)
    B, s = B.reshape(E, N, -1), s.reshape(E, N, -1)
    z = None if z is None else z.reshape(E, N, -1)
    C = torch.full((T + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
    lq.grouped_int4_mm(x.cuda(), dev(B), dev(s, torch.bfloat16), dev(off), b_zeros=dev(z), C=C[:T])
    torch.cuda.synchronize()
    assert lq.device_status(0) == 0
    H = np.maximum.accumulate(np.clip(off, 0, T))
    done = np.zeros(T + 3, dtype=bool)
    for e in range(E):
        lo, hi = int(H[e]), int(H[e + 1])
        if hi > lo:
            r, mag = I.int4_mm_ref(x[lo:hi].float().numpy(), B[e], s[e], None if z is None else z[e])
            check(C[lo:hi], r, mag, K, not pow2, what=(e, lo, hi))
            done[lo:hi] = True
    assert torch.all(C[torch.from_numpy(~done).cuda()] == 7.0)   # rows outside every expert, and past the last


@pytest.mark.parametrize("group,zeros", [(128, False), (64, True), (32, False)])
@pytest.mark.parametrize("counts", [[1], [0, 0, 1], [3, 0, 1, 17, 0, 0, 5, 40, 2, 1], [0, 150, 0], [129, 0, 64, 300],
                                    [1] * 70])
def test_grouped(cuda_device, counts, group, zeros):
    run_grouped(counts, 264, 384, group, zeros, seed=len(counts))


@pytest.mark.parametrize("offsets,T", [([0, 10, 5, 200], 20), ([0, 4, 4, 9], 20), ([3, 6, 9, 12], 12), ([-5, 2, 2, 8], 8)])
def test_grouped_offset_tables(cuda_device, offsets, T):
    """Offsets past T, decreasing, ending early or starting late: clamped; other rows untouched."""
    run_grouped([0] * 3, 136, 256, 64, True, seed=9, offsets=offsets, T=T)


@pytest.mark.parametrize("tokens", [1, 8, 64])
@pytest.mark.parametrize("layer", ["gate_up", "down"])
def test_grouped_qwen3_moe(cuda_device, layer, tokens):
    K, N = inputs.QWEN3_30B_A3B_EXPERTS[layer]
    counts = inputs.expert_counts(tokens, 16, 2, seed=tokens)
    run_grouped(list(counts), N, K, 128, False, seed=tokens, pow2=False)


def test_one_expert_is_the_dense_product(cuda_device):
    x = inputs.activations(13, 512, seed=1).cuda()
    B, s, z = weight(256, 512, 64, True, 2)
    B, s, z = dev(B), dev(s, torch.bfloat16), dev(z)
    off = torch.tensor([0, 13], dtype=torch.int32, device="cuda")
    C = lq.grouped_int4_mm(x, B[None], s[None], off, b_zeros=z[None])
    assert torch.equal(C, lq.int4_mm(x, B, s, b_zeros=z))


@pytest.mark.parametrize("M", [1, 20, 300])
def test_graph_replay_and_other_stream(cuda_device, M):
    K, N = 1024, 1536
    x = inputs.activations(M, K, seed=1).cuda()
    B, s, _ = weight(N, K, 128, False, 2)
    B, s = dev(B), dev(s, torch.bfloat16)
    ref = lq.int4_mm(x, B, s)
    st = torch.cuda.Stream()
    C = torch.empty_like(ref)
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        lq.int4_mm(x, B, s, C=C)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            lq.int4_mm(x, B, s, C=C)
    C.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(C, ref)
    side = lq.int4_mm(x, B, s, stream=st)
    st.synchronize()
    assert torch.equal(side, ref)


def test_no_tokens_no_columns(cuda_device):
    B, s, _ = weight(16, 128, 128, False, 2)
    assert lq.int4_mm(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"), dev(B),
                      dev(s, torch.bfloat16)).shape == (0, 16)
    assert lq.int4_mm(torch.zeros((3, 128), dtype=torch.bfloat16, device="cuda"), dev(B[:0]),
                      dev(s[:0], torch.bfloat16)).shape == (3, 0)
