"""Argument checks of the 4-bit weight products and of the token movement, on
the CPU: the binding refuses wrongly shaped, typed or placed tensors before
the C call (the library replaced by a recorder), and the C entry points refuse
bad arguments before any launch (made-up addresses that nothing reads)."""

import types

import pytest
import torch

from quantized_linear_gemm_b200 import lq

S = types.SimpleNamespace(cuda_stream=0)
BF, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
OK, INVALID, ALIGN, SHAPE = 0, 1, 2, 3


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(lq, "_DEVICE_TYPE", "cpu")
    monkeypatch.setattr(lq, "lib", lambda: r)
    return r


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def int4_args(M=3, N=16, K=256, G=64, zeros=False, lead=()):
    return (z(M, K), z(*lead, N, K // 2, dtype=U8), z(*lead, N, K // G), z(*lead, N, K // G, dtype=U8) if zeros else None)


def test_int4_mm_passes_shapes_on(rec):
    x, B, s, zp = int4_args(zeros=True)
    C = lq.int4_mm(x, B, s, b_zeros=zp, bias=z(16), stream=S)
    name, args = rec.calls[-1]
    assert name == "lq_int4_mm" and args[6:10] == (3, 16, 256, 64) and C.shape == (3, 16)
    x, B, s, _ = int4_args(lead=(5,), G=128)
    lq.grouped_int4_mm(x, B, s, z(6, dtype=I32), stream=S)
    name, args = rec.calls[-1]
    assert name == "lq_grouped_int4_mm" and args[6:11] == (5, 3, 16, 256, 128)


@pytest.mark.parametrize("bad", ["x_type", "x_strided", "B_rows", "B_type", "scales_type", "group", "no_groups", "zeros",
                                 "bias", "C", "not_a_tensor"])
def test_int4_mm_refuses(rec, bad):
    x, B, s, zp = int4_args(zeros=True)
    kw = dict(b_zeros=zp, bias=z(16), C=z(3, 16))
    if bad == "x_type":
        x = x.half()
    elif bad == "x_strided":
        x = z(3, 512)[:, ::2]
    elif bad == "B_rows":
        B = z(16, 120, dtype=U8)
    elif bad == "B_type":
        B = B.to(torch.int8)
    elif bad == "scales_type":
        s = s.float()
    elif bad == "group":
        s = z(16, 16)            # 16 weights per group
        kw["b_zeros"] = None
    elif bad == "no_groups":
        s = z(16, 0)
    elif bad == "zeros":
        kw["b_zeros"] = z(16, 3, dtype=U8)
    elif bad == "bias":
        kw["bias"] = z(15)
    elif bad == "C":
        kw["C"] = z(3, 17)
    elif bad == "not_a_tensor":
        x = [1.0]
    with pytest.raises((TypeError, ValueError)):
        lq.int4_mm(x, B, s, stream=S, **kw)
    assert not rec.calls


@pytest.mark.parametrize("bad", ["offsets_len", "offsets_type", "flat_B", "C", "scales"])
def test_grouped_int4_mm_refuses(rec, bad):
    x, B, s, _ = int4_args(lead=(4,))
    off, C = z(5, dtype=I32), None
    if bad == "offsets_len":
        off = z(4, dtype=I32)
    elif bad == "offsets_type":
        off = z(5, dtype=torch.int64)
    elif bad == "flat_B":
        B = B.view(64, 128)
    elif bad == "C":
        C = z(4, 16)
    elif bad == "scales":
        s = z(3, 16, 4)
    with pytest.raises((TypeError, ValueError)):
        lq.grouped_int4_mm(x, B, s, off, C=C, stream=S)
    assert not rec.calls


@pytest.mark.parametrize("bad", ["group", "divides", "type", "scales", "zeros"])
def test_quant_weight_int4_refuses(rec, bad):
    w, group, kw = z(4, 192), 64, {}
    if bad == "group":
        group = 48
    elif bad == "divides":
        group = 128
    elif bad == "type":
        w = w.float()
    elif bad == "scales":
        kw["scales"] = z(4, 3, dtype=F32)
    elif bad == "zeros":
        kw["zeros"] = z(4, 2, dtype=U8)
    with pytest.raises((TypeError, ValueError)):
        lq.quant_weight_int4(w, group, stream=S, **kw)
    assert not rec.calls


def test_token_calls_pass_shapes_on(rec):
    ids = z(5, 2, dtype=torch.int64)
    off, order, slots = lq.moe_sort(ids, 7, stream=S)
    assert rec.calls[-1][1][1:4] == (8, 10, 7) and off.shape == (8,) and order.shape == (10,) and slots.shape == (5, 2)
    xs = lq.moe_permute(z(5, 64), slots, stream=S)
    assert rec.calls[-1][1][3:7] == (5, 10, 2, 64) and xs.shape == (10, 64)
    lq.moe_permute(z(5, 64), slots, xs=z(6, 64), stream=S)
    assert rec.calls[-1][1][3:7] == (5, 6, 2, 64)
    q, s = lq.moe_permute_quant("w8a8_int8", z(5, 64), slots, stream=S)
    assert q.dtype == torch.int8 and q.shape == (10, 64) and s.shape == (10,)
    assert lq.moe_unpermute(xs, slots, z(5, 2, dtype=F32), stream=S).shape == (5, 64)
    assert lq.moe_permute_backward(xs, slots, stream=S).shape == (5, 64)
    dy, dw = lq.moe_unpermute_backward(z(5, 64), xs, slots, z(5, 2, dtype=F32), stream=S)
    assert dy.shape == (10, 64) and dw.shape == (5, 2) and dw.dtype == F32


CALLS = {
    "sort_type": lambda: lq.moe_sort(z(5, 2, dtype=torch.int16), 7, stream=S),
    "sort_1d": lambda: lq.moe_sort(z(5, dtype=I32), 7, stream=S),
    "sort_out": lambda: lq.moe_sort(z(5, 2, dtype=I32), 7, expert_offsets=z(7, dtype=I32), stream=S),
    "permute_tokens": lambda: lq.moe_permute(z(5, 64), z(4, 2, dtype=I32), stream=S),
    "permute_slots": lambda: lq.moe_permute(z(5, 64), z(5, 2, dtype=torch.int64), stream=S),
    "permute_width": lambda: lq.moe_permute(z(5, 64), z(5, 2, dtype=I32), xs=z(10, 32), stream=S),
    "permute_type": lambda: lq.moe_permute(z(5, 64, dtype=F32), z(5, 2, dtype=I32), stream=S),
    "quant_scales": lambda: lq.moe_permute_quant("fp8_dynamic", z(5, 64), z(5, 2, dtype=I32), scales=z(9, dtype=F32),
                                                 stream=S),
    "quant_q": lambda: lq.moe_permute_quant("fp8_dynamic", z(5, 64), z(5, 2, dtype=I32), q=z(10, 32, dtype=U8), stream=S),
    "unpermute_weights": lambda: lq.moe_unpermute(z(10, 64), z(5, 2, dtype=I32), z(5, 3, dtype=F32), stream=S),
    "unpermute_weights_type": lambda: lq.moe_unpermute(z(10, 64), z(5, 2, dtype=I32), z(5, 2), stream=S),
    "unpermute_out": lambda: lq.moe_unpermute(z(10, 64), z(5, 2, dtype=I32), out=z(4, 64), stream=S),
    "backward_dout": lambda: lq.moe_unpermute_backward(z(4, 64), z(10, 64), z(5, 2, dtype=I32), z(5, 2, dtype=F32),
                                                       stream=S),
    "backward_dy": lambda: lq.moe_unpermute_backward(z(5, 64), z(10, 64), z(5, 2, dtype=I32), z(5, 2, dtype=F32),
                                                     dy=z(9, 64), stream=S),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_token_calls_refuse(rec, name):
    with pytest.raises((TypeError, ValueError)):
        CALLS[name]()
    assert not rec.calls


A = 0x10000   # a made-up, aligned address


@pytest.mark.parametrize("args,want", [
    ((A, A, A, None, None, A, 4, 16, 128, 16, None), INVALID),        # group
    ((A, A, A, None, None, A, -1, 16, 128, 128, None), INVALID),
    ((None, A, A, None, None, A, 4, 16, 128, 128, None), INVALID),
    ((A, A, None, None, None, A, 4, 16, 128, 128, None), INVALID),
    ((A, A, A, None, None, None, 4, 16, 128, 128, None), INVALID),
    ((A + 2, A, A, None, None, A, 4, 16, 128, 128, None), ALIGN),
    ((A, A + 8, A, None, None, A, 4, 16, 128, 128, None), ALIGN),
    ((A, A, A + 1, None, None, A, 4, 16, 128, 128, None), ALIGN),
    ((A, A, A, None, A + 1, A, 4, 16, 128, 128, None), ALIGN),
    ((A, A, A, None, None, A, 4, 16, 192, 128, None), SHAPE),
    ((A, A, A, None, None, A, 4, 12, 128, 128, None), SHAPE),
    ((A, A, A, None, None, A, 4, 16, 0, 128, None), SHAPE),
    ((A, A, A, None, None, A, 1 << 31, 16, 128, 128, None), SHAPE),
    ((None, None, None, None, None, None, 0, 16, 128, 128, None), OK),
    ((None, None, None, None, None, None, 4, 0, 128, 128, None), OK),
])
def test_c_int4_mm(args, want):
    assert lq.call_raw("lq_int4_mm", *args) == want


@pytest.mark.parametrize("args,want", [
    ((A, A, A, None, A, None, 4, 8, 16, 128, 128, None), INVALID),    # no offsets
    ((A, A, A, None, A, A, 0, 8, 16, 128, 128, None), INVALID),       # no experts
    ((A, A, A, None, A, A + 2, 4, 8, 16, 128, 128, None), ALIGN),
    ((A, A, A, None, A, A, 1 << 28, 8, 16, 128, 128, None), SHAPE),   # E * N
    ((None, None, None, None, None, None, 4, 0, 16, 128, 128, None), OK),
])
def test_c_grouped_int4_mm(args, want):
    assert lq.call_raw("lq_grouped_int4_mm", *args) == want


@pytest.mark.parametrize("name,args,want", [
    ("lq_quant_weight_int4", (A, 48, A, A, None, 4, 96, None), INVALID),
    ("lq_quant_weight_int4", (A, 64, A, A, None, 4, 96, None), SHAPE),
    ("lq_quant_weight_int4", (A + 8, 32, A, A, None, 4, 96, None), ALIGN),
    ("lq_quant_weight_int4", (None, 32, A, A, None, 4, 96, None), INVALID),
    ("lq_quant_weight_int4", (None, 32, None, None, None, 0, 96, None), OK),
    ("lq_moe_sort", (A, 2, 8, 4, A, A, A, None), INVALID),
    ("lq_moe_sort", (A, 4, 8, 4, None, A, A, None), INVALID),
    ("lq_moe_sort", (A, 4, 8, 4, A, None, A, None), INVALID),
    ("lq_moe_sort", (A + 4, 8, 8, 4, A, A, A, None), ALIGN),
    ("lq_moe_sort", (A, 4, 8, 1025, A, A, A, None), SHAPE),
    ("lq_moe_sort", (A, 4, 8, 0, A, A, A, None), SHAPE),
    ("lq_moe_sort", (A, 4, 1 << 31, 4, A, A, A, None), SHAPE),
    ("lq_moe_permute", (A, A, A, 4, 8, 2, 12, None), SHAPE),
    ("lq_moe_permute", (A, A, A, 4, 8, 2, 1 << 26, None), SHAPE),
    ("lq_moe_permute", (A + 8, A, A, 4, 8, 2, 16, None), ALIGN),
    ("lq_moe_permute", (A, None, A, 4, 8, 2, 16, None), INVALID),
    ("lq_moe_permute", (A, A, A, -4, 8, 2, 16, None), INVALID),
    ("lq_moe_permute", (None, None, None, 0, 8, 2, 16, None), OK),
    ("lq_moe_permute_quant", (2, A, A, A, A, 4, 8, 2, 16, None), INVALID),
    ("lq_moe_permute_quant", (0, A, A, A, A, 4, 8, 2, 24, None), SHAPE),
    ("lq_moe_permute_quant", (0, A, A, A + 4, A, 4, 8, 2, 16, None), ALIGN),
    ("lq_moe_permute_quant", (0, A, A, A, None, 4, 8, 2, 16, None), INVALID),
    ("lq_moe_unpermute", (A, A, None, None, 4, 8, 2, 16, None), INVALID),
    ("lq_moe_unpermute", (A, None, None, A, 4, 8, 2, 16, None), INVALID),
    ("lq_moe_unpermute", (A, A, A + 2, A, 4, 8, 2, 16, None), ALIGN),
    ("lq_moe_unpermute", (A, A, None, A, 4, 8, 2, 4, None), SHAPE),
    ("lq_moe_unpermute", (None, None, None, None, 0, 8, 2, 16, None), OK),
    ("lq_moe_unpermute_backward", (A, A, A, None, A, A, 4, 8, 2, 16, None), INVALID),
    ("lq_moe_unpermute_backward", (A, A, A, A, A, None, 4, 8, 2, 16, None), INVALID),
    ("lq_moe_unpermute_backward", (A, A, A, A, A + 8, A, 4, 8, 2, 16, None), ALIGN),
    ("lq_moe_unpermute_backward", (None, None, None, None, None, None, 0, 8, 2, 16, None), OK),
])
def test_c_refusals(name, args, want):
    assert lq.call_raw(name, *args) == want


@pytest.mark.parametrize("name,args", [
    ("lq_int4_mm", (A, A, A, None, None, A, (1 << 31) - 255, 8, 32, 32, None)),       # rounded up to a tile: 2^31
    ("lq_int4_mm", (A, A, A, None, None, A, 4, 8, (1 << 24) + 32, 32, None)),
    ("lq_grouped_int4_mm", (A, A, A, None, A, A, 2, (1 << 31) - 255, 8, 32, 32, None)),
    ("lq_moe_permute", (A, A, A, 1, 8, (1 << 31) - 1, 16, None)),                     # slots counted in steps of 8
    ("lq_moe_permute_quant", (0, A, A, A, A, 1, 8, (1 << 31) - 1, 16, None)),
    ("lq_moe_unpermute", (A, A, None, A, 1, 8, (1 << 24) + 1, 16, None)),
    ("lq_moe_unpermute_backward", (A, A, A, A, A, A, 1, 8, (1 << 24) + 1, 16, None)),
])
def test_c_counts_past_32_bits(name, args):
    assert lq.call_raw(name, *args) == SHAPE
