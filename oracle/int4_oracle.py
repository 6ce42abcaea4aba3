"""Plain CPU oracle for 4-bit weights with group scales.

TEST INFRASTRUCTURE ONLY.  Only the test suite and
``__graft_entry__.smoke()`` may import or run this module.  The library under
``quantized_linear_gemm_b200/`` never calls it, links it or shares code with it.

The format (a weight-only one beside the 8-bit formats of ``lq_oracle``; no
page defines it):

* weight[n, k] = (q[n, k] - z[n, g]) * s[n, g], g = k // G, G in {32, 64, 128};
* q in 0..15, packed two per byte, the even k in the low half;
* s bf16; z in 0..15, or 8 everywhere without zero points.

Quantization of a bf16 weight, per group: symmetric
s = max(bf16(amax / 7), 2^-126), q = clamp(rint(w / s), -8, 7) + 8; with zero
points lo = min(0, min w), hi = max(0, max w),
s = max(bf16((hi - lo) / 15), 2^-126), z = clamp(rint(-lo / s), 0, 15),
q = clamp(rint(w / s) + z, 0, 15).  Differences and quotients are rounded to
fp32, rint rounds half to even.
"""

from __future__ import annotations

import numpy as np


def bf16_round(v) -> np.ndarray:
    """fp32 values rounded to bf16 (half to even), as float32."""
    b = np.asarray(v, dtype=np.float32).view(np.uint32).astype(np.uint64)
    b = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16
    return b.astype(np.uint32).view(np.float32)


def pack(q) -> np.ndarray:
    """Codes [..., K] -> bytes [..., K / 2]."""
    q = np.asarray(q, dtype=np.uint8)
    return (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)


def unpack(b) -> np.ndarray:
    """Bytes [..., K / 2] -> codes [..., K]."""
    b = np.asarray(b, dtype=np.uint8)
    out = np.empty((*b.shape[:-1], b.shape[-1] * 2), dtype=np.uint8)
    out[..., 0::2] = b & 15
    out[..., 1::2] = b >> 4
    return out


def quant_weight_int4(w, group: int, zero_points: bool):
    """(packed codes [N, K / 2], scales float32 holding bf16 values
    [N, K / group], zero points uint8 [N, K / group] or None)."""
    w = np.asarray(w, dtype=np.float32)
    N, K = w.shape
    g = w.reshape(N, K // group, group)
    tiny = np.float32(2.0 ** -126)
    if zero_points:
        lo = np.minimum(g.min(-1), np.float32(0))
        hi = np.maximum(g.max(-1), np.float32(0))
        s = np.maximum(bf16_round((hi - lo) / np.float32(15)), tiny)
        z = np.clip(np.rint(-lo / s), 0, 15).astype(np.int64)
    else:
        s = np.maximum(bf16_round(np.abs(g).max(-1) / np.float32(7)), tiny)
        z = np.full(s.shape, 8, dtype=np.int64)
    q = np.rint(g / s[..., None]).astype(np.int64) + z[..., None]
    q = np.clip(q, 0, 15).astype(np.uint8).reshape(N, K)
    return pack(q), s, (z.astype(np.uint8) if zero_points else None)


def dequant(B, scales, zeros) -> np.ndarray:
    """Weights [..., N, K] in fp64."""
    q = unpack(B).astype(np.float64)
    s = np.asarray(scales, dtype=np.float64)
    G = q.shape[-1] // s.shape[-1]
    q = q.reshape(*q.shape[:-1], s.shape[-1], G)
    z = 8.0 if zeros is None else (np.asarray(zeros) & 15).astype(np.float64)[..., None]
    out = (q - z) * s[..., None]
    return out.reshape(*out.shape[:-2], out.shape[-2] * G)


def int4_mm_ref(x, B, scales, zeros, bias=None):
    """(C in fp64 before rounding, sum of |x| |weight|) of one product."""
    x = np.asarray(x, dtype=np.float64)
    w = dequant(B, scales, zeros)
    c = x @ w.T
    mag = np.abs(x) @ np.abs(w).T
    if bias is not None:
        c = c + np.asarray(bias, dtype=np.float64)
        mag = mag + np.abs(np.asarray(bias, dtype=np.float64))
    return c, mag
