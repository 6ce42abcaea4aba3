"""Python binding of liblq (ctypes).  Argument marshalling only.

Every function here checks its tensors (dtype, rank, contiguity, the exact
shape the C function reads or writes, and one device: the current CUDA
device), then calls the C function of the same name in ``liblq.so`` on
torch's current CUDA stream, or on `stream`, whose memory the outputs then come
from.  All arithmetic runs in the library's CUDA kernels; there is no
fallback.  If ``liblq.so`` is missing the first call raises.

No function takes part in autograd: an output carries no graph even when an
input requires a gradient.  The gradients that the library has are functions of
their own (moe_permute_backward, moe_unpermute_backward).
"""

from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblq.so")

FP8_DYNAMIC = 0
W8A8_INT8 = 1
BLOCK_FP8 = 2
BLOCK_FP8_UE8M0 = 3
FORMATS = {"fp8_dynamic": FP8_DYNAMIC, "w8a8_int8": W8A8_INT8, "block_fp8": BLOCK_FP8,
           "block_fp8_ue8m0": BLOCK_FP8_UE8M0}

STATUS = {
    0: "LQ_OK", 1: "LQ_ERR_INVALID_ARG", 2: "LQ_ERR_ALIGNMENT", 3: "LQ_ERR_UNSUPPORTED_SHAPE",
    4: "LQ_ERR_WORKSPACE", 5: "LQ_ERR_CUDA", 6: "LQ_ERR_DEVICE_TIMEOUT", 7: "LQ_ERR_TABLE",
}

# every symbol that include/lq.h declares
EXPORTED = (
    "lq_scaled_mm", "lq_scaled_mm_i32acc", "lq_quant_per_token", "lq_quant_per_token_group128",
    "lq_quant_weight_block128", "lq_select_variant", "lq_load_dispatch_table", "lq_dispatch_table_size",
    "lq_init_device", "lq_reserve_workspace", "lq_workspace_bytes", "lq_device_status",
    "lq_status_string", "lq_version", "lq_set_trace", "lq_scaled_mm_noalloc", "lq_test_inject_stall",
    "lq_test_silu_bf16",
    "lq_quant_scaled_mm", "lq_set_fuse_limit", "lq_rms_norm_dynamic_per_token_quant",
    "lq_rms_norm_per_block_quant", "lq_silu_and_mul_dynamic_per_token_quant", "lq_silu_and_mul_per_block_quant",
    "lq_grouped_scaled_mm", "lq_quant_per_token_group128_ue8m0", "lq_quant_weight_block128_ue8m0",
    "lq_scaled_mm_bias", "lq_declare_static_weights", "lq_quant_weight_int4", "lq_int4_mm", "lq_grouped_int4_mm",
    "lq_moe_sort", "lq_moe_permute", "lq_moe_permute_quant", "lq_moe_unpermute", "lq_moe_unpermute_backward",
)


class LQError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)}")
        self.code = code


class Variant(ctypes.Structure):
    _fields_ = [("swap_ab", ctypes.c_int32), ("split_k", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("reduce", ctypes.c_int32), ("pdl", ctypes.c_int32),
                ("persistent", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {f: int(getattr(self, f)) for f, _ in self._fields_}


def make_variant(swap_ab=0, split_k=1, tile_n=None, stages=0, reduce=1, pdl=1, persistent=0) -> Variant:
    if tile_n is None:
        tile_n = 32 if swap_ab else 128
    return Variant(int(swap_ab), int(split_k), int(tile_n), int(stages), int(reduce), int(pdl), int(persistent))


_lib = None
_lock = threading.Lock()

_vp, _i64, _i32, _st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p


def lib() -> ctypes.CDLL:
    """The loaded liblq.so (loaded on first use)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m quantized_linear_gemm_b200.build`")
            L = ctypes.CDLL(LIB_PATH)
            L.lq_scaled_mm.argtypes = [_i32, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, ctypes.POINTER(Variant), _st]
            L.lq_quant_scaled_mm.argtypes = [_i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                             ctypes.POINTER(Variant), _st]
            L.lq_quant_scaled_mm.restype = _i32
            L.lq_scaled_mm_noalloc.argtypes = [_i32, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                               ctypes.POINTER(Variant), _st]
            L.lq_scaled_mm_noalloc.restype = _i32
            L.lq_scaled_mm_i32acc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                              ctypes.POINTER(Variant), _st]
            L.lq_quant_per_token.argtypes = [_i32, _vp, _vp, _vp, _i64, _i64, _st]
            L.lq_quant_per_token_group128.argtypes = [_vp, _vp, _vp, _i64, _i64, _st]
            L.lq_quant_weight_block128.argtypes = [_vp, _vp, _vp, _i64, _i64, _st]
            L.lq_select_variant.argtypes = [_i32, _i64, _i64, _i64, ctypes.POINTER(Variant)]
            L.lq_load_dispatch_table.argtypes = [ctypes.c_char_p]
            L.lq_dispatch_table_size.argtypes = []
            L.lq_dispatch_table_size.restype = _i64
            L.lq_init_device.argtypes = [_i32]
            L.lq_reserve_workspace.argtypes = [_i32, ctypes.c_size_t]
            L.lq_workspace_bytes.argtypes = [_i32, _i64, _i64, _i64, ctypes.POINTER(Variant)]
            L.lq_workspace_bytes.restype = ctypes.c_size_t
            L.lq_device_status.argtypes = [_i32]
            L.lq_status_string.argtypes = [_i32]
            L.lq_status_string.restype = ctypes.c_char_p
            L.lq_test_inject_stall.argtypes = [_i32, ctypes.c_uint64]
            L.lq_test_inject_stall.restype = _i32
            L.lq_test_silu_bf16.argtypes = [_vp, _vp, _i64, _vp]
            L.lq_test_silu_bf16.restype = _i32
            L.lq_set_trace.argtypes = [_vp]
            L.lq_set_trace.restype = _i32
            L.lq_declare_static_weights.argtypes = [_i32]
            L.lq_declare_static_weights.restype = _i32
            L.lq_set_fuse_limit.argtypes = [ctypes.c_int64]
            L.lq_set_fuse_limit.restype = ctypes.c_int64
            L.lq_rms_norm_dynamic_per_token_quant.argtypes = [_i32, _vp, _vp, _vp, ctypes.c_float, _vp, _vp,
                                                              _i64, _i64, _st]
            L.lq_rms_norm_per_block_quant.argtypes = [_vp, _vp, _vp, ctypes.c_float, _vp, _vp, _i64, _i64, _st]
            L.lq_silu_and_mul_dynamic_per_token_quant.argtypes = [_i32, _vp, _vp, _vp, _i64, _i64, _st]
            L.lq_silu_and_mul_per_block_quant.argtypes = [_vp, _vp, _vp, _i64, _i64, _st]
            for name in ("lq_rms_norm_dynamic_per_token_quant", "lq_rms_norm_per_block_quant",
                         "lq_silu_and_mul_dynamic_per_token_quant", "lq_silu_and_mul_per_block_quant"):
                getattr(L, name).restype = _i32
            L.lq_grouped_scaled_mm.argtypes = [_i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                               ctypes.POINTER(Variant), _st]
            L.lq_grouped_scaled_mm.restype = _i32
            for name in ("lq_quant_per_token_group128_ue8m0", "lq_quant_weight_block128_ue8m0"):
                getattr(L, name).argtypes = [_vp, _vp, _vp, _i64, _i64, _st]
                getattr(L, name).restype = _i32
            L.lq_scaled_mm_bias.argtypes = [_i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                            ctypes.POINTER(Variant), _st]
            L.lq_scaled_mm_bias.restype = _i32
            L.lq_quant_weight_int4.argtypes = [_vp, _i64, _vp, _vp, _vp, _i64, _i64, _st]
            L.lq_int4_mm.argtypes = [_vp] * 6 + [_i64] * 4 + [_st]
            L.lq_grouped_int4_mm.argtypes = [_vp] * 6 + [_i64] * 5 + [_st]
            L.lq_moe_sort.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _st]
            L.lq_moe_permute.argtypes = [_vp] * 3 + [_i64] * 4 + [_st]
            L.lq_moe_permute_quant.argtypes = [_i32] + [_vp] * 4 + [_i64] * 4 + [_st]
            L.lq_moe_unpermute.argtypes = [_vp] * 4 + [_i64] * 4 + [_st]
            L.lq_moe_unpermute_backward.argtypes = [_vp] * 6 + [_i64] * 4 + [_st]
            for name in ("lq_quant_weight_int4", "lq_int4_mm", "lq_grouped_int4_mm", "lq_moe_sort", "lq_moe_permute",
                         "lq_moe_permute_quant", "lq_moe_unpermute", "lq_moe_unpermute_backward"):
                getattr(L, name).restype = _i32
            L.lq_version.argtypes = []
            L.lq_version.restype = ctypes.c_char_p
            for name in ("lq_scaled_mm", "lq_scaled_mm_i32acc", "lq_quant_per_token", "lq_quant_per_token_group128",
                         "lq_quant_weight_block128", "lq_select_variant", "lq_load_dispatch_table",
                         "lq_init_device", "lq_reserve_workspace", "lq_device_status"):
                getattr(L, name).restype = _i32
            _lib = L
    return _lib


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise LQError(fn, rc)


def _stream(stream=None) -> int:
    """The handle of `stream`, or of torch's current stream (read directly once
    CUDA is up: building a Stream object costs as much as a launch)."""
    if stream is None:
        if torch.cuda.is_initialized():
            return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _alloc(like: torch.Tensor, shape, stream=None, dtype=None, zero: bool = False) -> torch.Tensor:
    """A new output beside `like`, from the memory of the stream that the call
    runs on (and cleared there): memory of another stream may still be in use
    by work queued on that one, and clearing there could come after the
    kernel's stores.  The caller's current stream is noted as a user, so that a
    dropped output is not handed out again before what was queued there."""
    make = like.new_zeros if zero else like.new_empty
    dtype = like.dtype if dtype is None else dtype
    if stream is None or not like.is_cuda:
        return make(shape, dtype=dtype)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream), device=like.device)
    current = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        out = make(shape, dtype=dtype)
    if current.cuda_stream != stream.cuda_stream:
        out.record_stream(current)
    return out


def _fmt(fmt) -> int:
    if isinstance(fmt, str):
        return FORMATS[fmt]
    return int(fmt)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


_DEVICE_TYPE = "cuda"   # the only device type the library runs on

_CODE_DTYPES = (torch.uint8, torch.int8, torch.float8_e4m3fn)   # one byte per code


def _need(t: torch.Tensor, name: str, dtypes, ndim: int, shape=None) -> None:
    """t is a contiguous ndim-d tensor of one of `dtypes` on the GPU, of
    exactly `shape` when given (the C ABI reads that many elements)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda if _DEVICE_TYPE == "cuda" else t.device.type != _DEVICE_TYPE:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _one_device(*ts) -> None:
    """All tensors on one device, the current CUDA device (the library
    launches on the current device and dereferences every pointer there)."""
    index = ts[0].get_device()
    if index >= 0 and index == torch.cuda.current_device():   # the usual case, without building device objects
        for t in ts:
            if t is not None and t.get_device() != index:
                break
        else:
            return
    ts = [t for t in ts if t is not None]
    dev = ts[0].device
    for t in ts[1:]:
        if t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")
    if dev.type == "cuda" and dev.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {dev} but the current CUDA device is cuda:{torch.cuda.current_device()}")


def _scales_spec(f: int, M: int, N: int, K: int):
    """dtype and shapes of (a_scales, b_scales) for format f: per token and
    per output channel, or per 1 x 128 group and per 128 x 128 block."""
    if f in (BLOCK_FP8, BLOCK_FP8_UE8M0):
        dt = (torch.uint8,) if f == BLOCK_FP8_UE8M0 else (torch.float32,)
        return dt, (M, K // 128), (N // 128, K // 128)
    return (torch.float32,), (M,), (N,)


def _gemm_operands(f: int, A, a_scales, B, b_scales, C):
    """Check the operands of one [M, K] x [N, K]^T product; returns (M, N, K)."""
    _need(A, "A", _CODE_DTYPES, 2)
    _need(B, "B", _CODE_DTYPES, 2)
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("A and B disagree on K")
    dt, sa, sb = _scales_spec(f, M, N, K)
    _need(a_scales, "a_scales", dt, len(sa), sa)
    _need(b_scales, "b_scales", dt, len(sb), sb)
    if C is not None:
        _need(C, "C", (torch.bfloat16,), 2, (M, N))
    _one_device(A, a_scales, B, b_scales, C)
    return M, N, K


def _outputs(like, stream, q, q_shape, q_dtype, scales, s_shape, s_dtype=torch.float32):
    """Allocate the codes / scales outputs of a call on `stream`, or check the caller's."""
    if q is None:
        q = _alloc(like, q_shape, stream, q_dtype)
    else:
        _need(q, "q", _CODE_DTYPES, len(q_shape), q_shape)
    if scales is None:
        scales = _alloc(like, s_shape, stream, s_dtype)
    else:
        _need(scales, "scales", (s_dtype,), len(s_shape), s_shape)
    return q, scales


def _code_dtype(f: int):
    return torch.int8 if f == W8A8_INT8 else torch.uint8


def scaled_mm(fmt, A: torch.Tensor, a_scales: torch.Tensor, B: torch.Tensor, b_scales: torch.Tensor,
              C: torch.Tensor | None = None, variant: Variant | None = None, stream=None) -> torch.Tensor:
    """C[M, N] (bf16) = dequant(A[M, K]) @ dequant(B[N, K])^T through ``lq_scaled_mm``."""
    f = _fmt(fmt)
    M, N, K = _gemm_operands(f, A, a_scales, B, b_scales, C)
    if C is None:
        C = _alloc(A, (M, N), stream, torch.bfloat16)
    rc = lib().lq_scaled_mm(f, _ptr(A), _ptr(a_scales), _ptr(B), _ptr(b_scales), _ptr(C), M, N, K,
                            ctypes.byref(variant) if variant is not None else None, _stream(stream))
    _check("lq_scaled_mm", rc)
    return C


def quant_scaled_mm(fmt, x: torch.Tensor, B: torch.Tensor, b_scales: torch.Tensor, C=None, q=None, s=None,
                    variant: Variant | None = None, stream=None):
    """``lq_quant_scaled_mm``: per-token quantization of bf16 ``x`` fused with
    scaled_mm.  Returns (C, codes, scales)."""
    f = _fmt(fmt)
    _need(x, "x", (torch.bfloat16,), 2)
    _need(B, "B", _CODE_DTYPES, 2)
    M, K = x.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("x and B disagree on K")
    _need(b_scales, "b_scales", (torch.float32,), 1, (N,))
    if C is None:
        C = _alloc(x, (M, N), stream, torch.bfloat16)
    _need(C, "C", (torch.bfloat16,), 2, (M, N))
    q, s = _outputs(x, stream, q, (M, K), _code_dtype(f), s, (M,))
    _one_device(x, B, b_scales, C, q, s)
    rc = lib().lq_quant_scaled_mm(f, _ptr(x), _ptr(B), _ptr(b_scales), _ptr(C), _ptr(q), _ptr(s), M, N, K,
                                  ctypes.byref(variant) if variant is not None else None, _stream(stream))
    _check("lq_quant_scaled_mm", rc)
    return C, q, s


def scaled_mm_bias(fmt, A: torch.Tensor, a_scales: torch.Tensor, B: torch.Tensor, b_scales: torch.Tensor,
                   bias: torch.Tensor, C: torch.Tensor | None = None, variant: Variant | None = None,
                   stream=None) -> torch.Tensor:
    """``lq_scaled_mm_bias``: scaled_mm plus a bf16 bias [N] added before the rounding."""
    f = _fmt(fmt)
    M, N, K = _gemm_operands(f, A, a_scales, B, b_scales, C)
    _need(bias, "bias", (torch.bfloat16,), 1, (N,))
    _one_device(A, bias)
    if C is None:
        C = _alloc(A, (M, N), stream, torch.bfloat16)
    rc = lib().lq_scaled_mm_bias(f, _ptr(A), _ptr(a_scales), _ptr(B), _ptr(b_scales), _ptr(bias), _ptr(C), M, N, K,
                                 ctypes.byref(variant) if variant is not None else None, _stream(stream))
    _check("lq_scaled_mm_bias", rc)
    return C


def grouped_scaled_mm(fmt, A: torch.Tensor, a_scales: torch.Tensor, B: torch.Tensor, b_scales: torch.Tensor,
                      expert_offsets: torch.Tensor, C: torch.Tensor | None = None, variant: Variant | None = None,
                      stream=None) -> torch.Tensor:
    """``lq_grouped_scaled_mm``: A [T, K] tokens sorted by expert, B [E, N, K]
    stacked expert weights, b_scales [E, N], expert_offsets int32 [E + 1] on
    the device.  Returns C [T, N] bf16."""
    f = _fmt(fmt)
    _need(A, "A", _CODE_DTYPES, 2)
    _need(B, "B", _CODE_DTYPES, 3)
    T, K = A.shape
    E, N, KB = B.shape
    if KB != K:
        raise ValueError("A and B disagree on K")
    _need(a_scales, "a_scales", (torch.float32,), 1, (T,))
    _need(b_scales, "b_scales", (torch.float32,), 2, (E, N))
    _need(expert_offsets, "expert_offsets", (torch.int32,), 1, (E + 1,))
    if C is None:
        C = _alloc(A, (T, N), stream, torch.bfloat16)
    _need(C, "C", (torch.bfloat16,), 2, (T, N))
    _one_device(A, a_scales, B, b_scales, expert_offsets, C)
    rc = lib().lq_grouped_scaled_mm(f, _ptr(A), _ptr(a_scales), _ptr(B), _ptr(b_scales), _ptr(C),
                                    _ptr(expert_offsets), E, T, N, K,
                                    ctypes.byref(variant) if variant is not None else None, _stream(stream))
    _check("lq_grouped_scaled_mm", rc)
    return C


def scaled_mm_noalloc(fmt, A: torch.Tensor, a_scales: torch.Tensor, B: torch.Tensor, b_scales: torch.Tensor,
                      C: torch.Tensor | None = None, variant: Variant | None = None, stream=None) -> torch.Tensor:
    """``lq_scaled_mm_noalloc``: scaled_mm whose Split-K partials use the library's
    fixed device array instead of allocated workspace (see include/lq.h)."""
    f = _fmt(fmt)
    M, N, K = _gemm_operands(f, A, a_scales, B, b_scales, C)
    if C is None:
        C = _alloc(A, (M, N), stream, torch.bfloat16)
    rc = lib().lq_scaled_mm_noalloc(f, _ptr(A), _ptr(a_scales), _ptr(B), _ptr(b_scales), _ptr(C), M, N, K,
                                    ctypes.byref(variant) if variant is not None else None, _stream(stream))
    _check("lq_scaled_mm_noalloc", rc)
    return C


def scaled_mm_i32acc(A, a_scales, B, b_scales, C=None, acc=None, variant: Variant | None = None, stream=None):
    """W8A8_INT8 scaled_mm that also returns the exact int32 accumulators."""
    _need(A, "A", (torch.int8,), 2)
    _need(B, "B", (torch.int8,), 2)
    M, N, K = _gemm_operands(W8A8_INT8, A, a_scales, B, b_scales, C)
    if C is None:
        C = _alloc(A, (M, N), stream, torch.bfloat16)
    if acc is None:
        acc = _alloc(A, (M, N), stream, torch.int32)
    _need(acc, "acc", (torch.int32,), 2, (M, N))
    _one_device(A, acc)
    rc = lib().lq_scaled_mm_i32acc(_ptr(A), _ptr(a_scales), _ptr(B), _ptr(b_scales), _ptr(C), _ptr(acc), M, N, K,
                                   ctypes.byref(variant) if variant is not None else None, _stream(stream))
    _check("lq_scaled_mm_i32acc", rc)
    return C, acc


def quant_per_token(fmt, x: torch.Tensor, q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                    stream=None):
    """(codes [M, K], scales [M]) of a bf16 [M, K] tensor; e4m3 codes as uint8, int8 codes as int8."""
    f = _fmt(fmt)
    _need(x, "x", (torch.bfloat16,), 2)
    M, K = x.shape
    q, scales = _outputs(x, stream, q, (M, K), _code_dtype(f), scales, (M,))
    _one_device(x, q, scales)
    rc = lib().lq_quant_per_token(f, _ptr(x), _ptr(q), _ptr(scales), M, K, _stream(stream))
    _check("lq_quant_per_token", rc)
    return q, scales


def quant_per_token_group128(x: torch.Tensor, q=None, scales=None, stream=None):
    """(e4m3 codes [M, K], scales [M, K/128]) of a bf16 [M, K] tensor."""
    _need(x, "x", (torch.bfloat16,), 2)
    M, K = x.shape
    q, scales = _outputs(x, stream, q, (M, K), torch.uint8, scales, (M, max(K // 128, 0)))
    _one_device(x, q, scales)
    rc = lib().lq_quant_per_token_group128(_ptr(x), _ptr(q), _ptr(scales), M, K, _stream(stream))
    _check("lq_quant_per_token_group128", rc)
    return q, scales


def _producer_out(f: int, M: int, K: int, per_block: bool, like, stream, q, scales):
    return _outputs(like, stream, q, (M, K), _code_dtype(f), scales, (M, max(K // 128, 0)) if per_block else (M,))


def _rms_inputs(x, weight, residual):
    _need(x, "x", (torch.bfloat16,), 2)
    M, K = x.shape
    _need(weight, "weight", (torch.bfloat16,), 1, (K,))
    if residual is not None:
        _need(residual, "residual", (torch.bfloat16,), 2, (M, K))
    return M, K


def rms_norm_dynamic_per_token_quant(fmt, x: torch.Tensor, weight: torch.Tensor, eps: float, residual=None,
                                     q=None, scales=None, stream=None):
    """(codes [M, K], scales [M]) of RMSNorm(x [+ residual]) * weight; the
    residual, when given, is overwritten with x + residual."""
    f = _fmt(fmt)
    M, K = _rms_inputs(x, weight, residual)
    q, scales = _producer_out(f, M, K, False, x, stream, q, scales)
    _one_device(x, weight, residual, q, scales)
    rc = lib().lq_rms_norm_dynamic_per_token_quant(f, _ptr(x), _ptr(residual) if residual is not None else None,
                                                   _ptr(weight), float(eps), _ptr(q), _ptr(scales), M, K,
                                                   _stream(stream))
    _check("lq_rms_norm_dynamic_per_token_quant", rc)
    return q, scales


def rms_norm_per_block_quant(x: torch.Tensor, weight: torch.Tensor, eps: float, residual=None, q=None,
                             scales=None, stream=None):
    """(e4m3 codes [M, K], scales [M, K/128]) of RMSNorm(x [+ residual]) * weight."""
    M, K = _rms_inputs(x, weight, residual)
    q, scales = _producer_out(FP8_DYNAMIC, M, K, True, x, stream, q, scales)
    _one_device(x, weight, residual, q, scales)
    rc = lib().lq_rms_norm_per_block_quant(_ptr(x), _ptr(residual) if residual is not None else None, _ptr(weight),
                                           float(eps), _ptr(q), _ptr(scales), M, K, _stream(stream))
    _check("lq_rms_norm_per_block_quant", rc)
    return q, scales


def _gate_up_width(gate_up) -> tuple[int, int]:
    _need(gate_up, "gate_up", (torch.bfloat16,), 2)
    M, two_i = gate_up.shape
    if two_i % 2:
        raise ValueError("gate_up must have an even number of columns ([g | u])")
    return M, two_i // 2


def silu_and_mul_dynamic_per_token_quant(fmt, gate_up: torch.Tensor, q=None, scales=None, stream=None):
    """(codes [M, I], scales [M]) of silu(gate_up[:, :I]) * gate_up[:, I:]."""
    f = _fmt(fmt)
    M, I = _gate_up_width(gate_up)
    q, scales = _producer_out(f, M, I, False, gate_up, stream, q, scales)
    _one_device(gate_up, q, scales)
    rc = lib().lq_silu_and_mul_dynamic_per_token_quant(f, _ptr(gate_up), _ptr(q), _ptr(scales), M, I,
                                                       _stream(stream))
    _check("lq_silu_and_mul_dynamic_per_token_quant", rc)
    return q, scales


def silu_and_mul_per_block_quant(gate_up: torch.Tensor, q=None, scales=None, stream=None):
    """(e4m3 codes [M, I], scales [M, I/128]) of silu(g) * u."""
    M, I = _gate_up_width(gate_up)
    q, scales = _producer_out(FP8_DYNAMIC, M, I, True, gate_up, stream, q, scales)
    _one_device(gate_up, q, scales)
    rc = lib().lq_silu_and_mul_per_block_quant(_ptr(gate_up), _ptr(q), _ptr(scales), M, I, _stream(stream))
    _check("lq_silu_and_mul_per_block_quant", rc)
    return q, scales


def quant_per_token_group128_ue8m0(x: torch.Tensor, q=None, scales=None, stream=None):
    """(e4m3 codes [M, K], UE8M0 scale bytes [M, K/128]) of a bf16 [M, K] tensor."""
    _need(x, "x", (torch.bfloat16,), 2)
    M, K = x.shape
    q, scales = _outputs(x, stream, q, (M, K), torch.uint8, scales, (M, max(K // 128, 0)), torch.uint8)
    _one_device(x, q, scales)
    rc = lib().lq_quant_per_token_group128_ue8m0(_ptr(x), _ptr(q), _ptr(scales), M, K, _stream(stream))
    _check("lq_quant_per_token_group128_ue8m0", rc)
    return q, scales


def quant_weight_block128_ue8m0(w: torch.Tensor, q=None, scales=None, stream=None):
    """(e4m3 codes [N, K], UE8M0 scale bytes [N/128, K/128]) of a bf16 weight [N, K]."""
    _need(w, "w", (torch.bfloat16,), 2)
    N, K = w.shape
    q, scales = _outputs(w, stream, q, (N, K), torch.uint8, scales, (max(N // 128, 0), max(K // 128, 0)),
                         torch.uint8)
    _one_device(w, q, scales)
    rc = lib().lq_quant_weight_block128_ue8m0(_ptr(w), _ptr(q), _ptr(scales), N, K, _stream(stream))
    _check("lq_quant_weight_block128_ue8m0", rc)
    return q, scales


def quant_weight_block128(w: torch.Tensor, q=None, scales=None, stream=None):
    """(e4m3 codes [N, K], scales [N/128, K/128]) of a bf16 weight [N, K]."""
    _need(w, "w", (torch.bfloat16,), 2)
    N, K = w.shape
    q, scales = _outputs(w, stream, q, (N, K), torch.uint8, scales, (max(N // 128, 0), max(K // 128, 0)))
    _one_device(w, q, scales)
    rc = lib().lq_quant_weight_block128(_ptr(w), _ptr(q), _ptr(scales), N, K, _stream(stream))
    _check("lq_quant_weight_block128", rc)
    return q, scales


INT4_GROUPS = (32, 64, 128)


def quant_weight_int4(w: torch.Tensor, group: int = 128, zero_points: bool = False, q=None, scales=None, zeros=None,
                      stream=None):
    """``lq_quant_weight_int4``: (packed codes uint8 [N, K/2], scales bf16
    [N, K/group], zero points uint8 [N, K/group] or None) of a bf16 weight
    [N, K]; symmetric unless ``zero_points`` (or ``zeros`` is given)."""
    _need(w, "w", (torch.bfloat16,), 2)
    N, K = w.shape
    if group not in INT4_GROUPS or K % group:
        raise ValueError(f"group must be one of {INT4_GROUPS} and divide K = {K}, got {group}")
    q, scales = _outputs(w, stream, q, (N, K // 2), torch.uint8, scales, (N, K // group), torch.bfloat16)
    if zeros is not None:
        _need(zeros, "zeros", (torch.uint8,), 2, (N, K // group))
    elif zero_points:
        zeros = _alloc(w, (N, K // group), stream, torch.uint8)
    _one_device(w, q, scales, zeros)
    _check("lq_quant_weight_int4", lib().lq_quant_weight_int4(_ptr(w), group, _ptr(q), _ptr(scales), _ptr(zeros), N, K,
                                                              _stream(stream)))
    return q, scales, zeros


def _int4_operands(x, B, b_scales, b_zeros, lead: tuple):
    """Check x [M, K] and a 4-bit weight with leading dimensions `lead`
    (() or (E,)); returns (M, N, K, group)."""
    _need(x, "x", (torch.bfloat16,), 2)
    _need(B, "B", (torch.uint8,), 2 + len(lead))
    M, K = x.shape
    *_, N, row = B.shape
    if row * 2 != K:
        raise ValueError(f"B has {row} bytes per row, expected K / 2 with K = {K}")
    _need(b_scales, "b_scales", (torch.bfloat16,), 2 + len(lead))
    have = b_scales.shape
    groups = have[-1]
    if groups == 0 or K % groups or K // groups not in INT4_GROUPS:
        raise ValueError(f"b_scales has {groups} groups per row: K = {K} must hold whole groups of {INT4_GROUPS}")
    want = (*lead, N, groups)
    if have != want:
        raise ValueError(f"b_scales has shape {tuple(have)}, expected {want}")
    if b_zeros is not None:
        _need(b_zeros, "b_zeros", (torch.uint8,), 2 + len(lead), want)
    return M, N, K, K // groups


def int4_mm(x: torch.Tensor, B: torch.Tensor, b_scales: torch.Tensor, b_zeros: torch.Tensor | None = None,
            bias: torch.Tensor | None = None, C: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``lq_int4_mm``: C [M, N] bf16 = x [M, K] bf16 times the 4-bit weight
    (packed codes B [N, K/2], scales [N, K/group], optional zero points), plus
    an optional bf16 bias [N].  The group size follows from the shapes."""
    M, N, K, group = _int4_operands(x, B, b_scales, b_zeros, ())
    if bias is not None:
        _need(bias, "bias", (torch.bfloat16,), 1, (N,))
    if C is None:
        C = _alloc(x, (M, N), stream)
    else:
        _need(C, "C", (torch.bfloat16,), 2, (M, N))
    _one_device(x, B, b_scales, b_zeros, bias, C)
    _check("lq_int4_mm", lib().lq_int4_mm(_ptr(x), _ptr(B), _ptr(b_scales), _ptr(b_zeros), _ptr(bias), _ptr(C), M, N, K,
                                          group, _stream(stream)))
    return C


def grouped_int4_mm(x: torch.Tensor, B: torch.Tensor, b_scales: torch.Tensor, expert_offsets: torch.Tensor,
                    b_zeros: torch.Tensor | None = None, C: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``lq_grouped_int4_mm``: x [T, K] bf16 sorted by expert, B [E, N, K/2]
    packed codes, b_scales (and b_zeros) [E, N, K/group], expert_offsets int32
    [E + 1] on the device.  Returns C [T, N] bf16; rows outside every expert
    are left as they were, which in a C allocated here is undefined."""
    if not isinstance(B, torch.Tensor):
        raise TypeError("B must be a tensor")
    if B.dim() != 3:
        raise ValueError("B must be a contiguous 3-d tensor [E, N, K / 2]")
    E = B.shape[0]
    T, N, K, group = _int4_operands(x, B, b_scales, b_zeros, (E,))
    _need(expert_offsets, "expert_offsets", (torch.int32,), 1, (E + 1,))
    if C is None:
        C = _alloc(x, (T, N), stream)
    else:
        _need(C, "C", (torch.bfloat16,), 2, (T, N))
    _one_device(x, B, b_scales, b_zeros, expert_offsets, C)
    _check("lq_grouped_int4_mm", lib().lq_grouped_int4_mm(_ptr(x), _ptr(B), _ptr(b_scales), _ptr(b_zeros), _ptr(C),
                                                          _ptr(expert_offsets), E, T, N, K, group, _stream(stream)))
    return C


def moe_sort(topk_ids: torch.Tensor, num_experts: int, expert_offsets=None, order=None, slots=None, stream=None):
    """``lq_moe_sort``: (expert_offsets int32 [E + 1], order int32 [T * k],
    slots int32 [T, k]) of the expert ids int32 or int64 [T, k]; ids outside
    [0, num_experts) take no row (slot -1)."""
    _need(topk_ids, "topk_ids", (torch.int32, torch.int64), 2)
    T, k = topk_ids.shape
    E, n = int(num_experts), T * k
    if expert_offsets is None and order is None and slots is None and E >= 0:   # one allocation, cut in three
        buf = _alloc(topk_ids, (E + 1 + 2 * n,), stream, torch.int32)
        offs, rows, cut = torch.unsafe_split_with_sizes(buf, (E + 1, n, n))
        outs = (offs, rows, cut.view(T, k))
        _one_device(topk_ids)
    else:
        outs = []
        for name, t, shape in (("expert_offsets", expert_offsets, (E + 1,)), ("order", order, (n,)),
                               ("slots", slots, (T, k))):
            if t is None:
                t = _alloc(topk_ids, shape, stream, torch.int32)
            else:
                _need(t, name, (torch.int32,), len(shape), shape)
            outs.append(t)
        _one_device(topk_ids, *outs)
    _check("lq_moe_sort", lib().lq_moe_sort(_ptr(topk_ids), topk_ids.element_size(), n, E, *map(_ptr, outs),
                                            _stream(stream)))
    return tuple(outs)


def _token_slots(slots, T: int) -> int:
    _need(slots, "slots", (torch.int32,), 2)
    if slots.shape[0] != T:
        raise ValueError(f"slots has {slots.shape[0]} tokens, expected {T}")
    return slots.shape[1]


def moe_permute(x: torch.Tensor, slots: torch.Tensor, xs: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``lq_moe_permute``: xs[slots[t, j]] = x[t] for bf16 x [T, H] and slots
    int32 [T, k].  xs [P, H] (default P = T * k); rows that no slot names are
    left as they were, which in an xs allocated here is undefined."""
    _need(x, "x", (torch.bfloat16,), 2)
    T, H = x.shape
    k = _token_slots(slots, T)
    if xs is None:
        xs = _alloc(x, (T * k, H), stream)
    else:
        _need(xs, "xs", (torch.bfloat16,), 2)
        if xs.shape[1] != H:
            raise ValueError(f"xs has rows of {xs.shape[1]} values, expected {H}")
    _one_device(x, slots, xs)
    _check("lq_moe_permute", lib().lq_moe_permute(_ptr(x), _ptr(slots), _ptr(xs), T, xs.shape[0], k, H,
                                                  _stream(stream)))
    return xs


def moe_permute_quant(fmt, x: torch.Tensor, slots: torch.Tensor, q: torch.Tensor | None = None,
                      scales: torch.Tensor | None = None, stream=None):
    """``lq_moe_permute_quant``: (codes [P, H], scales fp32 [P]) of x [T, H]
    quantized per token (``fp8_dynamic`` or ``w8a8_int8``) and placed at its
    slots; P = T * k unless q is given.  Rows that no slot names are left as
    they were, which in outputs allocated here is undefined."""
    f = _fmt(fmt)
    _need(x, "x", (torch.bfloat16,), 2)
    T, H = x.shape
    k = _token_slots(slots, T)
    if q is not None:
        _need(q, "q", _CODE_DTYPES, 2)
    P = T * k if q is None else q.shape[0]
    q, scales = _outputs(x, stream, q, (P, H), _code_dtype(f), scales, (P,))
    _one_device(x, slots, q, scales)
    _check("lq_moe_permute_quant", lib().lq_moe_permute_quant(f, _ptr(x), _ptr(slots), _ptr(q), _ptr(scales), T, P, k,
                                                              H, _stream(stream)))
    return q, scales


def moe_unpermute(y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``lq_moe_unpermute``: out[t] = sum_j weights[t, j] * y[slots[t, j]] for
    bf16 y [P, H], slots int32 [T, k] and fp32 weights [T, k] (None: ones);
    skipped slots (-1) add nothing.  Returns bf16 [T, H]."""
    _need(y, "y", (torch.bfloat16,), 2)
    _need(slots, "slots", (torch.int32,), 2)
    P, H = y.shape
    T, k = slots.shape
    if weights is not None:
        _need(weights, "weights", (torch.float32,), 2, (T, k))
    if out is None:
        out = _alloc(y, (T, H), stream)
    else:
        _need(out, "out", (torch.bfloat16,), 2, (T, H))
    _one_device(y, slots, weights, out)
    _check("lq_moe_unpermute", lib().lq_moe_unpermute(_ptr(y), _ptr(slots), _ptr(weights), _ptr(out), T, P, k, H,
                                                      _stream(stream)))
    return out


def moe_permute_backward(dxs: torch.Tensor, slots: torch.Tensor, dx: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Gradient of moe_permute: dx[t] = sum_j dxs[slots[t, j]]
    (``lq_moe_unpermute`` without weights); rows without a slot are not read."""
    return moe_unpermute(dxs, slots, None, out=dx, stream=stream)


def moe_unpermute_backward(dout: torch.Tensor, y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor,
                           dy: torch.Tensor | None = None, dweights: torch.Tensor | None = None, stream=None):
    """``lq_moe_unpermute_backward``: (dy bf16 [P, H], dweights fp32 [T, k]) of
    moe_unpermute(y, slots, weights) for the gradient dout bf16 [T, H].  Rows
    that no slot names have gradient zero in a dy allocated here; in the
    caller's dy they are left as they were, which saves clearing it.  (Without
    weights the gradient is moe_permute(dout, slots, xs=zeros).)"""
    _need(y, "y", (torch.bfloat16,), 2)
    _need(slots, "slots", (torch.int32,), 2)
    P, H = y.shape
    T, k = slots.shape
    _need(dout, "dout", (torch.bfloat16,), 2, (T, H))
    _need(weights, "weights", (torch.float32,), 2, (T, k))
    if dy is None:
        dy = _alloc(y, (P, H), stream, zero=True)
    else:
        _need(dy, "dy", (torch.bfloat16,), 2, (P, H))
    if dweights is None:
        dweights = _alloc(weights, (T, k), stream)
    else:
        _need(dweights, "dweights", (torch.float32,), 2, (T, k))
    _one_device(dout, y, slots, weights, dy, dweights)
    _check("lq_moe_unpermute_backward", lib().lq_moe_unpermute_backward(
        _ptr(dout), _ptr(y), _ptr(slots), _ptr(weights), _ptr(dy), _ptr(dweights), T, P, k, H, _stream(stream)))
    return dy, dweights


def select_variant(fmt, M: int, N: int, K: int) -> Variant:
    v = Variant()
    _check("lq_select_variant", lib().lq_select_variant(_fmt(fmt), M, N, K, ctypes.byref(v)))
    return v


def load_dispatch_table(path: str | None) -> None:
    _check("lq_load_dispatch_table", lib().lq_load_dispatch_table(None if path is None else path.encode()))


def dispatch_table_size() -> int:
    return int(lib().lq_dispatch_table_size())


def init_device(device: int = 0) -> None:
    _check("lq_init_device", lib().lq_init_device(device))


def reserve_workspace(device: int, nbytes: int) -> None:
    _check("lq_reserve_workspace", lib().lq_reserve_workspace(device, nbytes))


def workspace_bytes(fmt, M, N, K, variant: Variant | None = None) -> int:
    return int(lib().lq_workspace_bytes(_fmt(fmt), M, N, K, ctypes.byref(variant) if variant is not None else None))


def device_status(device: int = 0) -> int:
    """Read and clear the device status word: 0, or LQ_ERR_DEVICE_TIMEOUT (6)."""
    return int(lib().lq_device_status(device))


def set_trace(buf: torch.Tensor | None) -> None:
    """Record 12 globaltimer stamps per CTA of the following scaled_mm launches
    into ``buf`` (a contiguous 1-d int64 CUDA tensor), or stop (None).  The
    library cannot know the grids to come: ``buf`` must hold 12 entries for
    every CTA of the largest launch made while tracing is on."""
    if buf is not None:
        _need(buf, "buf", (torch.int64,), 1)
        _one_device(buf)
    lib().lq_set_trace(None if buf is None else buf.data_ptr())


def declare_static_weights(static: bool = True) -> bool:
    """Declare that weights are never written while a GEMM reading them may
    run, so that a default (None) variant may stream weight tiles before the
    previous kernel finishes; returns the previous setting."""
    return bool(lib().lq_declare_static_weights(1 if static else 0))


def set_fuse_limit(max_slice_bytes: int) -> int:
    """Largest per-CTA activation slice (bytes) for which quant_scaled_mm
    runs one kernel (0 = never, negative = default); returns the old limit."""
    return int(lib().lq_set_fuse_limit(int(max_slice_bytes)))


def test_inject_stall(k_tile: int, wait_limit_ns: int = 0) -> None:
    """Test hook: leave K tile `k_tile` of every CTA unloaded so that a bounded
    wait runs out (-1 = off); `wait_limit_ns` > 0 shortens every wait."""
    _check("lq_test_inject_stall", lib().lq_test_inject_stall(int(k_tile), int(wait_limit_ns)))


def test_silu_bf16(gate: torch.Tensor, stream=None) -> torch.Tensor:
    """Test hook: bf16(silu(gate)) by the producer kernels' own device code."""
    if gate.dtype != torch.bfloat16 or not gate.is_cuda or not gate.is_contiguous():
        raise ValueError("gate must be a contiguous bf16 CUDA tensor")
    out = _alloc(gate, gate.shape, stream)
    _check("lq_test_silu_bf16", lib().lq_test_silu_bf16(_ptr(gate), _ptr(out), gate.numel(), _stream(stream)))
    return out


def status_string(code: int) -> str:
    return lib().lq_status_string(code).decode()


def version() -> str:
    return lib().lq_version().decode()


def call_raw(name: str, *args) -> int:
    """Call a C entry point with raw arguments (for argument-check tests)."""
    return int(getattr(lib(), name)(*args))


@dataclass(frozen=True)
class Problem:
    """A (format, M, N, K) GEMM shape."""
    fmt: int
    M: int
    N: int
    K: int

    @property
    def flops(self) -> int:
        return 2 * self.M * self.N * self.K

    @property
    def bytes(self) -> int:
        """Algorithmic HBM bytes: weights + activations + scales + bf16 output."""
        if self.fmt in (BLOCK_FP8, BLOCK_FP8_UE8M0):
            per = 1 if self.fmt == BLOCK_FP8_UE8M0 else 4   # UE8M0 scales are bytes
            scales = per * (self.M * (self.K // 128) + (self.N // 128) * (self.K // 128))
        else:
            scales = 4 * (self.M + self.N)
        return self.N * self.K + self.M * self.K + scales + 2 * self.M * self.N
