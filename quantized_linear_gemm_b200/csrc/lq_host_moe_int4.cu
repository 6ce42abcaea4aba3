// Entry points of the 4-bit weight products and of the mixture-of-experts
// token movement: argument checks, then one launch each (include/lq.h).
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/lq.h"
#include "lq_kernels.h"

namespace {

constexpr int64_t kMaxInt = 0x7FFFFFFF;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

lq_status launched(cudaError_t e) {
  if (e == cudaSuccess) return LQ_OK;
  cudaGetLastError();
  return LQ_ERR_CUDA;
}

bool group_ok(int64_t group) { return group == 32 || group == 64 || group == 128; }

// Which kernel a product takes: 0, the streaming kernel (mma.sync, at most 16
// tokens per tile); else the tensor-core kernel with that many tokens per tile.
//
// Measured on B200, us (streaming / tensor core).  Dense, G = 128: 1 token
// [4096, 4096] 4.7 / 7.3, [24576, 4096] 15.5 / 19, [4096, 12288] 9.9 / 12.4,
// [5120, 25600] 32.8 / 21.5; 16 tokens 10.2 / 7.0, 27.3 / 22, 23.1 / 12.4,
// 66.5 / 22.  G = 64 (the streaming kernel loads 8 bytes at a time there):
// [24576, 4096] 1 token 24.3 / 21.3, 8 tokens 25.2 / 21.3, with zero points
// 31.1 / 25.2 and 32.3 / 24.8; [16384, 4096] 1 token 16.7 / 15.3; [12288, 4096]
// 1 token 12.9 / 15.1, 8 tokens 14.1 / 15.1.
// Grouped, 128 experts, [1536, 2048] each: 8 rows 7.1 / 10.6, 64 rows 35 / 29,
// 512 rows 86 / 56.  More experts than the tensor-core kernel keeps take the
// streaming kernel at any number of rows.
//
// A grouped tile covers one and a half times the average expert, since the
// offsets are on the device.  [1536, 2048], evenly routed: 256 rows 51, 55, 56 us
// with tiles of 16, 32, 64; 8008 rows 127, 88, 89, 123 with 32, 64, 128, 256;
// 32768 rows 266, 227, 214 with 64, 128, 256.  With half of the rows on four
// experts, or very uneven shares, the rule's tile is at most 17 % behind the best
// one: 1024 rows 66.0 (64.2 with 32) and 54.3 (46.3 with 32), 8008 rows 101
// (92.3 with 64) and 89.2 (the best), 32768 rows 230 (221 with 256) and 229 (222).
int tensor_tile(int64_t M, int64_t N, int64_t K, int64_t group, int64_t experts) {
  if (experts) {
    if (M <= (experts > 1 ? 16 : 8) || experts > lq::int4_mma_max_experts()) return 0;
    const int64_t want = (M + M / 2) / experts;
    return want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 ? 64 : want <= 1024 ? 128 : 256;
  }
  if (M <= 8 && K <= 16384 && (group != 64 || N < 16384)) return 0;
  return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
}

// Shared by the dense (E = 1) and grouped products.
lq_status int4_mm_impl(const void* x, const void* B, const void* scales, const void* zeros, const void* bias, void* C,
                       const int32_t* offsets, bool grouped, int64_t E, int64_t M, int64_t N, int64_t K,
                       int64_t group, lq_stream_t stream_) {
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (M < 0 || N < 0 || K < 0 || E < 0 || !group_ok(group)) return LQ_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return LQ_OK;
  if (!C || (grouped && (E == 0 || !offsets))) return LQ_ERR_INVALID_ARG;
  if (!x || !B || !scales) return LQ_ERR_INVALID_ARG;
  if (!aligned(C, 16) || !aligned(x, 16) || !aligned(B, 16) || !aligned(scales, 2) || (bias && !aligned(bias, 2)) ||
      (offsets && !aligned(offsets, 4)))
    return LQ_ERR_ALIGNMENT;
  if (K == 0 || K % group != 0 || N % 8 != 0) return LQ_ERR_UNSUPPORTED_SHAPE;
  // the kernels round M up to a token tile in 32 bits
  if (M > kMaxInt - 255 || K > (int64_t(1) << 24) || E > kMaxInt || N > kMaxInt || E * N > kMaxInt)
    return LQ_ERR_UNSUPPORTED_SHAPE;
  lq::Int4Params p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.B = static_cast<const uint8_t*>(B);
  p.scales = static_cast<const __nv_bfloat16*>(scales);
  p.zeros = static_cast<const uint8_t*>(zeros);
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.C = static_cast<__nv_bfloat16*>(C);
  p.M = M;
  p.N = N;
  p.K = K;
  p.expert_offsets = grouped ? offsets : nullptr;
  p.num_experts = static_cast<int>(E);
  p.early_weights = lq::static_weights_declared() ? 1 : 0;
  const int per_block = static_cast<int>(128 / group);   // groups per 128-wide block
  p.vec_scales = K % 128 == 0 && aligned(scales, 2 * per_block) && (!zeros || aligned(zeros, per_block));
  const int rc = lq::device_status_word(stream, &p.status, &p.wait_limit_ns);
  if (rc != LQ_OK) return static_cast<lq_status>(rc);
  p.skip_block = lq::skipped_block();
  const int tile = tensor_tile(M, N, K, group, grouped ? E : 0);
  if (tile) {
    const int64_t spare = grouped ? (E < M ? E : M) : 0;     // token tiles beyond M / tile, at most
    if (((N + 127) / 128) * ((M + tile - 1) / tile + spare) > kMaxInt / 2) return LQ_ERR_UNSUPPORTED_SHAPE;
    return launched(lq::launch_int4_mma(p, static_cast<int>(group), tile, stream));
  }
  return launched(lq::launch_int4_mm(p, static_cast<int>(group), stream));
}

// Shared checks of the row movements: T tokens of k slots, rows of H values.
lq_status check_rows(int64_t T, int64_t P, int64_t k, int64_t H, int64_t multiple) {
  if (T < 0 || P < 0 || k < 0 || H < 0) return LQ_ERR_INVALID_ARG;
  if (H % multiple != 0 || T > kMaxInt || k > (int64_t(1) << 24) || P > kMaxInt || H > (int64_t(1) << 25))
    return LQ_ERR_UNSUPPORTED_SHAPE;
  return LQ_OK;
}

}  // namespace

extern "C" {

lq_status lq_quant_weight_int4(const void* w, int64_t group, void* q, void* scales, void* zeros, int64_t N, int64_t K,
                               lq_stream_t stream) {
  if (N < 0 || K < 0 || !group_ok(group)) return LQ_ERR_INVALID_ARG;
  if (N == 0 || K == 0) return LQ_OK;
  if (!w || !q || !scales) return LQ_ERR_INVALID_ARG;
  if (!aligned(w, 16) || !aligned(q, 4) || !aligned(scales, 2)) return LQ_ERR_ALIGNMENT;
  if (K % group != 0 || K > kMaxInt || N > kMaxInt || (N * K / 8 + 255) / 256 > kMaxInt)
    return LQ_ERR_UNSUPPORTED_SHAPE;
  return launched(lq::launch_quant_weight_int4(w, static_cast<int>(group), q, scales, zeros, N, K,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

lq_status lq_int4_mm(const void* x, const void* B, const void* b_scales, const void* b_zeros, const void* bias,
                     void* C, int64_t M, int64_t N, int64_t K, int64_t group, lq_stream_t stream) {
  return int4_mm_impl(x, B, b_scales, b_zeros, bias, C, nullptr, false, 1, M, N, K, group, stream);
}

lq_status lq_grouped_int4_mm(const void* x, const void* B, const void* b_scales, const void* b_zeros, void* C,
                             const int32_t* expert_offsets, int64_t E, int64_t T, int64_t N, int64_t K, int64_t group,
                             lq_stream_t stream) {
  return int4_mm_impl(x, B, b_scales, b_zeros, nullptr, C, expert_offsets, true, E, T, N, K, group, stream);
}

lq_status lq_moe_sort(const void* ids, int64_t id_bytes, int64_t n, int64_t E, int32_t* expert_offsets,
                      int32_t* order, int32_t* slots, lq_stream_t stream) {
  if (n < 0 || E < 0 || (id_bytes != 4 && id_bytes != 8)) return LQ_ERR_INVALID_ARG;
  if (!expert_offsets || (n > 0 && (!ids || !order || !slots))) return LQ_ERR_INVALID_ARG;
  if (!aligned(ids, static_cast<uintptr_t>(id_bytes)) || !aligned(expert_offsets, 4) || !aligned(order, 4) ||
      !aligned(slots, 4))
    return LQ_ERR_ALIGNMENT;
  if (E == 0 || E > lq::moe_sort_max_experts() || n > kMaxInt) return LQ_ERR_UNSUPPORTED_SHAPE;
  return launched(lq::launch_moe_sort(ids, static_cast<int>(id_bytes), n, static_cast<int>(E), expert_offsets, order,
                                      slots, reinterpret_cast<cudaStream_t>(stream)));
}

lq_status lq_moe_permute(const void* x, const int32_t* slots, void* xs, int64_t T, int64_t P, int64_t k, int64_t H,
                         lq_stream_t stream) {
  const lq_status rc = check_rows(T, P, k, H, 8);
  if (rc != LQ_OK) return rc;
  if (T == 0 || P == 0 || k == 0 || H == 0) return LQ_OK;
  if (!x || !slots || !xs) return LQ_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(xs, 16) || !aligned(slots, 4)) return LQ_ERR_ALIGNMENT;
  return launched(lq::launch_moe_permute(x, slots, xs, T, P, static_cast<int>(k), H,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

lq_status lq_moe_permute_quant(lq_fmt fmt, const void* x, const int32_t* slots, void* q, float* scales, int64_t T,
                               int64_t P, int64_t k, int64_t H, lq_stream_t stream) {
  if (fmt != LQ_FP8_DYNAMIC && fmt != LQ_W8A8_INT8) return LQ_ERR_INVALID_ARG;
  const lq_status rc = check_rows(T, P, k, H, 16);
  if (rc != LQ_OK) return rc;
  if (T == 0 || P == 0 || k == 0) return LQ_OK;
  if (!x || !slots || !q || !scales) return LQ_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 8) || !aligned(scales, 4) || !aligned(slots, 4)) return LQ_ERR_ALIGNMENT;
  return launched(lq::launch_moe_permute_quant(static_cast<int>(fmt), x, slots, q, scales, T, P, static_cast<int>(k),
                                               H, reinterpret_cast<cudaStream_t>(stream)));
}

lq_status lq_moe_unpermute(const void* y, const int32_t* slots, const float* weights, void* out, int64_t T, int64_t P,
                           int64_t k, int64_t H, lq_stream_t stream) {
  const lq_status rc = check_rows(T, P, k, H, 8);
  if (rc != LQ_OK) return rc;
  if (T == 0 || H == 0) return LQ_OK;
  if (!out || (k > 0 && !slots) || (k > 0 && P > 0 && !y)) return LQ_ERR_INVALID_ARG;
  if (!aligned(y, 16) || !aligned(out, 16) || !aligned(slots, 4) || !aligned(weights, 4)) return LQ_ERR_ALIGNMENT;
  return launched(lq::launch_moe_unpermute(y, slots, weights, out, T, P, static_cast<int>(k), H,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

lq_status lq_moe_unpermute_backward(const void* dout, const void* y, const int32_t* slots, const float* weights,
                                    void* dy, float* dweights, int64_t T, int64_t P, int64_t k, int64_t H,
                                    lq_stream_t stream) {
  const lq_status rc = check_rows(T, P, k, H, 8);
  if (rc != LQ_OK) return rc;
  if (T == 0 || k == 0) return LQ_OK;
  if (!slots || !weights || !dweights) return LQ_ERR_INVALID_ARG;
  if (H > 0 && (!dout || (P > 0 && (!y || !dy)))) return LQ_ERR_INVALID_ARG;
  if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16) || !aligned(slots, 4) || !aligned(weights, 4) ||
      !aligned(dweights, 4))
    return LQ_ERR_ALIGNMENT;
  return launched(lq::launch_moe_unpermute_backward(dout, y, slots, weights, dy, dweights, T, P, static_cast<int>(k),
                                                    H, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
