// 4-bit weight codes -> bf16, shared by the 4-bit weight kernels.
//
// A 32-bit word holds the codes of 8 consecutive k, code i in bits
// [4 i, 4 i + 4).  Masking a shift of the word by 0x000F000F leaves codes i
// and i + 4 in the two halves; or-ing 0x4300 into each half makes them the
// bf16 values 128 + q (bf16 has 7 mantissa bits, so one unit at 128 is one
// code), and subtracting 128 + z gives q - z exactly: three instructions per
// two codes and no conversion.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

namespace lq {

// bf16x2 {128 + z, 128 + z}, z in 0..15
__device__ __forceinline__ uint32_t int4_offset(uint32_t z) { return (0x4300u | (z & 15u)) * 0x10001u; }
constexpr uint32_t kInt4MidOffset = 0x43084308u;   // z = 8: no zero points

__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// out[i] = bf16x2 {q_i - z, q_(i+4) - z}, offset = int4_offset(z)
__device__ __forceinline__ void int4_word_to_bf16(uint32_t w, uint32_t offset, uint32_t (&out)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = bf16x2_sub(((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u, offset);
}

}  // namespace lq
