// 4-bit weight codes -> bf16, shared by the 4-bit weight kernels.
//
// A 32-bit word holds the codes of 8 consecutive k, code i in bits
// [4 i, 4 i + 4).  A bf16 whose exponent field is 0 or 1 is the plain integer
// of its low 8 bits times 2^-133 (subnormals, then the first binade with the
// same step).  So with the even codes masked into one word and the odd ones
// (16 times their value) into another, a byte permutation puts codes 2 i and
// 2 i + 1 into the two halves as exact bf16 values, and one fused
// multiply-add per pair,
//   {q 2^-133, 16 q 2^-133} {2^127, 2^123} - z 2^-6,
// gives (q - z) / 64 exactly: six integer instructions per 8 codes, two of
// mask and four of permutation.  (Or-ing an exponent in, the 128 + q form,
// needs each nibble shifted to the bottom and its partner moved: eleven.  The
// integer pipe, at half the rate of the multiply-add pipe, is what bounds the
// conversion.)  The factor 64 is put back in fp32 or into the scale.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

namespace lq {

__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// prmt with the sign-replicating selectors (8 + byte)
__device__ __forceinline__ uint32_t byte_select(uint32_t a, uint32_t b, uint32_t selector) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(selector));
  return d;
}

constexpr uint32_t kInt4Factors = 0x7D007F00u;       // {2^127, 2^123}
constexpr uint32_t kInt4MidOffset = 0xBE00BE00u;     // {-8 / 64, -8 / 64}: no zero points
constexpr float kInt4Unit = 64.f;                    // the codes come out as (q - z) / 64

// bf16x2 {-z / 64, -z / 64}, z in 0..15, by the same subnormal reading
__device__ __forceinline__ uint32_t int4_offset(uint32_t z) {
  return bf16x2_fma((z & 15u) * 0x10001u, 0xFF00FF00u /* -2^127 */, 0u);
}

// out[i] = bf16x2 {(q_(2i) - z) / 64, (q_(2i+1) - z) / 64}, offset = int4_offset(z)
__device__ __forceinline__ void int4_word_to_bf16(uint32_t w, uint32_t offset, uint32_t (&out)[4]) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = w & 0xF0F0F0F0u;
  // bytes {lo.b, 0, hi.b, 0}: selector 8 + b replicates the sign bit of a byte of lo, which is 0
  out[0] = bf16x2_fma(byte_select(lo, hi, 0x8480), kInt4Factors, offset);
  out[1] = bf16x2_fma(byte_select(lo, hi, 0x8581), kInt4Factors, offset);
  out[2] = bf16x2_fma(byte_select(lo, hi, 0x8682), kInt4Factors, offset);
  out[3] = bf16x2_fma(byte_select(lo, hi, 0x8783), kInt4Factors, offset);
}

}  // namespace lq
