// 4-bit weight codes -> bf16, and the tiles of a grouped product, shared by the
// 4-bit weight kernels.
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

// The expert that owns token tile `tile` when every expert's rows are cut
// into tiles of `per` tokens: its rows [*lo, *hi) of the tile.  Offsets are
// clamped to [0, T] and to their running maximum, so a malformed table never
// leads outside the rows.  Called by whole warps; false: no such tile.
__device__ __forceinline__ bool find_expert_tile(const int* __restrict__ offsets, int E, int T, int per, int tile,
                                                 int* expert, int* lo, int* hi) {
  const int lane = threadIdx.x & 31;
  int before = 0;                        // tiles of the experts so far
  int carry = __ldg(offsets);            // running maximum so far
  carry = carry < 0 ? 0 : (carry > T ? T : carry);
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    int end = e < E ? __ldg(offsets + e + 1) : 0;
    end = end < 0 ? 0 : (end > T ? T : end);
    end = end > carry ? end : carry;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o && v > end) end = v;
    }
    int begin = __shfl_up_sync(0xffffffffu, end, 1);
    if (lane == 0) begin = carry;
    const int tiles = e < E ? (end - begin + per - 1) / per : 0;
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const int mine = before + upto - tiles;   // first tile of this lane's expert
    const uint32_t has = __ballot_sync(0xffffffffu, tile >= mine && tile < mine + tiles);
    if (has) {
      const int src = __ffs(has) - 1;
      const int b = __shfl_sync(0xffffffffu, begin, src), en = __shfl_sync(0xffffffffu, end, src);
      *expert = e0 + src;
      *lo = b + (tile - __shfl_sync(0xffffffffu, mine, src)) * per;
      *hi = *lo + per < en ? *lo + per : en;
      return true;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
    carry = __shfl_sync(0xffffffffu, end, 31);
  }
  return false;
}

}  // namespace lq
