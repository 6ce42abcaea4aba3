// 4-bit weights with a scale (and optionally a zero point) per group of G
// weights of a row: the quantizer, and the product with bf16 activations for
// few tokens.
//
//   C[m, n] = bf16( sum_g s[n, g] * sum_{k in g} (q[n, k] - z[n, g]) x[m, k]
//                   + bias[n] )
//
// A weight-only format beside the 8-bit ones of the PyTorch blog "Building a
// High-Performance and Portable vLLM Linear Backend with Helion", section
// "Helion Linear Backend > Scope": at decode the product is bound by the
// bytes of the weight, and this halves them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cfloat>
#include <cstdint>

#include "int4_common.cuh"
#include "lq_kernels.h"
#include "ptx.cuh"
#include "quant_common.cuh"

namespace lq {
namespace {

// ------------------------------------------------------------- quantizer
//
// One thread per 8 weights (16 bytes in, 4 out), a group's extrema by
// shuffles among its G / 8 lanes.  Symmetric: s = max(bf16(amax / 7), 2^-126),
// q = clamp(rint(w / s), -8, 7) + 8.  With zero points: lo = min(0, min w),
// hi = max(0, max w), s = max(bf16((hi - lo) / 15), 2^-126),
// z = clamp(rint(-lo / s), 0, 15), q = clamp(rint(w / s) + z, 0, 15).  Every
// quotient is the correctly rounded fp32 one and rint rounds half to even;
// the codes are those of the bf16 scale that is stored.
//
// Run once per weight.  Held back by the issue of eight correctly rounded
// divisions per thread, not by HBM: [24576, 4096], G = 128, 84 us (3.0 TB/s,
// 0.46 of the copy rate), with zero points 90 us; [4096, 4096] 15 us.  That is no
// floor: one reciprocal per group and corrected products (quotient8) would give
// the same quotients with fewer instructions.
template <int G, bool kZeros>
__global__ void __launch_bounds__(256) quant_weight_int4_kernel(const uint4* __restrict__ w,
                                                                uint32_t* __restrict__ q,
                                                                __nv_bfloat16* __restrict__ scales,
                                                                uint8_t* __restrict__ zeros, int64_t words) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const bool valid = i < words;   // groups are whole within a warp's lanes, valid or not
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (valid) bf16x8_to_f32(__ldg(w + i), f);
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo = fminf(lo, f[j]);
    hi = fmaxf(hi, f[j]);
  }
#pragma unroll
  for (int o = G / 16; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float raw = kZeros ? __fdiv_rn(hi - lo, 15.f) : __fdiv_rn(fmaxf(hi, -lo), 7.f);
  const float s = fmaxf(__bfloat162float(__float2bfloat16_rn(raw)), FLT_MIN);
  int z = 8;
  if (kZeros) {
    z = __float2int_rn(__fdiv_rn(-lo, s));
    z = z < 0 ? 0 : (z > 15 ? 15 : z);
  }
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    int c = __float2int_rn(__fdiv_rn(f[j], s)) + z;
    c = c < 0 ? 0 : (c > 15 ? 15 : c);
    word |= static_cast<uint32_t>(c) << (4 * j);
  }
  if (!valid) return;
  q[i] = word;
  if (i % (G / 8) == 0) {
    scales[i / (G / 8)] = __float2bfloat16_rn(s);
    if (kZeros) zeros[i / (G / 8)] = static_cast<uint8_t>(z);
  }
}

// ----------------------------------------------------- product, few tokens
//
// mma.sync m16n8k16 with 16 weight rows on the M side and 8 tokens on the N
// side.  The order of k within a product is free as long as both operands
// agree, so a thread's fragment is simply G / 32 consecutive words of its row
// for each group (16 bytes when G = 128) and the activations of the same k.
// The codes minus their zero points are exact in bf16, a group's products are
// summed in fp32 by the tensor core, and the group's scale multiplies that sum
// in fp32: the only rounding to fewer bits is C's.
//
// Each CTA owns kRows = 16 RT weight rows and 8 MT tokens; its W warps take
// the 128-wide K blocks in turn and add their sums through shared memory in
// warp order.
//
// Bound by the issue and the latency of load, conversion and product in the
// few warps that the registers allow, then by the launch (about 3 us): one
// token [24576, 4096] 15.5 us, 0.51 of the copy rate (floor 7.9), 8 tokens
// 17.4 us; [4096, 4096] 4.7 and 6.0 us (floor 1.3).  Fewer registers beat
// loading ahead: with the next block's loads before this block's products the
// first took 21 us.  Rings filled by TMA or cp.async, persistent CTAs and
// activations in shared memory were all slower: the codes go from memory to
// the registers that need them, and a ring adds a trip through shared memory.
template <bool kZeroInit>
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  if constexpr (kZeroInit)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// W consecutive words of global memory, read once
template <int W>
__device__ __forceinline__ void ldg_words(const uint8_t* p, uint32_t* out) {
  if constexpr (W == 4)
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
                 : "l"(p));
  else if constexpr (W == 2)
    asm volatile("ld.global.nc.L2::256B.v2.b32 {%0, %1}, [%2];" : "=r"(out[0]), "=r"(out[1]) : "l"(p));
  else
    asm volatile("ld.global.nc.L2::256B.b32 %0, [%1];" : "=r"(out[0]) : "l"(p));
}

template <int G, int MT, int RT, int W, bool kZeros>
__global__ void __launch_bounds__(32 * W) int4_stream_kernel(const Int4Params p) {
  constexpr int kRows = 16 * RT, kTokens = 8 * MT;
  constexpr int GB = 128 / G;           // groups per block
  constexpr int WG = G / 32;            // words per thread, row and group
  __shared__ float red[W][kTokens][kRows + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  grid_launch_dependents();
  const int K = static_cast<int>(p.K), groups = K / G, blocks = (K + 127) / 128;
  const int M = static_cast<int>(p.M);
  const int tile = static_cast<int>(blockIdx.z * gridDim.y + blockIdx.y);   // of kTokens tokens
  int m0 = 0, m1 = 0;
  int64_t first_row = static_cast<int64_t>(blockIdx.x) * kRows;
  const int rows_left = static_cast<int>(p.N - first_row < kRows ? p.N - first_row : kRows);
  grid_dependency_wait();
  if (p.expert_offsets) {
    int expert;
    if (!find_expert_tile(p.expert_offsets, p.num_experts, M, kTokens, tile, &expert, &m0, &m1)) return;
    first_row += expert * p.N;
  } else {
    m0 = tile * kTokens;
    if (m0 >= M) return;
    m1 = m0 + kTokens < M ? m0 + kTokens : M;
  }
  const int toks_left = m1 - m0;

  // tile-uniform bases and 32-bit offsets (the host bounds K)
  const uint8_t* Bt = p.B + first_row * (K / 2);
  const __nv_bfloat16* St = p.scales + first_row * groups;
  const uint8_t* Zt = kZeros ? p.zeros + first_row * groups : nullptr;
  const __nv_bfloat16* Xt = p.x + static_cast<int64_t>(m0) * K;
  uint32_t row[RT][2];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = r * 16 + h * 8 + g;
      row[r][h] = n < rows_left ? n : rows_left - 1;    // rows past N repeat the last; not stored
    }

  float acc[RT][MT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][m][i] = 0.f;

#pragma unroll 1
  for (int kb = warp; kb < blocks; kb += W) {
    uint32_t word[RT][2][4];
    uint4 xv[MT][4];
    __nv_bfloat16 scale[RT][2][GB];
    uint8_t zero[RT][2][GB];
    // all of the block's loads first
#pragma unroll
    for (int gi = 0; gi < GB; ++gi) {
      const bool in = GB == 1 || kb * GB + gi < groups;   // only a K that is no multiple of 128 has a short block
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < WG; ++i) word[r][h][gi * WG + i] = 0u;
          if (in)
            ldg_words<WG>(Bt + row[r][h] * (K / 2) + (kb * 64 + gi * (G / 2) + t * (4 * WG)), &word[r][h][gi * WG]);
        }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int wd = 0; wd < WG; ++wd)
          xv[m][gi * WG + wd] =
              in && m * 8 + g < toks_left
                  ? __ldg(reinterpret_cast<const uint4*>(Xt + (m * 8 + g) * K + (kb * 128 + gi * G + (t * WG + wd) * 8)))
                  : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = row[r][h] * groups + kb * GB;
        if (GB > 1 && p.vec_scales) {
          if constexpr (GB == 4) {
            *reinterpret_cast<uint2*>(scale[r][h]) = __ldg(reinterpret_cast<const uint2*>(St + at));
            if (kZeros) *reinterpret_cast<uint32_t*>(zero[r][h]) = __ldg(reinterpret_cast<const uint32_t*>(Zt + at));
          } else if constexpr (GB == 2) {
            *reinterpret_cast<uint32_t*>(scale[r][h]) = __ldg(reinterpret_cast<const uint32_t*>(St + at));
            if (kZeros) *reinterpret_cast<uint16_t*>(zero[r][h]) = __ldg(reinterpret_cast<const uint16_t*>(Zt + at));
          }
        } else {
#pragma unroll
          for (int gi = 0; gi < GB; ++gi) {   // a group past K repeats the last: its activations are zero
            const uint32_t a = GB == 1 || kb * GB + gi < groups ? at + gi : row[r][h] * groups + groups - 1;
            scale[r][h][gi] = __ldg(St + a);
            if (kZeros) zero[r][h][gi] = __ldg(Zt + a);
          }
        }
      }
#pragma unroll
    for (int gi = 0; gi < GB; ++gi) {
      float part[RT][MT][4];
      uint32_t offset[RT][2];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) offset[r][h] = kZeros ? int4_offset(zero[r][h][gi]) : kInt4MidOffset;
#pragma unroll
      for (int wd = 0; wd < WG; ++wd)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) int4_word_to_bf16(word[r][h][gi * WG + wd], offset[r][h], a[h]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint4 v = xv[m][gi * WG + wd];
            if (wd == 0)
              mma_bf16_16816<true>(part[r][m], a[0][0], a[1][0], a[0][1], a[1][1], v.x, v.y);
            else
              mma_bf16_16816<false>(part[r][m], a[0][0], a[1][0], a[0][1], a[1][1], v.x, v.y);
            mma_bf16_16816<false>(part[r][m], a[0][2], a[1][2], a[0][3], a[1][3], v.z, v.w);
          }
        }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float s0 = __bfloat162float(scale[r][0][gi]), s1 = __bfloat162float(scale[r][1][gi]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[r][m][0] = fmaf(s0, part[r][m][0], acc[r][m][0]);
          acc[r][m][1] = fmaf(s0, part[r][m][1], acc[r][m][1]);
          acc[r][m][2] = fmaf(s1, part[r][m][2], acc[r][m][2]);
          acc[r][m][3] = fmaf(s1, part[r][m][3], acc[r][m][3]);
        }
      }
    }
  }

#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[warp][m * 8 + 2 * t + (i & 1)][r * 16 + (i >> 1) * 8 + g] = acc[r][m][i];
  __syncthreads();
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kRows;
  for (int o = threadIdx.x; o < kRows * toks_left; o += 32 * W) {
    const int tok = o / kRows, rr = o % kRows;
    if (rr >= rows_left) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += red[w][tok][rr];
    v *= kInt4Unit;
    if (p.bias) v += __bfloat162float(p.bias[n0 + rr]);
    p.C[static_cast<int64_t>(m0 + tok) * p.N + n0 + rr] = __float2bfloat16_rn(v);
  }
}

template <int G, int MT, int RT, int W>
cudaError_t launch_stream_gmr(const Int4Params& p, cudaStream_t stream) {
  constexpr int kTokens = 8 * MT, kRows = 16 * RT;
  const int64_t gx = (p.N + kRows - 1) / kRows;
  int64_t gy = (p.M + kTokens - 1) / kTokens;
  if (p.expert_offsets) gy += p.num_experts < p.M ? p.num_experts : p.M;
  const int64_t gz = (gy + 65534) / 65535;               // token tiles over y and z; those past the last one return
  gy = (gy + gz - 1) / gz;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy), static_cast<unsigned>(gz));
  cfg.blockDim = dim3(32 * W);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.zeros ? cudaLaunchKernelEx(&cfg, int4_stream_kernel<G, MT, RT, W, true>, p)
                 : cudaLaunchKernelEx(&cfg, int4_stream_kernel<G, MT, RT, W, false>, p);
}

// Dense (at most 8 tokens): 16-row tiles with 16 warps per tile until there are
// enough rows to fill the GPU with 32-row tiles of 8 warps.  Measured on B200,
// one token, G = 128: [4096, 4096] 4.7 us with 16 rows / 16 warps, 8.0 us with
// 32 / 8; [4096, 12288] 9.8 and 20.0; [24576, 4096] 18.9 and 15.5.  An SM holds
// two CTAs of 16 warps, so more than 296 row tiles take a second, partly filled
// round: [6144, 4096], 384 tiles, 7.8 us.  Grouped: the tiles of many experts
// are enough rows; two 8-token tiles per CTA where the experts have more than 8
// rows on average (more than 1024 experts: fewer take the tensor-core kernel).
template <int G>
cudaError_t launch_stream_g(const Int4Params& p, cudaStream_t stream) {
  if (!p.expert_offsets)
    return p.N >= 16384 ? launch_stream_gmr<G, 1, 2, 8>(p, stream) : launch_stream_gmr<G, 1, 1, 16>(p, stream);
  const int64_t per = (p.M + p.num_experts - 1) / p.num_experts;
  return per <= 8 ? launch_stream_gmr<G, 1, 2, 8>(p, stream) : launch_stream_gmr<G, 2, 2, 8>(p, stream);
}

template <int G>
cudaError_t launch_quant_g(const void* w, void* q, void* scales, void* zeros, int64_t N, int64_t K,
                           cudaStream_t stream) {
  const int64_t words = N * K / 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((words + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto* wp = static_cast<const uint4*>(w);
  auto* qp = static_cast<uint32_t*>(q);
  auto* sp = static_cast<__nv_bfloat16*>(scales);
  auto* zp = static_cast<uint8_t*>(zeros);
  return zeros ? cudaLaunchKernelEx(&cfg, quant_weight_int4_kernel<G, true>, wp, qp, sp, zp, words)
               : cudaLaunchKernelEx(&cfg, quant_weight_int4_kernel<G, false>, wp, qp, sp, zp, words);
}

}  // namespace

cudaError_t launch_int4_mm(const Int4Params& p, int group, cudaStream_t stream) {
  switch (group) {
    case 32: return launch_stream_g<32>(p, stream);
    case 64: return launch_stream_g<64>(p, stream);
    default: return launch_stream_g<128>(p, stream);
  }
}

cudaError_t launch_quant_weight_int4(const void* w, int group, void* q, void* scales, void* zeros, int64_t N,
                                     int64_t K, cudaStream_t stream) {
  switch (group) {
    case 32: return launch_quant_g<32>(w, q, scales, zeros, N, K, stream);
    case 64: return launch_quant_g<64>(w, q, scales, zeros, N, K, stream);
    default: return launch_quant_g<128>(w, q, scales, zeros, N, K, stream);
  }
}

}  // namespace lq
