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
// side; the weights go from global memory to the tensor core through
// registers only.  The order of k within a product is free as long as both
// operands agree, so a thread's fragment is simply what it loads: G / 32
// consecutive words of its row for each group (16 bytes when G = 128), and
// the 8 activations of a word as the pairs (0, 4), (1, 5), (2, 6), (3, 7) in
// which int4_word_to_bf16 leaves the codes.  The codes minus their zero
// points are exact in bf16, a group's products are summed in fp32 by the
// tensor core, and the group's scale multiplies that sum in fp32: the only
// rounding to fewer bits is C's.
//
// Each CTA owns kRows = 16 RT weight rows and 8 MT tokens; its 8 warps take
// the 128-wide K blocks in turn and add their sums through shared memory in
// warp order.
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t ldg_stream_u32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.L1::no_allocate.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg_stream_u64(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ldg_stream_u128(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// W consecutive words from p (4 W-byte aligned)
template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* out) {
  if constexpr (W == 4) {
    const uint4 v = ldg_stream_u128(p);
    out[0] = v.x; out[1] = v.y; out[2] = v.z; out[3] = v.w;
  } else if constexpr (W == 2) {
    const uint2 v = ldg_stream_u64(p);
    out[0] = v.x; out[1] = v.y;
  } else {
    out[0] = ldg_stream_u32(p);
  }
}

// What a warp needs of one 128-wide K block of its rows.
template <int G, int RT>
struct WeightBlock {
  uint32_t word[RT][2][4];              // [16-row tile][row half][word]
  __nv_bfloat16 scale[RT][2][128 / G];
  uint8_t zero[RT][2][128 / G];
};

// The expert that owns token tile `tile` when every expert's rows are cut
// into tiles of `per` tokens: its rows [*lo, *hi) of the tile.  Offsets are
// clamped to [0, T] and to their running maximum, so a malformed table never
// leads outside the rows.  Called by whole warps; false: no such tile.
__device__ __forceinline__ bool find_expert_tile(const int* __restrict__ offsets, int E, int64_t T, int per,
                                                 int64_t tile, int* expert, int64_t* lo, int64_t* hi) {
  const int lane = threadIdx.x & 31;
  int64_t tiles_before = 0;
  int carry = 0;                        // running maximum so far
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    int end = e < E ? __ldg(offsets + e + 1) : 0;
    int first = lane == 0 && e0 == 0 ? __ldg(offsets) : 0;
    end = end < 0 ? 0 : (end > T ? static_cast<int>(T) : end);
    first = first < 0 ? 0 : (first > T ? static_cast<int>(T) : first);
    if (e0 == 0) carry = __shfl_sync(0xffffffffu, first, 0);
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
    const int64_t mine = tiles_before + upto - tiles;   // first tile of this lane's expert
    const uint32_t has = __ballot_sync(0xffffffffu, tile >= mine && tile < mine + tiles);
    if (has) {
      const int src = __ffs(has) - 1;
      const int64_t b = __shfl_sync(0xffffffffu, begin, src);
      const int64_t en = __shfl_sync(0xffffffffu, end, src);
      const int64_t idx = tile - __shfl_sync(0xffffffffu, mine, src);
      *expert = e0 + src;
      *lo = b + idx * per;
      *hi = *lo + per < en ? *lo + per : en;
      return true;
    }
    tiles_before += __shfl_sync(0xffffffffu, upto, 31);
    carry = __shfl_sync(0xffffffffu, end, 31);
  }
  return false;
}

template <int G, int MT, int RT, bool kZeros>
__global__ void __launch_bounds__(kThreads) int4_stream_kernel(Int4Params p) {
  constexpr int kRows = 16 * RT, kTokens = 8 * MT;
  constexpr int GB = 128 / G;           // groups per block
  constexpr int WG = G / 32;            // words per thread, row and group
  __shared__ float red[kWarps][kTokens][kRows + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  grid_launch_dependents();
  grid_dependency_wait();
  int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTokens, m1 = p.M;
  int expert = 0;
  if (p.expert_offsets &&
      !find_expert_tile(p.expert_offsets, p.num_experts, p.M, kTokens, blockIdx.y, &expert, &m0, &m1))
    return;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kRows;
  const int64_t row_base = static_cast<int64_t>(expert) * p.N;
  const int64_t groups = p.K / G;
  const int blocks = static_cast<int>((p.K + 127) / 128);

  int64_t row[RT][2];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = n0 + r * 16 + h * 8 + g;
      row[r][h] = row_base + (n < p.N ? n : p.N - 1);   // rows past N repeat the last; not stored
    }
  auto load_block = [&](WeightBlock<G, RT>& b, int kb) {
#pragma unroll
    for (int gi = 0; gi < GB; ++gi) {
      const int64_t grp = static_cast<int64_t>(kb) * GB + gi;
      const bool in = grp < groups;     // only the last block of a K that is no multiple of 128 is short
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t at = row[r][h] * groups + grp;
          if (in) {
            load_words<WG>(p.B + at * (G / 2) + t * (4 * WG), &b.word[r][h][gi * WG]);
            b.scale[r][h][gi] = p.scales[at];
            if (kZeros) b.zero[r][h][gi] = p.zeros[at];
          } else {
#pragma unroll
            for (int i = 0; i < WG; ++i) b.word[r][h][gi * WG + i] = 0x88888888u;
            b.scale[r][h][gi] = __float2bfloat16_rn(0.f);
            if (kZeros) b.zero[r][h][gi] = 8;
          }
        }
    }
  };

  float acc[RT][MT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][m][i] = 0.f;

  auto compute = [&](const WeightBlock<G, RT>& b, int kb) {
#pragma unroll
    for (int gi = 0; gi < GB; ++gi) {
      const int64_t grp = static_cast<int64_t>(kb) * GB + gi;
      float part[RT][MT][4];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) part[r][m][i] = 0.f;
#pragma unroll
      for (int wd = 0; wd < WG; ++wd) {
        uint4 xv[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int64_t tok = m0 + m * 8 + g;
          xv[m] = tok < m1 && grp < groups
                      ? __ldg(reinterpret_cast<const uint4*>(p.x + tok * p.K + grp * G + (t * WG + wd) * 8))
                      : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            int4_word_to_bf16(b.word[r][h][gi * WG + wd], kZeros ? int4_offset(b.zero[r][h][gi]) : kInt4MidOffset,
                              a[h]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            mma_bf16_16816(part[r][m], a[0][0], a[1][0], a[0][1], a[1][1], __byte_perm(xv[m].x, xv[m].z, 0x5410),
                           __byte_perm(xv[m].x, xv[m].z, 0x7632));
            mma_bf16_16816(part[r][m], a[0][2], a[1][2], a[0][3], a[1][3], __byte_perm(xv[m].y, xv[m].w, 0x5410),
                           __byte_perm(xv[m].y, xv[m].w, 0x7632));
          }
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float s0 = __bfloat162float(b.scale[r][0][gi]), s1 = __bfloat162float(b.scale[r][1][gi]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[r][m][0] = fmaf(s0, part[r][m][0], acc[r][m][0]);
          acc[r][m][1] = fmaf(s0, part[r][m][1], acc[r][m][1]);
          acc[r][m][2] = fmaf(s1, part[r][m][2], acc[r][m][2]);
          acc[r][m][3] = fmaf(s1, part[r][m][3], acc[r][m][3]);
        }
      }
    }
  };

  WeightBlock<G, RT> cur, nxt;
  if (warp < blocks) load_block(cur, warp);
  for (int kb = warp; kb < blocks; kb += kWarps) {
    if (kb + kWarps < blocks) load_block(nxt, kb + kWarps);
    compute(cur, kb);
    cur = nxt;
  }

#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[warp][m * 8 + 2 * t + (i & 1)][r * 16 + (i >> 1) * 8 + g] = acc[r][m][i];
  __syncthreads();
  for (int o = threadIdx.x; o < kRows * kTokens; o += kThreads) {
    const int tok = o / kRows, rr = o % kRows;
    const int64_t m = m0 + tok, n = n0 + rr;
    if (m >= m1 || n >= p.N) continue;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += red[w][tok][rr];
    if (p.bias) s += __bfloat162float(p.bias[n]);
    p.C[m * p.N + n] = __float2bfloat16_rn(s);
  }
}

template <int G, int MT, int RT>
cudaError_t launch_stream_gmr(const Int4Params& p, cudaStream_t stream) {
  constexpr int kTokens = 8 * MT;
  const int64_t gx = (p.N + 16 * RT - 1) / (16 * RT);
  int64_t gy = (p.M + kTokens - 1) / kTokens;
  if (p.expert_offsets) gy += p.num_experts < p.M ? p.num_experts : p.M;
  if (gy > 65535) return cudaErrorInvalidValue;   // the host checks this first
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.zeros ? cudaLaunchKernelEx(&cfg, int4_stream_kernel<G, MT, RT, true>, p)
                 : cudaLaunchKernelEx(&cfg, int4_stream_kernel<G, MT, RT, false>, p);
}

template <int G>
cudaError_t launch_stream_g(const Int4Params& p, cudaStream_t stream) {
  return p.M <= 8 ? launch_stream_gmr<G, 1, 1>(p, stream) : launch_stream_gmr<G, 2, 2>(p, stream);
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
