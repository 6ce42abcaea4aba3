// Product with 4-bit weights on the tensor core, for more than a few tokens:
//
//   C^T tile [128 weight rows, NT tokens] = W (q - z) s . x^T
//
// tcgen05.mma kind::f16 with the weights as the operand in tensor memory: the
// packed codes are staged in shared memory by TMA (64 bytes per row and
// 128-wide K block), eight warps convert them to bf16 weights in registers,
// one row per lane, and store them straight into tensor memory, where a row
// is a lane and a column two k.  The converted weights never touch shared
// memory, whose bandwidth the activations need.
//
// Rounding: a weight (q - z) s is rounded once to bf16 (relative error at most
// 2^-8, like the activations' own rounding); everything after it is summed in
// fp32.  Scaling the sums of each group in fp32 instead would read the
// accumulator back once per group.  The weights are kept times 2^-40, so that
// without zero points one multiply-add does both the conversion and the scale
// (int4_common.cuh: the codes come as q 2^-133, and s 2^93 is a bf16 value for
// every |s| < 2^34); the epilogue multiplies by 2^40.
//
// Roles: warp 0 issues the TMA copies, warp 1 the MMAs, warps 2..9 convert and,
// at the end, read the accumulator.  The CTAs of a cluster along z share a
// tile's K and add their fp32 sums through distributed shared memory in rank
// order.  Every wait is bounded.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "int4_common.cuh"
#include "lq_kernels.h"
#include "ptx.cuh"

namespace lq {
namespace {

constexpr int kConvWarps = 8;           // two groups of four; group g converts blocks g, g + 2, ...
constexpr int kMmaThreads = 32 * (2 + kConvWarps);
constexpr int kMaxRing = 8, kMaxA = 4;
constexpr int kWeightTile = 128 * 64;   // bytes of a 128-row, 128-wide block of codes

template <int NT>
struct MmaShape {
  static constexpr int kTokenTile = NT * 256;                    // bytes of NT tokens x 128 k
  static constexpr int kStage = kWeightTile + kTokenTile;
  static constexpr bool kTwo = NT <= 64;                         // two CTAs per SM
  static constexpr int kRing = (kTwo ? 96 : 200) * 1024 / kStage < kMaxRing
                                   ? (NT == 256 ? 3 : (kTwo ? 96 : 200) * 1024 / kStage)
                                   : kMaxRing;
  static constexpr int kA = kTwo ? 3 : 4;                        // converted weight blocks in tensor memory
  static constexpr int kCols = kTwo ? 256 : 512;                 // tensor-memory columns
  static constexpr int kSmem = kRing * kStage + 1024;
};

// 40 is the exponent taken out of the weights and put back into the sums
constexpr float kSumScale = 1099511627776.f;   // 2^40

// bf16x2 factors {s 2^93, s 2^89} of the codes' two halves, q 2^-133 and 16 q 2^-133 (exact)
__device__ __forceinline__ uint32_t scale_factors(float s) {
  const __nv_bfloat162 f = __floats2bfloat162_rn(s * 0x1p93f, s * 0x1p89f);
  return *reinterpret_cast<const uint32_t*>(&f);
}
__device__ __forceinline__ uint32_t bf16x2_same(float v) {
  const __nv_bfloat162 f = __floats2bfloat162_rn(v, v);
  return *reinterpret_cast<const uint32_t*>(&f);
}

template <int G, int NT, bool kZeros>
__global__ void __launch_bounds__(kMmaThreads, MmaShape<NT>::kTwo ? 2 : 1)
    int4_mma_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const Int4Params p) {
  using Sh = MmaShape<NT>;
  constexpr int kRing = Sh::kRing, kA = Sh::kA;
  extern __shared__ uint8_t mma_smem_raw[];
  uint8_t* ring = mma_smem_raw + ((1024u - (smem_addr(mma_smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[kMaxRing], empty[kMaxRing], a_full[kMaxA], a_empty[kMaxA], done;
  __shared__ uint32_t tmem_base;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = static_cast<int>(gridDim.z), rank = static_cast<int>(blockIdx.z);
  const int K = static_cast<int>(p.K), groups = K / G, all_blocks = (K + 127) / 128;
  const int M = static_cast<int>(p.M);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 128;

  grid_launch_dependents();
  const bool early = p.early_weights && !p.expert_offsets;
  int m0 = static_cast<int>(blockIdx.y) * NT, m1 = m0 + NT < M ? m0 + NT : M, expert = 0;
  if (p.expert_offsets) {
    grid_dependency_wait();
    if (!find_expert_tile(p.expert_offsets, p.num_experts, M, NT, blockIdx.y, &expert, &m0, &m1)) return;
  }
  const int64_t first_row = expert * p.N + n0;
  const int kb_lo = static_cast<int>(static_cast<int64_t>(all_blocks) * rank / split);
  const int blocks = static_cast<int>(static_cast<int64_t>(all_blocks) * (rank + 1) / split) - kb_lo;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4 + 1);
    }
    for (int b = 0; b < kA; ++b) {
      mbar_init(&a_full[b], 4);
      mbar_init(&a_empty[b], 1);
    }
    mbar_init(&done, 1);
    fence_barrier_init();
    prefetch_tensor_map(&tmW);
    prefetch_tensor_map(&tmX);
  }
  if (warp == 1) tmem_alloc(&tmem_base, Sh::kCols);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tm_a = tmem_base;        // kA converted blocks of 64 columns,
  const uint32_t tm = tm_a + kA * 64;     // then the accumulator
  auto give_up = [&](int site) {
    if (p.status) atomicOr(p.status, 1 << site);
  };

  // Warps 0 and 1 walk the blocks as whole warps, so that addresses and
  // descriptors stay in uniform registers, and one elected lane issues.  (From
  // a one-lane branch a block's three copies took 550 cycles and its eight MMAs
  // 570, several times their own time at few tokens, and bounded every shape.)
  if (warp == 0) {
    const bool leader = elect_one();
    const uint64_t keep = policy_evict_last(), weight_policy = p.M > NT ? keep : policy_evict_first();
    const int w_row = static_cast<int>(first_row);
    auto load_weights = [&](int i, int s) {
      mbar_arrive_expect_tx(&full[s], Sh::kStage);
      tma_load_2d(&tmW, &full[s], ring + s * Sh::kStage, (kb_lo + i) * 64, w_row, weight_policy);
    };
    auto load_tokens = [&](int i, int s) {
      uint8_t* x = ring + s * Sh::kStage + kWeightTile;
      tma_load_2d(&tmX, &full[s], x, (kb_lo + i) * 128, m0, keep);
      tma_load_2d(&tmX, &full[s], x + NT * 128, (kb_lo + i) * 128 + 64, m0, keep);
    };
    if (early && leader)
      for (int i = 0; i < blocks && i < kRing; ++i)
        if (kb_lo + i != p.skip_block) load_weights(i, i);
    __syncwarp();
    grid_dependency_wait();
    bool fed = true;
    int issued = 0, s = 0;
    uint32_t phase = 1;                    // the first kRing blocks find their slot free
    for (; issued < blocks; ++issued) {
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], phase, p.wait_limit_ns))) {
        if (leader) give_up(9);
        fed = false;
        break;
      }
      if (leader && kb_lo + issued != p.skip_block) {   // test hook: a block that never arrives
        if (!early || issued >= kRing) load_weights(issued, s);
        load_tokens(issued, s);
      }
      __syncwarp();
      if (++s == kRing) {
        s = 0;
        phase ^= 1;
      }
    }
    if (leader && (!fed || p.skip_block >= 0))   // copies still under way land before the memory is given back
      for (int i = issued > kRing ? issued - kRing : 0; i < issued; ++i)
        if (kb_lo + i != p.skip_block) mbar_wait(&full[i % kRing], (i / kRing) & 1, p.wait_limit_ns);
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idesc = make_idesc_bf16(128, NT);
    const uint64_t desc0 = smem_desc_k_sw128(ring + kWeightTile);
    const bool leader = elect_one();
    int s = 0, b = 0;
    uint32_t b_phase = 0;
    for (int i = 0; i < blocks; ++i) {
      // the converting warps waited for the block's copies, activations included, before they arrived here
      if (!__all_sync(0xffffffffu, mbar_wait(&a_full[b], b_phase, p.wait_limit_ns))) {
        if (leader) give_up(10);
        break;
      }
      tc_fence_after_sync();
      const uint64_t desc = desc0 + static_cast<uint32_t>(s * (Sh::kStage >> 4));
      const uint32_t a = tm_a + b * 64;
      if (leader) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          mma_f16_a_tmem(tm, a + j * 8, desc + (j >> 2) * (NT * 128 >> 4) + (j & 3) * 2, idesc, i > 0 || j > 0);
        mma_commit(&a_empty[b]);
        mma_commit(&empty[s]);
      }
      __syncwarp();
      s = s + 1 == kRing ? 0 : s + 1;
      if (++b == kA) {
        b = 0;
        b_phase ^= 1;
      }
    }
    if (leader) mma_commit(&done);
  }
  __syncwarp();
  grid_dependency_wait();
  bool ok = true;
  const int quad = warp & 3, half = (warp - 2) >> 2;   // of a converting warp: its 32 rows, its group
  if (warp >= 2) {
    const int row = quad * 32 + lane;
    const int64_t left = p.N - n0;
    const int64_t wrow = first_row + (row < left ? row : left - 1);   // rows past N repeat the last; not stored
    const __nv_bfloat16* sr = p.scales + wrow * groups;
    const uint8_t* zr = kZeros ? p.zeros + wrow * groups : nullptr;
    constexpr int GB = 128 / G;           // groups in a block
    __nv_bfloat16 s_next[GB];
    uint8_t z_next[GB];
    auto load_scales = [&](int i) {
      int at = (kb_lo + i) * GB;
#pragma unroll
      for (int j = 0; j < GB; ++j) {
        const int a = GB == 1 || at + j < groups ? at + j : groups - 1;   // past K: the activations are zero
        s_next[j] = __ldg(sr + a);
        if (kZeros) z_next[j] = __ldg(zr + a);
      }
    };
    if (half < blocks) load_scales(half);
    int s = half, b = half;               // ring slot and converted-block slot of block i
    uint32_t s_phase = 0, b_phase = 1;    // b: the first kA blocks find their slot free
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t swizzle = (row >> 1) & 3;
    for (int i = half; i < blocks; i += 2) {
      uint32_t factor[GB], offset[GB];
#pragma unroll
      for (int j = 0; j < GB; ++j) {
        const float sf = __bfloat162float(s_next[j]);
        if constexpr (kZeros) {
          factor[j] = bf16x2_same(sf * 0x1p-34f);      // of (q - z) / 64
          offset[j] = int4_offset(z_next[j]);
        } else {
          factor[j] = scale_factors(sf);
          offset[j] = bf16x2_same(sf * -0x1p-37f);     // -8 s 2^-40
        }
      }
      if (i + 2 < blocks) load_scales(i + 2);
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], s_phase, p.wait_limit_ns))) {   // the warp stays together
        ok = false;
        break;
      }
      uint32_t w[16];
      const uint32_t at = smem_addr(ring + s * Sh::kStage) + row * 64;
#pragma unroll
      for (int c = 0; c < 4; ++c)          // 16-byte pieces, exchanged by (row / 2) mod 4 (the 64-byte swizzle)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * c]), "=r"(w[4 * c + 1]), "=r"(w[4 * c + 2]), "=r"(w[4 * c + 3])
                     : "r"(at + ((c ^ swizzle) << 4)));
      if (!__all_sync(0xffffffffu, mbar_wait(&a_empty[b], b_phase, p.wait_limit_ns))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t a[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int gj = (q * 8 + j) * GB / 16;
          const uint32_t word = w[q * 8 + j], lo = word & 0x0F0F0F0Fu, hi = word & 0xF0F0F0F0u;
          const uint32_t mul = kZeros ? kInt4Factors : factor[gj];
          a[4 * j] = bf16x2_fma(byte_select(lo, hi, 0x8480), mul, offset[gj]);
          a[4 * j + 1] = bf16x2_fma(byte_select(lo, hi, 0x8581), mul, offset[gj]);
          a[4 * j + 2] = bf16x2_fma(byte_select(lo, hi, 0x8682), mul, offset[gj]);
          a[4 * j + 3] = bf16x2_fma(byte_select(lo, hi, 0x8783), mul, offset[gj]);
          if constexpr (kZeros)            // (q - z) / 64 is exact; one rounding here
#pragma unroll
            for (int e = 0; e < 4; ++e) a[4 * j + e] = bf16x2_fma(a[4 * j + e], factor[gj], 0x80008000u);
        }
        tmem_st_32x32b_x32(tm_a + b * 64 + q * 32 + lanes, a);
      }
      if (lane == 0) mbar_arrive(&empty[s]);   // the codes are in registers (every lane has converted them)
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&a_full[b]);
      s += 2;
      if (s >= kRing) {
        s -= kRing;
        s_phase ^= 1;
      }
      b += 2;
      if (b >= kA) {
        b -= kA;
        b_phase ^= 1;
      }
    }
    ok = ok && mbar_wait(&done, 0, p.wait_limit_ns);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) give_up(11);
    tc_fence_after_sync();
  }

  // ---- epilogue: lanes are weight rows, columns tokens; through shared memory (the ring is free:
  // every copy into it has been waited for) to rows of C
  const int toks_left = m1 - m0;
  constexpr int kChunk = NT >= 64 ? 32 : NT / 2;
  auto columns = [&](auto&& put) {
#pragma unroll 1
    for (int c = half * (NT / 2); c < (half + 1) * (NT / 2); c += kChunk) {
      uint32_t r[kChunk];
      const uint32_t at = tm + c + (static_cast<uint32_t>(quad * 32) << 16);
      if constexpr (kChunk == 32) tmem_ld_32x32b_x32(at, r);
      else if constexpr (kChunk == 16) tmem_ld_32x32b_x16(at, r);
      else tmem_ld_32x32b_x8(at, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < kChunk; ++j) put(c + j, __uint_as_float(r[j]) * kSumScale);
    }
  };
  if (split == 1) {
    if (warp >= 2) {
      const int n = quad * 32 + lane;
      const float bias = p.bias && n0 + n < p.N ? __bfloat162float(p.bias[n0 + n]) : 0.f;
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(ring);     // [NT][128]
      if (ok && blocks > 0) columns([&](int tok, float v) { out[tok * 128 + n] = __float2bfloat16_rn(v + bias); });
      named_barrier_sync(1, 32 * kConvWarps);
      for (int i = threadIdx.x - 64; i < toks_left * 16; i += 32 * kConvWarps) {
        const int tok = i >> 4, c = (i & 15) * 8;
        if (n0 + c < p.N)
          *reinterpret_cast<uint4*>(p.C + static_cast<int64_t>(m0 + tok) * p.N + n0 + c) =
              *reinterpret_cast<const uint4*>(out + tok * 128 + c);
      }
    }
  } else {
    float* part = reinterpret_cast<float*>(ring);                        // [NT][128]
    if (warp >= 2) {
      const int n = quad * 32 + lane;
      if (blocks > 0) {
        if (ok) columns([&](int tok, float v) { part[tok * 128 + n] = v; });
      } else {
        for (int tok = half * (NT / 2); tok < (half + 1) * (NT / 2); ++tok) part[tok * 128 + n] = 0.f;
      }
    }
    cluster_sync_all();
    for (int i = threadIdx.x; ; i += kMmaThreads) {
      const int tok = (i >> 4) * split + rank, c = (i & 15) * 8;
      if (tok >= toks_left) break;
      if (n0 + c >= p.N) continue;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      const uint32_t at = smem_addr(part + tok * 128 + c);
      for (int r = 0; r < split; ++r) {
        const uint32_t from = dsmem_map(at, r);
        const float4 a = dsmem_ld_f32x4(from), b = dsmem_ld_f32x4(from + 16);
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
      }
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (p.bias) {
          v[2 * j] += __bfloat162float(p.bias[n0 + c + 2 * j]);
          v[2 * j + 1] += __bfloat162float(p.bias[n0 + c + 2 * j + 1]);
        }
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p.C + static_cast<int64_t>(m0 + tok) * p.N + n0 + c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    cluster_sync_all();                   // nobody reads this CTA's sums any more
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_relinquish();
    tmem_dealloc(tm_a, Sh::kCols);
  }
}

template <int G, int NT>
cudaError_t launch_mma_gn(const Int4Params& p, int split, cudaStream_t stream) {
  using Sh = MmaShape<NT>;
  const int64_t gx = (p.N + 127) / 128;
  int64_t gy = (p.M + NT - 1) / NT;
  if (p.expert_offsets) gy += p.num_experts < p.M ? p.num_experts : p.M;
  if (gy > 65535) return cudaErrorInvalidValue;
  CUtensorMap tmW, tmX;
  const int64_t rows = p.N * (p.expert_offsets ? p.num_experts : 1);
  if (!encode_tma_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.B, p.K / 2, rows, p.K / 2, 64, 128,
                     CU_TENSOR_MAP_SWIZZLE_64B) ||
      !encode_tma_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.x, p.K, p.M, p.K * 2, 64, NT,
                     CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto kernel = p.zeros ? int4_mma_kernel<G, NT, true> : int4_mma_kernel<G, NT, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy), static_cast<unsigned>(split));
  cfg.blockDim = dim3(kMmaThreads);
  cfg.dynamicSmemBytes = Sh::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = static_cast<unsigned>(split);
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, p);
}

template <int G>
cudaError_t launch_mma_g(const Int4Params& p, int tile, int split, cudaStream_t stream) {
  switch (tile) {
    case 16: return launch_mma_gn<G, 16>(p, split, stream);
    case 32: return launch_mma_gn<G, 32>(p, split, stream);
    case 64: return launch_mma_gn<G, 64>(p, split, stream);
    case 128: return launch_mma_gn<G, 128>(p, split, stream);
    default: return launch_mma_gn<G, 256>(p, split, stream);
  }
}

}  // namespace

cudaError_t launch_int4_mma(const Int4Params& p, int group, int tile, int split, cudaStream_t stream) {
  switch (group) {
    case 32: return launch_mma_g<32>(p, tile, split, stream);
    case 64: return launch_mma_g<64>(p, tile, split, stream);
    default: return launch_mma_g<128>(p, tile, split, stream);
  }
}

}  // namespace lq
