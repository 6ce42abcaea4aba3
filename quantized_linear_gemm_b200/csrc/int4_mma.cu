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
// Roles: warp 0 issues the TMA copies, warp 1 the MMAs, warps 2..9 convert; the
// epilogue has its own warps or is theirs too.  Every role walks the CTA's
// tiles and their K blocks on its own, the rings run on across tiles.  With
// Split-K the CTAs of a cluster share a tile's K and add their fp32 sums
// through distributed shared memory in rank order.  Every wait is bounded.
//
// What bounds it.  Few tokens: in steady state an SM takes a 128 x 128 block of
// weights every 400 cycles, with one CTA as with two, where HBM alone needs
// 370; what remains is the launch, the first block's way through the roles and
// the last, partly filled round of tiles.  [37888, 4096], 16 tokens: 20.5 us,
// 4.0 TB/s, 0.61 of the copy rate; [5120, 25600], 37 tokens: 25.3 us, 0.42 (six
// CTAs share a tile's K: 240 on 148 SMs, so the SMs with two of them set the
// time).  Many tokens: the tensor core, and the converting warps that compete
// with it for power and issue slots: [24576, 4096], 2048 tokens, 321 to 335 us
// call after call, 1.23 to 1.29 PFLOP/s, 0.73 to 0.76 of the burst rate of a bf16
// library product (0.89 of the sustained one); 286 us in a short burst.  Several accumulators per
// tile, or one MMA per block instead of eight, change nothing at few tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "int4_common.cuh"
#include "int4_mma_shape.h"
#include "lq_kernels.h"
#include "ptx.cuh"

namespace lq {
namespace {

constexpr int kMaxGroupedExperts = 1024;

constexpr float kSumScale = 1099511627776.f;   // 2^40: taken out of the weights, put back into the sums

// bf16x2 factors {s 2^93, s 2^89} of the codes' two halves, q 2^-133 and 16 q 2^-133 (exact)
__device__ __forceinline__ uint32_t scale_factors(float s) {
  const __nv_bfloat162 f = __floats2bfloat162_rn(s * 0x1p93f, s * 0x1p89f);
  return *reinterpret_cast<const uint32_t*>(&f);
}
__device__ __forceinline__ uint32_t bf16x2_same(float v) {
  const __nv_bfloat162 f = __floats2bfloat162_rn(v, v);
  return *reinterpret_cast<const uint32_t*>(&f);
}

// One output tile: 128 weight rows of an expert and the tokens [m0, m1).
struct Tile {
  int expert, n_tile, m0, m1;
};

template <int G, int NT, bool kZeros>
__global__ void __launch_bounds__(MmaShape<NT>::kThreads, MmaShape<NT>::kTwo ? 2 : 1)
    int4_mma_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const Int4Params p) {
  using Sh = MmaShape<NT>;
  constexpr int kRing = Sh::kRing, kA = Sh::kA, kD = Sh::kD, kGroups = Sh::kGroups;
  extern __shared__ uint8_t mma_smem_raw[];
  uint8_t* ring = mma_smem_raw + ((1024u - (smem_addr(mma_smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[kMaxRing], empty[kMaxRing], a_full[kMaxA], a_empty[kMaxA], d_full[2], d_empty[2];
  __shared__ uint32_t tmem_base;
  __shared__ int end_row[kMaxGroupedExperts + 1], first_tile[kMaxGroupedExperts + 1];   // grouped
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = p.split, rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int K = static_cast<int>(p.K), groups = K / G, all_blocks = (K + 127) / 128;
  const int M = static_cast<int>(p.M), ntiles = static_cast<int>((p.N + 127) / 128);
  const int worker = static_cast<int>(blockIdx.x) / split, workers = static_cast<int>(gridDim.x) / split;
  const int kb_lo = static_cast<int>(static_cast<int64_t>(all_blocks) * rank / split);
  const int blocks = static_cast<int>(static_cast<int64_t>(all_blocks) * (rank + 1) / split) - kb_lo;
  const bool grouped = p.expert_offsets != nullptr;
  const bool early = p.early_weights && !grouped;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4 + 1);
    }
    for (int b = 0; b < kA; ++b) {
      mbar_init(&a_full[b], 4);
      mbar_init(&a_empty[b], 1);
    }
    for (int d = 0; d < kD; ++d) {
      mbar_init(&d_full[d], 1);
      mbar_init(&d_empty[d], 8);
    }
    fence_barrier_init();
    prefetch_tensor_map(&tmW);
    prefetch_tensor_map(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base, Sh::kCols);
    tmem_relinquish();                    // until then the SM's other CTA cannot allocate
  }
  int token_tiles = (M + NT - 1) / NT;
  if (grouped) {
    // end_row[e] = last row of the experts before e (offsets clamped to [0, T] and to their running
    // maximum), first_tile[e] = token tiles of the experts before e
    grid_dependency_wait();
    const int E = p.num_experts;
    for (int e = threadIdx.x; e <= E; e += Sh::kThreads) {
      const int o = __ldg(p.expert_offsets + e);
      end_row[e] = o < 0 ? 0 : (o > M ? M : o);
    }
    __syncthreads();
    if (warp == 0) {
      int top = 0, tiles = 0;
      for (int e0 = 0; e0 <= E; e0 += 32) {
        const int e = e0 + lane;
        int v = e <= E ? end_row[e] : 0;
        v = v > top ? v : top;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o && u > v) v = u;
        }
        int before = __shfl_up_sync(0xffffffffu, v, 1);
        if (lane == 0) before = e0 ? top : v;
        int c = (v - before + NT - 1) / NT;      // of expert e - 1
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, c, o);
          if (lane >= o) c += u;
        }
        if (e <= E) {
          end_row[e] = v;
          first_tile[e] = tiles + c;
        }
        top = __shfl_sync(0xffffffffu, v, 31);
        tiles += __shfl_sync(0xffffffffu, c, 31);
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (grouped) token_tiles = first_tile[p.num_experts];
  const int tiles = token_tiles * ntiles;        // numbered token tile by token tile
  const int mine = tiles > worker ? (tiles - worker + workers - 1) / workers : 0;   // worker, worker + workers, ...
  auto tile_at = [&](int k) {
    const int t = worker + k * workers, y = t / ntiles;
    Tile r{0, t - y * ntiles, y * NT, 0};
    if (grouped) {
      int lo = 0, hi = p.num_experts;            // the expert with first_tile[e] <= y < first_tile[e + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first_tile[mid] <= y) lo = mid;
        else hi = mid;
      }
      r.expert = lo;
      r.m0 = end_row[lo] + (y - first_tile[lo]) * NT;
      r.m1 = r.m0 + NT < end_row[lo + 1] ? r.m0 + NT : end_row[lo + 1];
    } else {
      r.m1 = r.m0 + NT < M ? r.m0 + NT : M;
    }
    return r;
  };
  const uint32_t tm_a = tmem_base;        // kA converted blocks of 64 columns,
  const uint32_t tm_d = tm_a + kA * 64;   // then the accumulators
  auto give_up = [&](int site) {
    if (p.status) atomicOr(p.status, 1 << site);
  };
  bool ok = true;

  // The issuing warps walk the blocks as whole warps, so that addresses and
  // descriptors stay in uniform registers, and one elected lane issues.  (From
  // a one-lane branch a block's three copies took 550 cycles and its eight MMAs
  // 570, several times their own time at few tokens, and bounded every shape.)
  const uint64_t keep = policy_evict_last(), weight_policy = M > NT ? keep : policy_evict_first();
  const bool leader = elect_one();
  const int ahead = blocks < kRing ? blocks : kRing;   // of the first tile, before the dependency wait
  auto load_weights = [&](int w_row, int i, int s) {
    mbar_arrive_expect_tx(&full[s], Sh::kStage);
    tma_load_2d(&tmW, &full[s], ring + s * Sh::kStage, (kb_lo + i) * 64, w_row, weight_policy);
  };
  if (early && warp == 0 && leader && mine > 0)
    for (int i = 0; i < ahead; ++i)
      if (kb_lo + i != p.skip_block) load_weights(tile_at(0).n_tile * 128, i, i);
  __syncwarp();
  grid_dependency_wait();                 // every role: polling would take issue slots from the launch before
  // Only now: were the next launch let in earlier, the one after it would take
  // this one's places before this one has run, and CTAs pair up unevenly
  // ([4096, 4096] at 16 tokens, split 4: 8.8 us instead of 7.3).
  grid_launch_dependents();
  if (warp == 0) {
    auto load_tokens = [&](int m0, int i, int s) {
      uint8_t* x = ring + s * Sh::kStage + kWeightTile;
      tma_load_2d(&tmX, &full[s], x, (kb_lo + i) * 128, m0, keep);
      tma_load_2d(&tmX, &full[s], x + NT * 128, (kb_lo + i) * 128 + 64, m0, keep);
    };
    int s = 0, issued = 0;
    uint32_t phase = 1;                    // the first kRing blocks find their slot free
    for (int k = 0; k < mine && ok; ++k) {
      const Tile t = tile_at(k);
      const int w_row = static_cast<int>(t.expert * p.N + t.n_tile * 128);
      for (int i = 0; i < blocks; ++i) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], phase, p.wait_limit_ns))) {
          if (leader) give_up(9);
          ok = false;
          break;
        }
        if (leader && kb_lo + i != p.skip_block) {   // test hook: a block that never arrives
          if (!early || issued >= ahead) load_weights(w_row, i, s);
          load_tokens(t.m0, i, s);
        }
        __syncwarp();
        ++issued;
        if (++s == kRing) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    if (leader && (!ok || p.skip_block >= 0))   // copies still under way land before the memory is given back
      for (int j = issued > kRing ? issued - kRing : 0; j < issued; ++j)
        if (kb_lo + j % blocks != p.skip_block) mbar_wait(&full[j % kRing], (j / kRing) & 1, p.wait_limit_ns);
    __syncwarp();
  } else if (warp == 1) {
    const uint64_t desc0 = smem_desc_k_sw128(ring + kWeightTile);
    int s = 0, b = 0, d = 0;
    uint32_t b_phase = 0, d_phase = 1;     // the first kD tiles find their accumulator free
    for (int k = 0; k < mine && ok; ++k) {
      const Tile t = tile_at(k);
      const uint32_t idesc = make_idesc_bf16(128, (t.m1 - t.m0 + 15) & ~15);   // only the tile's tokens
      if (!__all_sync(0xffffffffu, mbar_wait(&d_empty[d], d_phase, p.wait_limit_ns))) {
        if (leader) give_up(10);
        ok = false;
        break;
      }
      const uint32_t acc = tm_d + d * NT;
      for (int i = 0; i < blocks; ++i) {
        // the converting warps waited for the block's copies, activations included, before they arrived here
        if (!__all_sync(0xffffffffu, mbar_wait(&a_full[b], b_phase, p.wait_limit_ns))) {
          if (leader) give_up(10);
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint64_t desc = desc0 + static_cast<uint32_t>(s * (Sh::kStage >> 4));
        const uint32_t a = tm_a + b * 64;
        if (leader) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mma_f16_a_tmem(acc, a + j * 8, desc + (j >> 2) * (NT * 128 >> 4) + (j & 3) * 2, idesc, i > 0 || j > 0);
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
      if (leader) mma_commit(&d_full[d]);
      if (++d == kD) {
        d = 0;
        d_phase ^= 1;
      }
    }
  }
  __syncwarp();
  const int quad = warp & 3;              // the 32 tensor-memory lanes (weight rows) of a converting or epilogue warp

  // ---- epilogue of tile k (eight warps: four quadrants, two halves of the columns): lanes are weight
  // rows, columns tokens.  The sums are read, rounded and packed first, so that the accumulator is free
  // for the next tile before the stores; a store writes 32 neighbouring channels of one token, whole sectors.
  auto epilogue = [&](int k, int d, uint32_t d_phase) {
    const int part = (warp - Sh::kEpiFirst) >> 2;
    if (!__all_sync(0xffffffffu, mbar_wait(&d_full[d], d_phase, p.wait_limit_ns))) {
      if (lane == 0) give_up(11);
      ok = false;
      return;
    }
    tc_fence_after_sync();
    const Tile t = tile_at(k);
    const int toks = t.m1 - t.m0;
    constexpr int kCols = NT / 2, kChunk = kCols % 32 == 0 ? 32 : (kCols % 16 == 0 ? 16 : 8);
    const int c0 = part * kCols;
    const uint32_t at = tm_d + d * NT + c0 + (static_cast<uint32_t>(quad * 32) << 16);
    const int64_t n = static_cast<int64_t>(t.n_tile) * 128 + quad * 32 + lane;
    if (split > 1) {                      // fp32 sums for the cluster's reduction, [NT][128] in the ring:
      float* sums = reinterpret_cast<float*>(ring);   // one tile per CTA, every copy has been waited for
#pragma unroll 1
      for (int c = 0; c < kCols; c += kChunk) {
        uint32_t r[kChunk];
        if constexpr (kChunk == 32) tmem_ld_32x32b_x32(at + c, r);
        else if constexpr (kChunk == 16) tmem_ld_32x32b_x16(at + c, r);
        else tmem_ld_32x32b_x8(at + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
          sums[(c0 + c + j) * 128 + quad * 32 + lane] = __uint_as_float(r[j]) * kSumScale;
      }
      return;
    }
    const float bias = p.bias && n < p.N ? __bfloat162float(p.bias[n]) : 0.f;
    uint32_t packed[kCols / 2];
#pragma unroll
    for (int c = 0; c < kCols; c += kChunk) {
      uint32_t r[kChunk];
      if constexpr (kChunk == 32) tmem_ld_32x32b_x32(at + c, r);
      else if constexpr (kChunk == 16) tmem_ld_32x32b_x16(at + c, r);
      else tmem_ld_32x32b_x8(at + c, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(fmaf(__uint_as_float(r[2 * j]), kSumScale, bias),
                                                       fmaf(__uint_as_float(r[2 * j + 1]), kSumScale, bias));
        packed[c / 2 + j] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(&d_empty[d]);
    if (n < p.N) {
      uint16_t* out = reinterpret_cast<uint16_t*>(p.C) + static_cast<int64_t>(t.m0 + c0) * p.N + n;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        if (c0 + c < toks) *out = static_cast<uint16_t>(packed[c / 2] >> (16 * (c & 1)));
        out += p.N;
      }
    }
  };

  if (warp >= 2 && warp < 2 + Sh::kConvWarps) {
    const int group_id = (warp - 2) >> 2;      // group
    const int row = quad * 32 + lane;
    constexpr int GB = 128 / G;            // groups in a block
    // cursor of the scales, one block (of this group) ahead of the conversion
    int sc_tile = 0, sc_block = group_id;
    const __nv_bfloat16* sr = nullptr;
    const uint8_t* zr = nullptr;
    auto enter_tile = [&] {
      const Tile t = tile_at(sc_tile);
      const int64_t left = p.N - t.n_tile * 128ll;
      const int64_t w = t.expert * p.N + t.n_tile * 128ll + (row < left ? row : left - 1);   // past N: not stored
      sr = p.scales + w * groups;
      zr = kZeros ? p.zeros + w * groups : nullptr;
    };
    // of a block's groups, packed as they lie in memory and taken apart at their use: a load whose result
    // is unpacked where two ways of loading meet would be waited for there.  One load instead of one per
    // group: [24576, 4096], 64 tokens, G = 32 with zero points 55 -> 27 us; [5120, 25600], 37 tokens, G = 64
    // with zero points 35.7 -> 31.6 us.
    uint32_t s_next[(GB + 1) / 2], z_next = 0;
    auto load_scales = [&] {
      if (sc_tile >= mine) return;
      const int at = (kb_lo + sc_block) * GB;
      if constexpr (GB == 1) {
        s_next[0] = __bfloat16_as_ushort(__ldg(sr + at));
        if (kZeros) z_next = __ldg(zr + at);
        return;
      }
      if (p.vec_scales) {                  // in one load each
        if constexpr (GB == 4) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(sr + at));
          s_next[0] = v.x;
          s_next[GB / 2 - 1] = v.y;
          if (kZeros) z_next = __ldg(reinterpret_cast<const uint32_t*>(zr + at));
        } else {
          s_next[0] = __ldg(reinterpret_cast<const uint32_t*>(sr + at));
          if (kZeros) z_next = __ldg(reinterpret_cast<const uint16_t*>(zr + at));
        }
        return;
      }
      z_next = 0;
#pragma unroll
      for (int j = 0; j < GB; ++j) {
        const int a = at + j < groups ? at + j : groups - 1;   // past K: the activations are zero
        const uint32_t v = __bfloat16_as_ushort(__ldg(sr + a));
        s_next[j / 2] = j & 1 ? s_next[j / 2] | v << 16 : v;
        if (kZeros) z_next |= static_cast<uint32_t>(__ldg(zr + a)) << (8 * j);
      }
    };
    auto next_scales = [&] {               // this group's next block
      sc_block += kGroups;
      if (sc_block >= blocks) {
        do {
          sc_block -= blocks;
          ++sc_tile;
        } while (sc_block >= blocks);
        if (sc_tile < mine) enter_tile();
      }
      load_scales();
    };
    while (sc_block >= blocks) {
      sc_block -= blocks;
      ++sc_tile;
    }
    if (sc_tile < mine) enter_tile();
    load_scales();
    int s = group_id % kRing, b = group_id;        // ring slot and converted-block slot
    uint32_t s_phase = 0, b_phase = 1;     // the first kA blocks find their slot free
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t swizzle = (row >> 1) & 3;
    int k = 0, i = group_id;               // tile, block
    // With one accumulator and no warps of its own, the epilogue of a tile runs
    // after this group's first block of the next one: the MMAs of the tile end
    // meanwhile, and the next tile starts with converted blocks at hand.
    auto epilogue_of = [&](int tile) {
      if (ok) epilogue(tile, 0, tile & 1);
    };
    for (; k < mine && ok; ++k) {
      bool due = Sh::kTwo && k > 0;
      for (; i < blocks; i += kGroups) {
        uint32_t factor[GB], offset[GB];
#pragma unroll
        for (int j = 0; j < GB; ++j) {
          const float sf = __uint_as_float(j & 1 ? s_next[j / 2] & 0xFFFF0000u : s_next[j / 2] << 16);   // bf16
          if constexpr (kZeros) {
            factor[j] = bf16x2_same(sf * 0x1p-34f);      // of (q - z) / 64
            offset[j] = int4_offset(z_next >> (8 * j));
          } else {
            factor[j] = scale_factors(sf);
            offset[j] = bf16x2_same(sf * -0x1p-37f);     // -8 s 2^-40
          }
        }
        next_scales();
        if (!__all_sync(0xffffffffu, mbar_wait(&full[s], s_phase, p.wait_limit_ns))) {   // the warp stays together
          ok = false;
          break;
        }
        uint32_t w[16];
        const uint32_t at = smem_addr(ring + s * Sh::kStage) + row * 64;
#pragma unroll
        for (int c = 0; c < 4; ++c)        // 16-byte pieces, exchanged by (row / 2) mod 4 (the 64-byte swizzle)
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
            if constexpr (kZeros)          // (q - z) / 64 is exact; one rounding here
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
        s += kGroups;
        if (s >= kRing) {
          s -= kRing;
          s_phase ^= 1;
        }
        b += kGroups;
        if (b >= kA) {
          b -= kA;
          b_phase ^= 1;
        }
        if (due) {
          epilogue_of(k - 1);
          due = false;
        }
      }
      if (due) epilogue_of(k - 1);
      i -= blocks;                         // the first block of the next tile that is this group's
    }
    if (Sh::kTwo && mine > 0) epilogue_of(mine - 1);
  }
  if constexpr (!Sh::kTwo) {
    if (warp >= Sh::kEpiFirst) {
      int d = 0;
      uint32_t d_phase = 0;
      for (int k = 0; k < mine && ok; ++k) {
        epilogue(k, d, d_phase);
        if (++d == kD) {
          d = 0;
          d_phase ^= 1;
        }
      }
    }
  }

  if (split > 1) {                        // one tile per cluster: add the ranks' sums in rank order
    const Tile t = tile_at(0);
    const int toks = t.m1 - t.m0;
    const int64_t n0 = static_cast<int64_t>(t.n_tile) * 128;
    const float* sums = reinterpret_cast<const float*>(ring);
    __syncwarp();
    cluster_sync_all();
    for (int j = threadIdx.x;; j += Sh::kThreads) {
      const int tok = (j >> 4) * split + rank, c = (j & 15) * 8;
      if (tok >= toks) break;
      if (n0 + c >= p.N) continue;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      const uint32_t at = smem_addr(sums + tok * 128 + c);
      for (int r = 0; r < split; ++r) {
        const uint32_t from = dsmem_map(at, r);
        const float4 a = dsmem_ld_f32x4(from), b = dsmem_ld_f32x4(from + 16);
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
      }
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (p.bias) {
          v[2 * e] += __bfloat162float(p.bias[n0 + c + 2 * e]);
          v[2 * e + 1] += __bfloat162float(p.bias[n0 + c + 2 * e + 1]);
        }
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
        o[e] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p.C + static_cast<int64_t>(t.m0 + tok) * p.N + n0 + c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    __syncwarp();
    cluster_sync_all();                   // nobody reads this CTA's sums any more
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tm_a, Sh::kCols);
  }
}

constexpr int kMaxSplit = 8;

// Clusters of `split` CTAs that fit on the current device at once with one CTA
// per SM (what the runtime's query counts for these kernels also where two run
// side by side): 148 CTAs less what does not pack into a GPC, which differs
// from GPU to GPU.  Cached; 0 if the query fails.
int cluster_room(const void* kernel, cudaLaunchConfig_t cfg, int dev, std::atomic<int> (&cache)[64][kMaxSplit + 1],
                 int split) {
  std::atomic<int>& slot = cache[dev & 63][split];
  int n = slot.load();
  if (n == 0) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(split);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(split));
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    slot.store(n > 0 ? n : -1);
  }
  return n > 0 ? n : 0;
}

template <int G, int NT>
cudaError_t launch_mma_gn(const Int4Params& params, cudaStream_t stream) {
  using Sh = MmaShape<NT>;
  Int4Params p = params;
  const int64_t ntiles = (p.N + 127) / 128;
  int64_t token_tiles = (p.M + NT - 1) / NT;
  if (p.expert_offsets) token_tiles += p.num_experts < p.M ? p.num_experts : p.M;   // a bound
  const int64_t tiles = ntiles * token_tiles;
  if (tiles > 0x7FFFFFFF / 2) return cudaErrorInvalidValue;   // the host checks this first
  CUtensorMap tmW, tmX;
  const int64_t rows = p.N * (p.expert_offsets ? p.num_experts : 1);
  if (!encode_tma_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.B, p.K / 2, rows, p.K / 2, 64, 128,
                     CU_TENSOR_MAP_SWIZZLE_64B) ||
      !encode_tma_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.x, p.K, p.M, p.K * 2, 64, NT,
                     CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const bool zeros = p.zeros != nullptr;
  auto kernel = zeros ? int4_mma_kernel<G, NT, true> : int4_mma_kernel<G, NT, false>;
  static std::atomic<uint64_t> prepared[2];   // devices (by bit) whose kernel has its attributes, per kZeros
  static std::atomic<int> smem_bytes[2];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(prepared[zeros].load() & bit)) {
    // Half an SM's shared memory exactly (228 KB, 1 KB reserved per CTA) where two CTAs run side by
    // side: then no CTA that allocates all tensor-memory columns fits beside one (those of this library
    // take more than half), and CTAs of clusters never wait for columns held by each other's peers.
    cudaFuncAttributes attributes;
    e = cudaFuncGetAttributes(&attributes, kernel);
    if (e != cudaSuccess) return e;
    const int half = 114 * 1024 - 1024 - static_cast<int>(attributes.sharedSizeBytes);
    const int bytes = Sh::kTwo ? half : Sh::kSmem;
    if (bytes < Sh::kSmem) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    // without it the driver may size the shared memory for one CTA per SM
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    smem_bytes[zeros].store(bytes);
    prepared[zeros].fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(Sh::kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes[zeros].load());
  cfg.stream = stream;

  // Split-K: few tiles, each shared by a cluster of as many CTAs as find an SM
  // of their own and keep at least 8 blocks each; as many as fit two per SM where
  // those with an SM of their own would have 48 blocks or more.  Measured on
  // B200, us with splits 1..8:
  // [4096, 4096], 16 tokens: 13.0 9.2 7.9 7.3 | 8.8 8.8 8.6 8.4 (two per SM from 5);
  // [4096, 12288], 64 tokens: 42.2 25.2 19.8 16.8 | 20.3 18.8 18.8 18.6;
  // [5120, 25600], 64 tokens: 86.9 47.9 34.6 | 35.7 31.4 28.3 44.5 40.6 (7 and 8 do not fit; 6 it is).
  p.split = 1;
  static std::atomic<int> room[2][64][kMaxSplit + 1];
  if (!p.expert_offsets && tiles <= 148) {
    const int64_t blocks = (p.K + 127) / 128;
    auto widest = [&](int per_sm) {
      for (int c = kMaxSplit; c > 1; --c)
        if (blocks >= 8 * c &&
            tiles <= per_sm * cluster_room(reinterpret_cast<const void*>(kernel), cfg, dev, room[zeros], c))
          return c;
      return 1;
    };
    p.split = widest(1);
    if (Sh::kTwo && blocks >= 48 * p.split) p.split = widest(2);
  }
  int64_t ctas = sm_count() * (Sh::kTwo ? 2 : 1);
  if (p.split > 1 || ctas > tiles) ctas = tiles;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas * p.split));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, p);
}

template <int G>
cudaError_t launch_mma_g(const Int4Params& p, int tile, cudaStream_t stream) {
  switch (tile) {
    case 16: return launch_mma_gn<G, 16>(p, stream);
    case 32: return launch_mma_gn<G, 32>(p, stream);
    case 64: return launch_mma_gn<G, 64>(p, stream);
    case 128: return launch_mma_gn<G, 128>(p, stream);
    default: return launch_mma_gn<G, 256>(p, stream);
  }
}

}  // namespace

int int4_mma_max_experts() { return kMaxGroupedExperts; }

cudaError_t launch_int4_mma(const Int4Params& p, int group, int tile, cudaStream_t stream) {
  switch (group) {
    case 32: return launch_mma_g<32>(p, tile, stream);
    case 64: return launch_mma_g<64>(p, tile, stream);
    default: return launch_mma_g<128>(p, tile, stream);
  }
}

}  // namespace lq
