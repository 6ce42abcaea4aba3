// Token movement of a mixture-of-experts layer around the grouped products:
//
//   sort       ids [n] -> offsets [E + 1], order [n], slots [n]: a stable
//              counting sort by expert (order[p] = i and slots[i] = p when the
//              i-th id is the p-th row); ids outside [0, E) get slot -1;
//   permute    xs[slots[t, j]] = x[t], in bf16 or quantized per token;
//   unpermute  out[t] = sum_j w[t, j] y[slots[t, j]] (w = 1 without weights:
//              the gradient of permute);
//   backward   dy[slots[t, j]] = w[t, j] dout[t],
//              dw[t, j] = sum_h dout[t, h] y[slots[t, j], h].
//
// The grouped product's expert offsets (ai-radar.it, "Helion in vLLM: il
// tuning dei GEMM diventa ricerca, non artigianato GPU", section "Oltre
// Hopper: Blackwell, AMD, TPU e il perimetro del fork") are the sort's output.
// Nothing here uses atomics: every output is written by one thread and every
// sum has a fixed order, so results are reproducible bit for bit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "lq_kernels.h"
#include "moe_sort_shape.h"
#include "ptx.cuh"
#include "quant_common.cuh"

namespace lq {
namespace {

constexpr int kSortMaxExperts = 1024;   // one scan thread per expert, 4 KB of counts per expert row of a warp

// ------------------------------------------------------------------ sort
//
// One cluster of up to 16 CTAs does the whole sort in one launch and without
// a workspace.  Each warp owns a contiguous segment of ids and counts it into
// its own row of shared memory, 32 ids at a time: lanes with the same expert
// find each other by one ballot per bit of the expert's number (the match
// instruction takes time in proportion to the different values, over 1 us with
// 128 experts), and one of them adds their number.  Prefix sums over the warps
// of a CTA, the CTAs of the cluster (distributed shared memory) and the experts
// give every (warp, expert) its first row; a second pass over the segment places the ids.  No two warps
// share a counter, so the order within an expert is the order of the ids.
// Latency bound: 64 ids of 128 experts 2.9 us, 4096 5.6 us, 65536 10.1 us (64-bit
// ids 10.7; 22.6 us with the match instruction and 8 CTAs); one CTA per 1024 ids.
// The second pass reads the ids and takes the ballots again.

// lanes whose key, of `bits` bits, is this lane's
__device__ __forceinline__ uint32_t same_key(int key, int bits) {
  uint32_t same = 0xffffffffu;
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b) & 1;
    const uint32_t v = __ballot_sync(0xffffffffu, one);
    same &= one ? v : ~v;
  }
  return same;
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads) moe_sort_kernel(const Id* __restrict__ ids, int64_t n, int E,
                                                                int64_t seg, int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ order,
                                                                int32_t* __restrict__ slots) {
  extern __shared__ int32_t sort_smem[];
  const int stride = E | 1;                        // odd: a column's rows lie in different banks
  int32_t* counts = sort_smem;                     // [kSortWarps][stride]
  int32_t* cta_total = counts + kSortWarps * stride;    // [E], read by the cluster's other CTAs
  int32_t* base = cta_total + E;                   // [E] first row of this CTA's ids of each expert
  __shared__ int32_t warp_sum[kSortWarps];
  __shared__ int32_t grand_total;
  grid_launch_dependents();
  grid_dependency_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  const int bits = 32 - __clz(E);                  // keys 0..E
  int32_t* mine = counts + warp * stride;
  for (int e = lane; e < E; e += 32) mine[e] = 0;
  __syncwarp();
  const int64_t lo = (static_cast<int64_t>(cta) * kSortWarps + warp) * seg;
  const int64_t hi = lo + seg < n ? lo + seg : n;
  auto key_at = [&](int64_t i) -> int {            // E for ids outside [0, E) and past the end
    if (i >= hi) return E;
    const Id id = ids[i];
    return id >= 0 && id < static_cast<Id>(E) ? static_cast<int>(id) : E;
  };
  constexpr int kBatch = 8;                        // ids in flight per lane
  for (int64_t i0 = lo; i0 < hi; i0 += 32 * kBatch) {
    int key[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) key[b] = key_at(i0 + 32 * b + lane);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (i0 + 32 * b >= hi) break;
      const uint32_t same = same_key(key[b], bits);
      if (key[b] < E && (__ffs(same) - 1) == lane) mine[key[b]] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  // exclusive prefix over the warps, expert by expert: 8 threads per expert, 4 warps' counts each
  for (int e0 = 0; e0 < E; e0 += kSortThreads / 8) {
    const int e = e0 + (tid >> 3), r = tid & 7;
    int c[4] = {0, 0, 0, 0};
    if (e < E)
#pragma unroll
      for (int q = 0; q < 4; ++q) c[q] = counts[(4 * r + q) * stride + e];
    const int sum = c[0] + c[1] + c[2] + c[3];
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o, 8);
      if (r >= o) upto += v;
    }
    int run = upto - sum;
    if (e < E) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        counts[(4 * r + q) * stride + e] = run;
        run += c[q];
      }
      if (r == 7) cta_total[e] = upto;
    }
  }
  __syncthreads();
  int total = tid < E ? cta_total[tid] : 0, before = 0;   // of expert `tid`: rows in the batch, rows in earlier CTAs
  if (ctas > 1) {
    cluster_sync_all();
    if (tid < E) {
      total = 0;
      const uint32_t at = smem_addr(cta_total + tid);
      for (int c = 0; c < ctas; ++c) {
        const int v = static_cast<int>(dsmem_ld_u32(dsmem_map(at, c)));
        before += c < cta ? v : 0;
        total += v;
      }
    }
    cluster_arrive_release();                      // this CTA no longer reads the others' totals
  }
  // exclusive prefix over the experts
  int incl = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int v = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    warp_sum[lane] = v;
    if (lane == 31) grand_total = v;
  }
  __syncthreads();
  const int first = incl - total + (warp ? warp_sum[warp - 1] : 0);
  if (tid < E) {
    base[tid] = first + before;
    if (cta == 0) offsets[tid] = first;
  }
  if (cta == 0 && tid == 0) offsets[E] = grand_total;
  __syncthreads();
  for (int64_t i0 = lo; i0 < hi; i0 += 32 * kBatch) {
    int key[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) key[b] = key_at(i0 + 32 * b + lane);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int64_t i = i0 + 32 * b + lane;
      if (i0 + 32 * b >= hi) break;
      const uint32_t same = same_key(key[b], bits);
      int at = 0;
      if (key[b] < E) at = mine[key[b]];
      __syncwarp();
      if (key[b] < E) {
        const int slot = base[key[b]] + at + __popc(same & ((1u << lane) - 1u));
        slots[i] = slot;
        order[slot] = static_cast<int32_t>(i);
        if ((__ffs(same) - 1) == lane) mine[key[b]] = at + __popc(same);
      } else if (i < hi) {
        slots[i] = -1;
      }
      __syncwarp();
    }
  }
  // rows behind the last expert's
  for (int64_t p = grand_total + static_cast<int64_t>(cta) * kSortThreads + tid; p < n;
       p += static_cast<int64_t>(ctas) * kSortThreads)
    order[p] = -1;
  if (ctas > 1) cluster_wait_acquire();            // the others may still have been reading cta_total
}

// --------------------------------------------------------------- permute
//
// One thread holds one 16-byte piece of a token's row and stores it at each of
// the token's slots: x is read once and every copy written once.  Bound by
// the writes: 4096 tokens of 2048 values at 8 slots 25.3 us, 0.91 of the copy
// rate; 32 tokens 1.5 us, the launch.
constexpr int kRowThreads = 128;
constexpr int kSlotBatch = 8;   // slots (and, in the sums, rows) in flight per thread

__device__ __forceinline__ bool row_ok(int32_t slot, int64_t P) { return slot >= 0 && slot < P; }

__global__ void __launch_bounds__(kRowThreads) moe_permute_kernel(const uint4* __restrict__ x,
                                                                  const int32_t* __restrict__ slots,
                                                                  uint4* __restrict__ xs, int64_t P, int k,
                                                                  int64_t nvec) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t t = blockIdx.x;
  const int64_t v = static_cast<int64_t>(blockIdx.y) * kRowThreads + threadIdx.x;
  if (v >= nvec) return;
  const uint4 val = __ldg(x + t * nvec + v);
  const int32_t* st = slots + t * k;
  for (int j0 = 0; j0 < k; j0 += kSlotBatch) {
    int32_t s[kSlotBatch];
#pragma unroll
    for (int j = 0; j < kSlotBatch; ++j) s[j] = j0 + j < k ? __ldg(st + j0 + j) : -1;
#pragma unroll
    for (int j = 0; j < kSlotBatch; ++j)
      if (row_ok(s[j], P)) xs[static_cast<int64_t>(s[j]) * nvec + v] = val;
  }
}

// ... with the per-token quantization of quant_kernels.cu: one CTA per token,
// the row in registers (VPT pieces of 8 values per thread; VPT = 0: longer
// rows, read twice), its codes stored at each slot.  Same codes and scales,
// bit for bit, as quantizing x first.  Bound by the writes at many tokens, by
// the row's maximum before them at fewer: 8192 tokens of 2048 values at 8 slots
// 29.4 us, 0.87 of the copy rate, 4096 tokens 16.2 us, 0.79; 32 tokens 1.8 us.
constexpr int kQuantThreads = 256;

__device__ __forceinline__ float block_max_256(float v, float* red) {
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) v = fmaxf(v, red[w]);
  return v;
}

template <bool kInt8, int VPT>
__global__ void __launch_bounds__(kQuantThreads) moe_permute_quant_kernel(const uint4* __restrict__ x,
                                                                          const int32_t* __restrict__ slots,
                                                                          uint2* __restrict__ q,
                                                                          float* __restrict__ scales, int64_t P,
                                                                          int k, int64_t nvec) {
  __shared__ float red[kQuantThreads / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t t = blockIdx.x;
  const uint4* xr = x + t * nvec;
  const int32_t* st = slots + t * k;
  uint4 v[VPT ? VPT : 1];
  float a = 0.f;
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t idx = threadIdx.x + i * kQuantThreads;
      v[i] = idx < nvec ? __ldg(xr + idx) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[8];
      bf16x8_to_f32(v[i], f);
      a = fmaxf(a, amax8(f));
    }
  } else {
    for (int64_t idx = threadIdx.x; idx < nvec; idx += kQuantThreads) {
      float f[8];
      bf16x8_to_f32(__ldg(xr + idx), f);
      a = fmaxf(a, amax8(f));
    }
  }
  const float amax = block_max_256(a, red);
  const float s = scale_from_amax(amax, kInt8 ? kInt8Max : kE4m3Max);
  const Divisor d = make_divisor(amax, s);
  for (int j = threadIdx.x; j < k; j += kQuantThreads) {
    const int32_t slot = __ldg(st + j);
    if (row_ok(slot, P)) scales[slot] = s;
  }
  auto put = [&](const uint4& val, int64_t idx) {
    float f[8];
    bf16x8_to_f32(val, f);
    const uint2 code = kInt8 ? encode8_int8(f, d) : encode8_e4m3(f, d);
    for (int j0 = 0; j0 < k; j0 += kSlotBatch) {
      int32_t sl[kSlotBatch];
#pragma unroll
      for (int j = 0; j < kSlotBatch; ++j) sl[j] = j0 + j < k ? __ldg(st + j0 + j) : -1;
#pragma unroll
      for (int j = 0; j < kSlotBatch; ++j)
        if (row_ok(sl[j], P)) q[static_cast<int64_t>(sl[j]) * nvec + idx] = code;
    }
  };
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t idx = threadIdx.x + i * kQuantThreads;
      if (idx < nvec) put(v[i], idx);
    }
  } else {
    for (int64_t idx = threadIdx.x; idx < nvec; idx += kQuantThreads) put(__ldg(xr + idx), idx);
  }
}

// ------------------------------------------------------------- unpermute
//
// One thread sums one 16-byte piece over the token's rows, in the order
// j = 0..k-1 in fp32, and rounds once to bf16.  Up to eight rows are in
// flight per thread.  A row whose slot is outside [0, P) is not read, so
// whatever it would hold (NaN included) cannot reach the sum.  Bound by the
// reads: 4096 tokens of 8 rows of 2048 values 25.3 us, 0.91 of the copy rate;
// 32 tokens 2.1 us, the launch and two dependent loads.
__global__ void __launch_bounds__(kRowThreads) moe_unpermute_kernel(const uint4* __restrict__ y,
                                                                    const int32_t* __restrict__ slots,
                                                                    const float* __restrict__ weights,
                                                                    uint4* __restrict__ out, int64_t P, int k,
                                                                    int64_t nvec) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t t = blockIdx.x;
  const int64_t v = static_cast<int64_t>(blockIdx.y) * kRowThreads + threadIdx.x;
  if (v >= nvec) return;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < k; j0 += kSlotBatch) {
    int32_t s[kSlotBatch];
    float w[kSlotBatch];
    uint4 r[kSlotBatch];
#pragma unroll
    for (int j = 0; j < kSlotBatch; ++j) {
      s[j] = j0 + j < k ? __ldg(slots + t * k + j0 + j) : -1;
      w[j] = j0 + j < k && weights ? __ldg(weights + t * k + j0 + j) : 1.f;
    }
#pragma unroll
    for (int j = 0; j < kSlotBatch; ++j)
      if (row_ok(s[j], P)) r[j] = __ldg(y + static_cast<int64_t>(s[j]) * nvec + v);
#pragma unroll
    for (int j = 0; j < kSlotBatch; ++j)
      if (row_ok(s[j], P)) {
        float f[8];
        bf16x8_to_f32(r[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[j], f[i], acc[i]);
      }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
    o[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  out[t * nvec + v] = make_uint4(o[0], o[1], o[2], o[3]);
}

// Gradients of the weighted sum: one CTA per token.  Each thread holds its
// pieces of dout, writes w dout at every slot and adds up its part of the dot
// products with the rows of y; the CTA's parts are summed in a fixed order
// (lanes by shuffles, then the warps in turn).  Eight slots at a time, so dout
// (in L1 after the first time) is read again only when k > 8.  Bound by HBM:
// 4096 tokens of 8 rows of 2048, 45.4 us, 0.96 of the copy rate (52.5 us with
// 256 threads per token and cached loads and stores: the barrier of the sum
// held too many loads back).
constexpr int kBwdThreads = 128;

__global__ void __launch_bounds__(kBwdThreads) moe_unpermute_backward_kernel(
    const uint4* __restrict__ dout, const uint4* __restrict__ y, const int32_t* __restrict__ slots,
    const float* __restrict__ weights, uint4* __restrict__ dy, float* __restrict__ dweights, int64_t P, int k,
    int64_t nvec) {
  __shared__ float part[kBwdThreads / 32][kSlotBatch];
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j0 = 0; j0 < k; j0 += kSlotBatch) {
    int32_t s[kSlotBatch];
    float w[kSlotBatch], dot[kSlotBatch];
#pragma unroll
    for (int j = 0; j < kSlotBatch; ++j) {
      s[j] = j0 + j < k ? __ldg(slots + t * k + j0 + j) : -1;
      w[j] = j0 + j < k ? __ldg(weights + t * k + j0 + j) : 0.f;
      dot[j] = 0.f;
    }
    for (int64_t v = threadIdx.x; v < nvec; v += kBwdThreads) {
      uint4 r[kSlotBatch];
#pragma unroll
      for (int j = 0; j < kSlotBatch; ++j)
        if (row_ok(s[j], P)) r[j] = __ldcs(y + static_cast<int64_t>(s[j]) * nvec + v);
      float d[8];
      bf16x8_to_f32(__ldg(dout + t * nvec + v), d);
#pragma unroll
      for (int j = 0; j < kSlotBatch; ++j)
        if (row_ok(s[j], P)) {
          float f[8];
          bf16x8_to_f32(r[j], f);
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            dot[j] = fmaf(d[2 * i], f[2 * i], dot[j]);
            dot[j] = fmaf(d[2 * i + 1], f[2 * i + 1], dot[j]);
            const __nv_bfloat162 p = __floats2bfloat162_rn(w[j] * d[2 * i], w[j] * d[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t*>(&p);
          }
          __stcs(dy + static_cast<int64_t>(s[j]) * nvec + v, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
#pragma unroll
    for (int j = 0; j < kSlotBatch; ++j)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
    if (lane == 0)
#pragma unroll
      for (int j = 0; j < kSlotBatch; ++j) part[warp][j] = dot[j];
    __syncthreads();
    if (threadIdx.x < kSlotBatch && j0 + static_cast<int>(threadIdx.x) < k) {
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < kBwdThreads / 32; ++q) sum += part[q][threadIdx.x];
      dweights[t * k + j0 + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

cudaLaunchConfig_t pdl_config(dim3 grid, dim3 block, size_t smem, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

dim3 row_grid(int64_t T, int64_t nvec) {
  return dim3(static_cast<unsigned>(T), static_cast<unsigned>((nvec + kRowThreads - 1) / kRowThreads));
}

constexpr size_t sort_smem_bytes(int E) {
  return sizeof(int32_t) * (static_cast<size_t>(E | 1) * kSortWarps + 2 * static_cast<size_t>(E));
}

// The kernel's limits, set once per device to what the most experts need: a
// limit that followed each call's E would be lowered by one host thread between
// another's setting and its launch.  With them the widest cluster: 16 CTAs where
// the device has room for one with that much shared memory, else 8, which every
// device takes.
template <typename Id>
cudaError_t prepare_sort(int* widest) {
  static std::atomic<int> prepared[64];   // per device: the widest cluster, 0 before the first call
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>& slot = prepared[dev & 63];
  *widest = slot.load();
  if (*widest) return cudaSuccess;
  constexpr size_t most = sort_smem_bytes(kSortMaxExperts);
  e = cudaFuncSetAttribute(moe_sort_kernel<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
  if (e != cudaSuccess) return e;
  int fitting = 0;
  e = cudaFuncSetAttribute(moe_sort_kernel<Id>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kSortMaxCluster;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSortMaxCluster);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = most;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&fitting, moe_sort_kernel<Id>, &cfg);
  }
  if (e != cudaSuccess) cudaGetLastError();
  *widest = sort_widest(static_cast<int>(e), fitting);
  slot.store(*widest);
  return cudaSuccess;
}

template <typename Id>
cudaError_t launch_sort_t(const void* ids, int64_t n, int E, int32_t* offsets, int32_t* order, int32_t* slots,
                          cudaStream_t stream) {
  int widest = 0;
  const cudaError_t e = prepare_sort<Id>(&widest);
  if (e != cudaSuccess) return e;
  const SortShape shape = sort_shape(n, widest);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pdl_config(dim3(shape.ctas), dim3(kSortThreads), sort_smem_bytes(E), stream, attr);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = shape.ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, moe_sort_kernel<Id>, static_cast<const Id*>(ids), n, E, shape.seg, offsets,
                            order, slots);
}

}  // namespace

int moe_sort_max_experts() { return kSortMaxExperts; }

cudaError_t launch_moe_sort(const void* ids, int id_bytes, int64_t n, int E, int32_t* offsets, int32_t* order,
                            int32_t* slots, cudaStream_t stream) {
  return id_bytes == 8 ? launch_sort_t<int64_t>(ids, n, E, offsets, order, slots, stream)
                       : launch_sort_t<int32_t>(ids, n, E, offsets, order, slots, stream);
}

cudaError_t launch_moe_permute(const void* x, const int32_t* slots, void* xs, int64_t T, int64_t P, int k, int64_t H,
                               cudaStream_t stream) {
  const int64_t nvec = H / 8;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(row_grid(T, nvec), dim3(kRowThreads), 0, stream, attr);
  return cudaLaunchKernelEx(&cfg, moe_permute_kernel, static_cast<const uint4*>(x), slots, static_cast<uint4*>(xs), P,
                            k, nvec);
}

cudaError_t launch_moe_permute_quant(int fmt, const void* x, const int32_t* slots, void* q, float* scales, int64_t T,
                                     int64_t P, int k, int64_t H, cudaStream_t stream) {
  const int64_t nvec = H / 8;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(T)), dim3(kQuantThreads), 0, stream, attr);
  const auto* xp = static_cast<const uint4*>(x);
  auto* qp = static_cast<uint2*>(q);
  const bool i8 = fmt == kFmtInt8;
#define LQ_PERM(V)                                                                                                   \
  return i8 ? cudaLaunchKernelEx(&cfg, moe_permute_quant_kernel<true, V>, xp, slots, qp, scales, P, k, nvec)         \
            : cudaLaunchKernelEx(&cfg, moe_permute_quant_kernel<false, V>, xp, slots, qp, scales, P, k, nvec);
  if (nvec <= kQuantThreads) { LQ_PERM(1) }
  if (nvec <= 2 * kQuantThreads) { LQ_PERM(2) }
  if (nvec <= 4 * kQuantThreads) { LQ_PERM(4) }
  if (nvec <= 8 * kQuantThreads) { LQ_PERM(8) }
  LQ_PERM(0)
#undef LQ_PERM
}

cudaError_t launch_moe_unpermute(const void* y, const int32_t* slots, const float* weights, void* out, int64_t T,
                                 int64_t P, int k, int64_t H, cudaStream_t stream) {
  const int64_t nvec = H / 8;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(row_grid(T, nvec), dim3(kRowThreads), 0, stream, attr);
  return cudaLaunchKernelEx(&cfg, moe_unpermute_kernel, static_cast<const uint4*>(y), slots, weights,
                            static_cast<uint4*>(out), P, k, nvec);
}

cudaError_t launch_moe_unpermute_backward(const void* dout, const void* y, const int32_t* slots, const float* weights,
                                          void* dy, float* dweights, int64_t T, int64_t P, int k, int64_t H,
                                          cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(T)), dim3(kBwdThreads), 0, stream, attr);
  return cudaLaunchKernelEx(&cfg, moe_unpermute_backward_kernel, static_cast<const uint4*>(dout),
                            static_cast<const uint4*>(y), slots, weights, static_cast<uint4*>(dy), dweights, P, k,
                            H / 8);
}

}  // namespace lq
