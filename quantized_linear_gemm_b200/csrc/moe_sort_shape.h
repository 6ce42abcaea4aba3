// How the sort of a mixture-of-experts batch (moe_kernels.cu) is cut into CTAs
// and warps.  Plain C++, so that a host program can check it.
#pragma once

#include <cstdint>

namespace lq {

constexpr int kSortWarps = 32;
constexpr int kSortThreads = 32 * kSortWarps;
constexpr int kSortPortableCluster = 8;
constexpr int kSortMaxCluster = 16;     // more than 8 CTAs need the non-portable attribute and 16 free SMs of one GPC

struct SortShape {
  int ctas;      // one cluster
  int64_t seg;   // consecutive ids of a warp, a multiple of 32
};

// One CTA per 1024 ids, a power of two, at most `widest`.
constexpr SortShape sort_shape(int64_t n, int widest) {
  int ctas = 1;
  while (ctas < widest && n > static_cast<int64_t>(ctas) * kSortThreads) ctas *= 2;
  const int64_t warps = static_cast<int64_t>(ctas) * kSortWarps;
  return {ctas, (((n + warps - 1) / warps) + 31) / 32 * 32};
}

// The widest cluster, from what the occupancy query says: CUDA's error code of
// the query (0: success) and the clusters of kSortMaxCluster CTAs that fit.
constexpr int sort_widest(int query_error, int fitting) {
  return query_error == 0 && fitting > 0 ? kSortMaxCluster : kSortPortableCluster;
}

}  // namespace lq
