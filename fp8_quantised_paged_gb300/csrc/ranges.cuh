// ranges.cuh -- what the planners of the prefill and the tree attention share: the row
// blocks' tiles cut into one contiguous range per SM.
#pragma once

#include "prefill.cuh"
#include "scan.cuh"

namespace fp8pa {

namespace {

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Bound of a batch's blocks of `rows` rows.
inline int block_bound(int total_q, int batch, int G, int rows = kRows) {
  return static_cast<int>((static_cast<long long>(total_q) * G + rows - 1) / rows) + batch;
}

// Largest i in [0, n) with a[i] <= x (a nondecreasing, a[0] <= x).
__device__ __forceinline__ int last_le(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Cuts the blocks' `tiles` token tiles (v.rb_pre), for every KV head, into ranges; a cut
// within kSnap tiles of an item's edge moves there.  Run by one CTA.
__device__ __forceinline__ void cut_ranges(const PlanView& v, int blocks, int tiles, int hkv,
                                           int ranges) {
  const int tid = threadIdx.x;
  const int U = tiles * hkv;
  const int upw = max(1, (U + ranges - 1) / ranges);
  if (tid == 0) {
    v.head[0] = U;
    v.head[1] = upw;
  }
  for (int w = tid; w <= ranges; w += kPlanThreads) {
    const long long want = static_cast<long long>(w) * upw;
    int u = want < U ? static_cast<int>(want) : U, it = blocks * hkv;
    if (u < U) {
      const int rb = last_le(v.rb_pre, blocks, u / hkv);
      const int pre = v.rb_pre[rb], c = v.rb_pre[rb + 1] - pre;
      const int h = (u - pre * hkv) / c, f = pre * hkv + h * c;
      it = rb * hkv + h;
      if (u - f < kSnap) {
        u = f;
      } else if (f + c - u < kSnap) {
        u = f + c;
        ++it;
      }
    }
    v.start[w] = u;
    v.item[w] = it;
  }
}

}  // namespace

}  // namespace fp8pa
