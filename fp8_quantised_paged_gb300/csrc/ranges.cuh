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

// Cuts the blocks' `tiles` token tiles (v.rb_pre), for every KV head, into ranges of the
// same cost.  cost(i): of the blocks before block i (of one KV head), where an item (a block
// and KV head) costs `item` and as much for each of its tiles.  A cut within kSnap tiles of an
// item's edge moves there.  Run by one CTA.
template <typename Cost>
__device__ __forceinline__ void cut_ranges(const PlanView& v, int blocks, int tiles, int hkv,
                                           int ranges, int item, const Cost& cost) {
  const int tid = threadIdx.x;
  const int U = tiles * hkv;
  const long long all = cost(blocks) * hkv;
  const long long upw = max(1ll, (all + ranges - 1) / ranges);
  if (tid == 0) v.head[0] = U;
  for (int w = tid; w <= ranges; w += kPlanThreads) {
    const long long want = w * upw;
    int u = U, it = blocks * hkv;
    if (want < all) {
      int lo = 0, hi = blocks;  // the block that holds it
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cost(mid) * hkv <= want) lo = mid;
        else hi = mid;
      }
      const int rb = lo, pre = v.rb_pre[rb], c = v.rb_pre[rb + 1] - pre;
      const long long first = cost(rb), each = cost(rb + 1) - first, in = want - first * hkv;
      const int h = static_cast<int>(in / each), f = pre * hkv + h * c;
      const int tile = static_cast<int>(max(in - h * each - item, 0ll) * c / (each - item));
      it = rb * hkv + h;
      u = f + tile;
      if (tile < kSnap) {
        u = f;
      } else if (c - tile < kSnap) {
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
