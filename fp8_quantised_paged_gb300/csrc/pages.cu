// pages.cu -- the pages of sequences that branch: keeping the accepted path of a
// drafted tree, forking, resizing and compacting.
//
// A page is free where its count is zero, and the free page with the lowest number is
// taken first, in the order of the rows, so that the result is the same whatever order
// the threads come in.  Counts are added to and taken from by atomics on integers,
// whose order does not show.
//
// Device times of the calls, in a captured graph (a plain call takes longer for its host side,
// 13 to 23 us): keep 2.8 us for one request's layer, 13.6 for 64 requests of 16 layers (3.1 and
// 15.9 where the pages' counts are looked at); fork 7.6 for one row to 4, 20.8 for 16 rows to
// 128 in 16 layers; resize 8.2 for 256 rows, 22.3 for 1024 rows of which many end or begin;
// compact 12.0 for 2K pages, 195.6 for 16K pages of 4 layers, half of them free.
#include "pages.cuh"

#include "common.cuh"
#include "scan.cuh"

namespace fp8pa {

namespace {

constexpr int kWarps = kPlanThreads / 32;
constexpr int kChunk = 2048;  // bytes that a warp copies at a time: four 16-byte loads a lane
constexpr int kCopyThreads = 256;

__host__ __device__ __forceinline__ int pages_of(int len, int bs) {
  return static_cast<int>((static_cast<long long>(len) + bs - 1) / bs);
}
__device__ __forceinline__ bool good_len(const PageRows& r, int len) {
  return len >= 0 && len <= r.max_blocks * r.bs;
}
__device__ __forceinline__ bool good_page(const PageRows& r, int page) {
  return page >= 0 && page < r.num_blocks;
}
__device__ __forceinline__ int32_t* row_of(const PageRows& r, int row) {
  return r.tables + static_cast<long>(row) * r.max_blocks;
}

// The counts of a stretch of pages, a bit per page that is free.  A warp holds kSpan
// consecutive groups of 32; all loads of a stretch are in flight at once, as one CTA
// reads them all and a round trip is what a stretch costs.
constexpr int kSpan = 16;
constexpr int kStretch = kPlanThreads * kSpan;
struct FreeBits {
  uint32_t w[kSpan];
  int base;  // page of the warp's first bit
};
__device__ __forceinline__ void load_free(const PageRows& r, int from, FreeBits& f) {
  const int lane = threadIdx.x & 31;
  f.base = from + (threadIdx.x >> 5) * (32 * kSpan);
  int c[kSpan];
#pragma unroll
  for (int i = 0; i < kSpan; ++i) {
    const int p = f.base + i * 32 + lane;
    c[i] = p < r.num_blocks && p >= from ? r.refs[p] : 1;
  }
#pragma unroll
  for (int i = 0; i < kSpan; ++i) f.w[i] = __ballot_sync(0xffffffffu, c[i] == 0);
}

// Writes the numbers of the lowest `want` free pages to list, in order; returns how
// many there are, at most `want`.  One whole CTA.
__device__ __forceinline__ int take_free(const PageRows& r, int want, int32_t* list, int* s_warp) {
  const int lane = threadIdx.x & 31;
  int got = 0;
  for (long long from = 0; from < r.num_blocks && got < want; from += kStretch) {
    FreeBits f;
    load_free(r, static_cast<int>(from), f);
    int n = 0;
#pragma unroll
    for (int i = 0; i < kSpan; ++i) n += __popc(f.w[i]);
    int at;
    const int total = block_scan(lane == 0 ? n : 0, &at, s_warp);
    at = got + __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
      const int k = at + __popc(f.w[i] & ((1u << lane) - 1u));
      if ((f.w[i] >> lane & 1u) && k < want) list[k] = f.base + i * 32 + lane;
      at += __popc(f.w[i]);
    }
    got += total;
  }
  return min(got, want);
}

// ---------------------------------------------------------------- copies of pages
// Chunk c (of every array's, a.first) of page `from` to page `to`, by one warp.
__device__ __forceinline__ void copy_chunk(const PageArrays& a, uint32_t c, int from, int to) {
  int lo = 0, hi = a.n;  // the array that holds chunk c
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= c) lo = mid;
    else hi = mid;
  }
  const uint32_t bytes = a.page_bytes[lo], at = (c - a.first[lo]) * kChunk;
  const uint8_t* src = a.ptr[lo] + static_cast<size_t>(from) * bytes + at;
  uint8_t* dst = a.ptr[lo] + static_cast<size_t>(to) * bytes + at;
  const uint32_t left = min(bytes - at, static_cast<uint32_t>(kChunk));
  uint4 v[kChunk / 512];
#pragma unroll
  for (int i = 0; i < kChunk / 512; ++i) {
    const uint32_t o = (i * 32 + (threadIdx.x & 31)) * 16;
    if (o < left) v[i] = *reinterpret_cast<const uint4*>(src + o);
  }
#pragma unroll
  for (int i = 0; i < kChunk / 512; ++i) {
    const uint32_t o = (i * 32 + (threadIdx.x & 31)) * 16;
    if (o < left) *reinterpret_cast<uint4*>(dst + o) = v[i];
  }
}

// Bound by HBM where pages are many: 1.1 GB read and written at 5.7 TB/s, 85 % of the rate of
// a plain copy (16K pages of 4 layers, half of them moved).
// Every pair's chunks, dealt over the warps of the grid: pair(k, &from, &to) says
// whether pair k < pairs is copied, and from where to where.
template <class Pair>
__device__ __forceinline__ void copy_pairs(const PageArrays& a, int pairs, Pair pair) {
  const uint32_t per = a.first[a.n];
  if (per == 0) return;
  constexpr int kW = kCopyThreads / 32;
  const uint32_t groups = (per + kW - 1) / kW;
  const unsigned long long total = static_cast<unsigned long long>(groups) * pairs;
  for (unsigned long long g = blockIdx.x; g < total; g += gridDim.x) {
    const int k = static_cast<int>(g / groups);
    const uint32_t c = static_cast<uint32_t>(g - static_cast<unsigned long long>(k) * groups) * kW +
                       (threadIdx.x >> 5);
    int from, to;
    if (c < per && pair(k, &from, &to)) copy_chunk(a, c, from, to);
  }
}

// ---------------------------------------------------------------- accepted paths
// The rows of the kept nodes move to the front of the tree's tokens: node a[t] to
// place t.  A path's nodes rise and a[t] >= t, so a move never writes a row that a
// later move reads; a warp takes one (request, array, KV head) and its moves in order,
// up to four rows' units a lane, all read before any is written.  Bound by latency: a table
// entry, a row, a write, for a few rows of 128 bytes a warp.
template <class T>
__device__ __forceinline__ void keep_rows(const PageRows& r, const int32_t* acc, int count,
                                          int ctx, const int32_t* table, uint8_t* base, int hkv,
                                          int head, int row_bytes) {
  constexpr int kDeep = 4;
  const int lane = threadIdx.x & 31;
  const int units = row_bytes / static_cast<int>(sizeof(T));
  const int total = count * units;
  auto where = [&](int place, int k) -> T* {
    const int pos = ctx + place;
    const int page = __ldg(table + pos / r.bs);
    if (!good_page(r, page)) return nullptr;
    const size_t row = (static_cast<size_t>(page) * hkv + head) * r.bs + pos % r.bs;
    return reinterpret_cast<T*>(base + row * row_bytes) + k;
  };
  for (int x0 = 0; x0 < total; x0 += 32 * kDeep) {
    T v[kDeep];
    T* to[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int x = x0 + i * 32 + lane;
      to[i] = nullptr;
      if (x >= total) continue;
      const int t = x / units, k = x - t * units, a = __ldg(acc + t);
      if (a == t) continue;
      const T* from = where(a, k);
      T* into = where(t, k);
      if (!from || !into) {
        raise_error(r.err, FP8PA_DEVERR_BLOCK_RANGE);
        continue;
      }
      v[i] = *from;
      to[i] = into;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
      if (to[i]) *to[i] = v[i];
  }
}

__global__ void __launch_bounds__(kCopyThreads) keep_kernel(const int32_t* accepted,
                                                            int max_accepted,
                                                            const int32_t* q_offsets,
                                                            const PageRows r,
                                                            const __grid_constant__ PageArrays a,
                                                            int hkv, int32_t* new_lens) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const int32_t* acc = accepted + static_cast<long>(b) * max_accepted;
  const int lo = __ldg(q_offsets + b), hi = __ldg(q_offsets + b + 1), len = __ldg(r.lens + b);
  const bool first = blockIdx.y == 0 && threadIdx.x < 32;
  const bool bad_off = lo < 0 || hi < lo, bad_len = !good_len(r, len) || (!bad_off && len < hi - lo);
  if (bad_off || bad_len) {
    if (first && lane == 0) {
      raise_error(r.err, bad_off ? FP8PA_DEVERR_Q_OFFSETS : FP8PA_DEVERR_SEQ_LEN);
      if (new_lens) new_lens[b] = len;
    }
    return;
  }
  // the path: up to the first entry that is negative, not a node, or not behind the
  // one before it
  const int n = hi - lo;
  int count = 0, last = -1;
  bool end = false;
  while (count < max_accepted && !end) {
    const int t = count + lane;
    const int x = t < max_accepted ? __ldg(acc + t) : -1;
    int before = __shfl_up_sync(0xffffffffu, x, 1);
    if (lane == 0) before = last;
    const uint32_t stop = __ballot_sync(0xffffffffu, x < 0 || x >= n || x <= before);
    if (first && stop && lane == __ffs(stop) - 1 && x >= 0) raise_error(r.err, FP8PA_DEVERR_TREE);
    end = stop != 0;
    count += end ? __ffs(stop) - 1 : 32;
    last = __shfl_sync(0xffffffffu, x, 31);
  }
  const int ctx = len - n;
  const int32_t* table = row_of(r, b);
  if (r.refs) {  // no row moves into a page that another table holds, too
    bool shared = false;
    for (int t = lane; t < count; t += 32) {
      if (__ldg(acc + t) == t) continue;
      const int page = __ldg(table + (ctx + t) / r.bs);
      shared = shared || (good_page(r, page) && __ldg(r.refs + page) > 1);
    }
    if (__any_sync(0xffffffffu, shared)) {
      if (first && lane == 0) {
        raise_error(r.err, FP8PA_DEVERR_SHARED);
        if (new_lens) new_lens[b] = len;
      }
      return;
    }
  }
  if (first && lane == 0 && new_lens) new_lens[b] = ctx + count;
  for (int w = blockIdx.y * (kCopyThreads / 32) + (threadIdx.x >> 5); w < a.n * hkv;
       w += gridDim.y * (kCopyThreads / 32)) {
    const int i = w / hkv, head = w - i * hkv;
    const int row = static_cast<int>(a.page_bytes[i] / (hkv * r.bs));
    auto run = [&](auto unit) {
      keep_rows<decltype(unit)>(r, acc, count, ctx, table, a.ptr[i], hkv, head, row);
    };
    if (row % 16 == 0) run(uint4{});
    else if (row % 4 == 0) run(uint32_t{});
    else if (row % 2 == 0) run(uint16_t{});
    else run(uint8_t{});
  }
}

// ---------------------------------------------------------------- forks
// Workspace: claim[rows] the first sound fork that wants a row; by fork, page[rows] the page
// that its last, partly filled page is copied to, kWhole where there is none, kSkip
// where the fork is not made, and size[rows] the length that it takes over (a source may
// be another fork's row: all see the rows as they were); then the free pages.  One CTA
// plans, bound by the round trips of the counts and of the rows' lengths; the copies of the
// last pages are bound by HBM (16 rows to 128: 20.8 us in all, 138 MB).
constexpr int kSkip = -2, kWhole = -1, kTail = 0;

// What fork i needs: a page of its own for the last tokens (kTail) or none (kWhole); kSkip,
// with its error raised, where its rows or its source are not as a fork needs them.
__device__ __forceinline__ int look_at_fork(const PageRows& r, int s, int d, int* size) {
  if (s < 0 || s >= r.rows || d < 0 || d >= r.rows || s == d || r.lens[d] != 0) {
    raise_error(r.err, FP8PA_DEVERR_ROW);
    return kSkip;
  }
  const int len = r.lens[s];
  *size = len;
  if (!good_len(r, len)) {
    raise_error(r.err, FP8PA_DEVERR_SEQ_LEN);
    return kSkip;
  }
  if (len % r.bs == 0) return kWhole;
  if (good_page(r, row_of(r, s)[len / r.bs])) return kTail;
  raise_error(r.err, FP8PA_DEVERR_BLOCK_RANGE);
  return kSkip;
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const int32_t* src,
                                                                 const int32_t* dst, int forks,
                                                                 const PageRows r, int32_t* ws) {
  __shared__ int s_warp[kWarps];
  griddep_wait();
  griddep_launch_dependents();
  int32_t *claim = ws, *page = claim + r.rows, *size = page + r.rows, *list = size + r.rows;
  const int tid = threadIdx.x;
  for (int i = tid; i < r.rows; i += kPlanThreads) claim[i] = forks;
  __syncthreads();
  for (int i = tid; i < forks; i += kPlanThreads) {
    const int d = __ldg(dst + i), what = look_at_fork(r, __ldg(src + i), d, size + i);
    page[i] = what;
    if (what != kSkip) atomicMin(claim + d, i);
  }
  __syncthreads();
  int want = 0;
  for (int base = 0; base < forks; base += kPlanThreads) {
    const int i = base + tid;
    int what = kSkip;
    if (i < forks) {
      what = page[i];
      if (what != kSkip && __ldcg(claim + __ldg(dst + i)) != i) {
        raise_error(r.err, FP8PA_DEVERR_ROW);
        what = kSkip;
      }
    }
    int at;
    const int total = block_scan(what == kTail ? 1 : 0, &at, s_warp);
    if (i < forks) page[i] = what == kTail ? want + at : what;
    want += total;
  }
  const int got = take_free(r, want, list, s_warp);
  __syncthreads();
  for (int i = tid; i < forks; i += kPlanThreads) {
    const int k = page[i];
    if (k < 0) continue;
    if (k >= got) raise_error(r.err, FP8PA_DEVERR_NO_BLOCK);
    page[i] = k < got ? list[k] : kSkip;
  }
}

// The rows are written by the launch over the last arrays.
__global__ void __launch_bounds__(kCopyThreads) fork_kernel(const int32_t* src, const int32_t* dst,
                                                            int forks, const PageRows r,
                                                            const int32_t* page, bool rows,
                                                            const __grid_constant__ PageArrays a) {
  griddep_wait();
  griddep_launch_dependents();
  const int32_t* size = page + r.rows;
  if (rows) {
    for (int i = blockIdx.x; i < forks; i += gridDim.x) {
      const int fresh = page[i];
      if (fresh == kSkip) continue;
      const int s = __ldg(src + i), d = __ldg(dst + i), len = size[i];
      const int n = pages_of(len, r.bs);
      const int32_t* from = row_of(r, s);
      int32_t* to = row_of(r, d);
      for (int c = threadIdx.x; c < r.max_blocks; c += kCopyThreads) {
        int p = -1;
        if (c < n) {
          p = c == n - 1 && fresh >= 0 ? fresh : from[c];
          if (good_page(r, p)) atomicAdd(r.refs + p, 1);
          else raise_error(r.err, FP8PA_DEVERR_BLOCK_RANGE);
        }
        to[c] = p;
      }
      if (threadIdx.x == 0) r.lens[d] = len;
    }
  }
  copy_pairs(a, forks, [&](int k, int* from, int* to) {
    *to = page[k];
    if (*to < 0) return false;
    *from = row_of(r, __ldg(src + k))[size[k] / r.bs];
    return true;
  });
}

// ---------------------------------------------------------------- resizing
// Workspace: the rows' new page counts (kSkip: the row is left), the prefix of the
// pages that rows grow by, then the free pages.  All rows are looked at before any
// page is given back, so that what a row may do does not depend on its neighbours'
// order.  Three launches: the first two take a thread and a CTA for each row, the last is one
// CTA, which gives out the free pages in order and is bound by its round trips.  (One CTA
// behind barriers could take all three steps of as many rows as it has threads; not tried.)
__global__ void __launch_bounds__(256) resize_check_kernel(const int32_t* new_lens,
                                                           const PageRows r, int32_t* target) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= r.rows) return;
  const int len = r.lens[i], then = new_lens[i];
  int t = kSkip;
  if (!good_len(r, len) || !good_len(r, then)) {
    raise_error(r.err, FP8PA_DEVERR_SEQ_LEN);
  } else {
    t = pages_of(then, r.bs);
    // the page that the row's next token goes to, where it holds tokens already, has to be
    // the row's own
    const int keep = min(len, then);
    if (then != len && keep % r.bs != 0) {
      const int p = row_of(r, i)[keep / r.bs];
      const bool there = good_page(r, p);
      if (!there || r.refs[p] > 1) {
        raise_error(r.err, there ? FP8PA_DEVERR_SHARED : FP8PA_DEVERR_BLOCK_RANGE);
        t = kSkip;
      }
    }
  }
  target[i] = t;
}

__global__ void __launch_bounds__(128) resize_release_kernel(const PageRows r,
                                                             const int32_t* target) {
  griddep_wait();
  griddep_launch_dependents();
  for (int i = blockIdx.x; i < r.rows; i += gridDim.x) {
    const int t = target[i];
    if (t == kSkip) continue;
    const int n = pages_of(r.lens[i], r.bs);
    int32_t* row = row_of(r, i);
    for (int c = t + threadIdx.x; c < n; c += 128) {
      const int p = row[c];
      if (good_page(r, p)) atomicSub(r.refs + p, 1);
      else raise_error(r.err, FP8PA_DEVERR_BLOCK_RANGE);
      row[c] = -1;
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) resize_grow_kernel(const int32_t* new_lens,
                                                                   const PageRows r,
                                                                   const int32_t* target,
                                                                   int32_t* prefix,
                                                                   int32_t* list) {
  __shared__ int s_warp[kWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  // more pages than the pool has are not there: the sum stops at one more than that (in 64
  // bits, as rows of 2^20 pages each pass 32 before it is looked at)
  const int most = r.num_blocks + 1;
  long long want = 0;
  for (int base = 0; base < r.rows; base += kPlanThreads) {
    const int i = base + tid;
    int n = 0;
    if (i < r.rows && target[i] != kSkip) n = max(target[i] - pages_of(r.lens[i], r.bs), 0);
    int at;
    // (a chunk's sum stays below 1024 (2^20 + 1): larger growths fit no pool of fewer pages)
    const int total = block_scan(min(n, min(most, 1 << 20)), &at, s_warp);
    if (i < r.rows) prefix[i] = static_cast<int>(min(want + at, static_cast<long long>(most)));
    want = min(want + total, static_cast<long long>(most));
  }
  if (tid == 0) prefix[r.rows] = static_cast<int>(want);
  const int got = take_free(r, static_cast<int>(want), list, s_warp);
  __syncthreads();
  // rows that got all their pages: those whose prefix ends within them
  for (int k = tid; k < got; k += kPlanThreads) {
    int lo = 0, hi = r.rows;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= k) lo = mid;
      else hi = mid;
    }
    if (prefix[lo + 1] > got) continue;
    row_of(r, lo)[pages_of(r.lens[lo], r.bs) + k - prefix[lo]] = list[k];
    r.refs[list[k]] = 1;
  }
  __syncthreads();
  for (int i = tid; i < r.rows; i += kPlanThreads) {
    if (target[i] == kSkip) continue;
    if (target[i] > pages_of(r.lens[i], r.bs) && prefix[i + 1] > got)
      raise_error(r.err, FP8PA_DEVERR_NO_BLOCK);
    else
      r.lens[i] = new_lens[i];
  }
}

// ---------------------------------------------------------------- compacting
// Workspace: the number of moves, then low[k] and high[k]: the k-th free page below the
// number of live ones, and the k-th live page at or above it, which moves there.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PageRows r,
                                                                    int32_t* page_map,
                                                                    int32_t* ws) {
  __shared__ int s_warp[kWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  int32_t *low = ws + 1, *high = low + r.num_blocks / 2;
  int n = 0;
  for (long long from = 0; from < r.num_blocks; from += kStretch) {
    FreeBits f;
    load_free(r, static_cast<int>(from), f);
#pragma unroll
    for (int i = 0; i < kSpan; ++i) n += __popc(f.w[i]);
  }
  int at;
  const int live = r.num_blocks - block_scan(lane == 0 ? n : 0, &at, s_warp);
  // free pages below `live`, and live pages from there on, are as many
  int lows = 0, highs = 0;
  for (long long from = 0; from < r.num_blocks; from += kStretch) {
    FreeBits f;
    load_free(r, static_cast<int>(from), f);
    int nl = 0, nh = 0;
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
      const int p0 = f.base + i * 32;
      const int below = min(max(live - p0, 0), 32), held = min(max(r.num_blocks - p0, 0), 32);
      const uint32_t lo = below == 32 ? 0xFFFFFFFFu : (1u << below) - 1u;
      const uint32_t in = held == 32 ? 0xFFFFFFFFu : (1u << held) - 1u;
      nl += __popc(f.w[i] & lo);
      nh += __popc(~f.w[i] & in & ~lo);
    }
    int al, ah;
    const int tl = block_scan(lane == 0 ? nl : 0, &al, s_warp);
    const int th = block_scan(lane == 0 ? nh : 0, &ah, s_warp);
    al = lows + __shfl_sync(0xffffffffu, al, 0);
    ah = highs + __shfl_sync(0xffffffffu, ah, 0);
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
      const int p = f.base + i * 32 + lane;
      const bool in = p < r.num_blocks, free = f.w[i] >> lane & 1u;
      const uint32_t ml = __ballot_sync(0xffffffffu, in && free && p < live);
      const uint32_t mh = __ballot_sync(0xffffffffu, in && !free && p >= live);
      const uint32_t before = (1u << lane) - 1u;
      if (ml >> lane & 1u) low[al + __popc(ml & before)] = p;
      if (mh >> lane & 1u) high[ah + __popc(mh & before)] = p;
      if (in) page_map[p] = free ? -1 : p;
      al += __popc(ml);
      ah += __popc(mh);
    }
    lows += tl;
    highs += th;
  }
  __syncthreads();
  if (tid == 0) ws[0] = highs;
  for (int k = tid; k < highs; k += kPlanThreads) page_map[high[k]] = low[k];
}

__global__ void __launch_bounds__(kCopyThreads) compact_kernel(const PageRows r,
                                                               const int32_t* page_map,
                                                               const int32_t* ws, bool rows,
                                                               const __grid_constant__
                                                               PageArrays a) {
  griddep_wait();
  griddep_launch_dependents();
  const int moves = ws[0];
  const int32_t *low = ws + 1, *high = low + r.num_blocks / 2;
  if (rows) {
    for (int i = blockIdx.x; i < r.rows; i += gridDim.x) {
      const int len = r.lens[i];
      if (!good_len(r, len)) {
        raise_error(r.err, FP8PA_DEVERR_SEQ_LEN);
        continue;
      }
      int32_t* row = row_of(r, i);
      for (int c = threadIdx.x; c < pages_of(len, r.bs); c += kCopyThreads) {
        const int p = row[c];
        const int to = good_page(r, p) ? page_map[p] : -1;
        if (to < 0) raise_error(r.err, FP8PA_DEVERR_BLOCK_RANGE);
        else if (to != p) row[c] = to;
      }
    }
    for (int k = blockIdx.x * kCopyThreads + threadIdx.x; k < moves;
         k += gridDim.x * kCopyThreads) {
      r.refs[low[k]] = r.refs[high[k]];
      r.refs[high[k]] = 0;
    }
  }
  copy_pairs(a, moves, [&](int k, int* from, int* to) {
    *from = high[k];
    *to = low[k];
    return true;
  });
}

// ---------------------------------------------------------------- host
template <class... P, class... A>
cudaError_t launch(void (*fn)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

// Arrays [at, at + kMaxArrays) of a cache.
PageArrays some_arrays(void* const* pages, const long long* page_bytes, int arrays, int at) {
  PageArrays a;
  a.n = arrays - at < kMaxArrays ? arrays - at : kMaxArrays;
  a.first[0] = 0;
  for (int i = 0; i < a.n; ++i) {
    a.ptr[i] = static_cast<uint8_t*>(pages[at + i]);
    a.page_bytes[i] = static_cast<uint32_t>(page_bytes[at + i]);
    a.first[i + 1] = a.first[i] + (a.page_bytes[i] + kChunk - 1) / kChunk;
  }
  return a;
}

// One launch per kMaxArrays arrays, and one at least; go(arrays, whether it is the last).
template <class Go>
cudaError_t over_arrays(void* const* pages, const long long* page_bytes, int arrays, Go go) {
  int at = 0;
  do {
    const PageArrays a = some_arrays(pages, page_bytes, arrays, at);
    at += kMaxArrays;
    const cudaError_t e = go(a, at >= arrays);
    if (e != cudaSuccess) return e;
  } while (at < arrays);
  return cudaSuccess;
}

// CTAs of a copying kernel: eight an SM, which is what its registers and threads allow.
cudaError_t copy_grid(dim3* grid) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) *grid = dim3(static_cast<unsigned>(sm_count(dev)) * 8);
  return e;
}

}  // namespace

cudaError_t launch_keep_accepted(const int32_t* accepted, int max_accepted,
                                 const int32_t* q_offsets, const PageRows& r, void* const* pages,
                                 const long long* page_bytes, int arrays, int hkv,
                                 int32_t* new_lens, cudaStream_t stream) {
  return over_arrays(pages, page_bytes, arrays, [&](const PageArrays& a, bool last) {
    const long long warps = static_cast<long long>(a.n) * hkv;
    const long long y = (warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    const dim3 grid(static_cast<unsigned>(r.rows),
                    static_cast<unsigned>(y < 1 ? 1 : (y > 1024 ? 1024 : y)));
    return launch(keep_kernel, grid, kCopyThreads, stream, accepted, max_accepted, q_offsets, r, a,
                  hkv, last ? new_lens : nullptr);
  });
}

cudaError_t launch_fork(const int32_t* src, const int32_t* dst, int forks, const PageRows& r,
                        void* const* pages, const long long* page_bytes, int arrays,
                        int32_t* workspace, cudaStream_t stream) {
  dim3 grid;
  cudaError_t e = copy_grid(&grid);
  if (e != cudaSuccess) return e;
  e = launch(fork_plan_kernel, dim3(1), kPlanThreads, stream, src, dst, forks, r, workspace);
  if (e != cudaSuccess) return e;
  return over_arrays(pages, page_bytes, arrays, [&](const PageArrays& a, bool last) {
    return launch(fork_kernel, grid, kCopyThreads, stream, src, dst, forks, r,
                  workspace + r.rows, last, a);
  });
}

cudaError_t launch_resize(const int32_t* new_lens, const PageRows& r, int32_t* workspace,
                          cudaStream_t stream) {
  int32_t *target = workspace, *prefix = target + r.rows, *list = prefix + r.rows + 1;
  cudaError_t e = launch(resize_check_kernel, dim3(static_cast<unsigned>((r.rows + 255) / 256)),
                         256, stream, new_lens, r, target);
  if (e != cudaSuccess) return e;
  e = launch(resize_release_kernel, dim3(static_cast<unsigned>(r.rows < 4096 ? r.rows : 4096)),
             128, stream, r, target);
  if (e != cudaSuccess) return e;
  return launch(resize_grow_kernel, dim3(1), kPlanThreads, stream, new_lens, r, target, prefix,
                list);
}

cudaError_t launch_compact(const PageRows& r, void* const* pages, const long long* page_bytes,
                           int arrays, int32_t* page_map, int32_t* workspace,
                           cudaStream_t stream) {
  dim3 grid;
  cudaError_t e = copy_grid(&grid);
  if (e != cudaSuccess) return e;
  e = launch(compact_plan_kernel, dim3(1), kPlanThreads, stream, r, page_map, workspace);
  if (e != cudaSuccess) return e;
  return over_arrays(pages, page_bytes, arrays, [&](const PageArrays& a, bool last) {
    return launch(compact_kernel, grid, kCopyThreads, stream, r, page_map, workspace, last, a);
  });
}

}  // namespace fp8pa
