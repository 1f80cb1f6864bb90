// prefill.cu -- attention of ragged query chunks over the paged cache, causal
// with score modifiers, on the fifth-generation tensor cores.
//
//   z_j = sm_scale q_i . k^_j;  z_j = cap tanh(z_j / cap);  z_j -= slope |i - j|
//   out_i = sum_j softmax(z)_j v^_j over j < prefix or i - window < j <= i
//
// Rows.  The G heads that share a KV head see the same keys, so the (query,
// head) pairs of one request and KV head are flattened into rows r = query * G
// + head; a CTA takes a block of 256 rows as two tiles of M = 128, one TMEM
// lane per row, and walks the 128-token tiles of its visible context:
//   S_t = Q_t K^T (A, B in shared memory), P_t = softmax part (TMEM -> registers
//   -> TMEM), O_t += P_t V (A = P_t in TMEM, B in shared memory).
// Each K or V code is read and converted once for 256 rows.
//
// Work is the flat list of (row block, KV head, token tile) units.  A planner
// kernel counts the tiles that each row block can see and cuts the list into
// one contiguous range per SM; where a cut falls inside an item (it is moved
// to an item's edge when that is a few tiles away) the pieces leave partial
// results that a merge kernel folds with the log-sum-exp rule.  A long chunk
// and a few rows over a long context are balanced alike.
//
// Numerics.  Codes become f16 exactly (E4M3 scaled by 2^-8).  q is exact in
// f16 after a power-of-two normaliser per row (CHANNEL_STATIC folds the K
// scales into it and rounds once, 2^-11).  K scales multiply the fp32 scores;
// V scales go into P, which enters the second product as f16 (2^-11).  The
// running reference of a row is a bound of max(z + log2 v_scale), so P stays
// inside f16 whatever the scales; it moves only when passed by 2^kTau, which
// is exact, as sums and O carry the same reference.
//
// Roles (24 warps): 0-7 and 8-15 the softmax of row tiles 0 and 1, two threads
// per row, each with 64 of a tile's 128 tokens (four warps per scheduler hide
// one another's waits; the two agree on the row's reference through shared
// memory); 16-22 convert codes into shared memory, 23 issues the MMAs (one
// thread).  While the tensor cores work on one row tile, the other's softmax
// runs.  Every wait is bounded.
#include <float.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "score_mods.cuh"
#include "tc.cuh"

namespace fp8pa {

namespace {

constexpr int kRows = 256;   // rows of a block: two tiles of 128
constexpr int kT = 128;      // tokens per tile
constexpr int kHalf = 64;    // ... of which a softmax thread has half
constexpr int kThreads = 768;
constexpr int kAhead = 3;    // jobs that a converting warp asks L2 for ahead
constexpr int kConvWarp = 16, kConvWarps = 7, kIssueWarp = 23;
constexpr int kSnap = 4;     // a cut this near an item's edge moves to it
constexpr float kShift = 12.f;  // P = 2^(z - ref + 12): at most 2^15 with the lazy bound
constexpr float kTau = 3.f;     // the reference may lag by 2^3
constexpr float kNegBig = -1e30f;

// ---------------------------------------------------------------- plan
// Workspace: header, block prefix of the requests, then per row block its
// request and the prefix of its tiles, then the ranges' first units, then the
// partial pieces.
struct PlanView {
  int* head;     // [0] units, [1] units per range (before cuts move)
  int* rbase;    // [batch + 1] first row block of a request
  int* rb_b;     // [blocks] request of a row block
  int* rb_pre;   // [blocks + 1] tiles before a row block (of one KV head)
  int* start;    // [ranges + 1] first unit of a range
  int* item;     // [ranges + 1] the item that holds it
  float2* ml;    // [2 * ranges][kRows] reference and sum of a piece
  float* o;      // [2 * ranges][kRows][d]
  int blocks;    // bound of the row blocks
};

__host__ __device__ inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline int block_bound(int total_q, int batch, int G) {
  return static_cast<int>((static_cast<long long>(total_q) * G + kRows - 1) / kRows) + batch;
}

inline size_t plan_layout(char* ws, int total_q, int batch, int G, int d, int ranges,
                          PlanView* v) {
  const int nb = block_bound(total_q, batch, G);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = ws + at;
    at += align256(bytes);
    return p;
  };
  PlanView t;
  t.head = reinterpret_cast<int*>(take(16));
  t.rbase = reinterpret_cast<int*>(take(sizeof(int) * (batch + 1)));
  t.rb_b = reinterpret_cast<int*>(take(sizeof(int) * nb));
  t.rb_pre = reinterpret_cast<int*>(take(sizeof(int) * (nb + 1)));
  t.start = reinterpret_cast<int*>(take(sizeof(int) * (ranges + 1)));
  t.item = reinterpret_cast<int*>(take(sizeof(int) * (ranges + 1)));
  t.ml = reinterpret_cast<float2*>(take(sizeof(float2) * 2 * ranges * kRows));
  t.o = reinterpret_cast<float*>(take(sizeof(float) * 2 * ranges * kRows * d));
  t.blocks = nb;
  if (v) *v = t;
  return at;
}

// A request's chunk and its visible extent.
struct Chunk {
  int qlo, n, L, pre;
};
__device__ __forceinline__ Chunk load_chunk(const PrefillArgs& a, int b, bool* bad_off,
                                            bool* bad_len) {
  Chunk c;
  const int lo = __ldg(a.q_offsets + b), hi = __ldg(a.q_offsets + b + 1);
  *bad_off = lo < 0 || hi < lo || hi > a.total_q;
  c.qlo = lo;
  c.n = *bad_off ? 0 : hi - lo;
  const int cap = a.max_blocks * a.bs;
  const int L = __ldg(a.seq_lens + b);
  *bad_len = L < 0 || L > cap || L < c.n;
  c.L = min(max(L, 0), cap);
  const ScoreMods m{a.prefix_lens, nullptr, 0.f, a.window};
  c.pre = prefix_len(m, b, c.L);
  return c;
}

// The token tiles of row block t of a chunk: tiles [0, np) of the prefix, then
// from tile np + skip on; `count` in all (at least one, so that rows that see
// nothing are written).
struct Tiles {
  int np, skip, count;
};
__device__ __forceinline__ Tiles block_tiles(const Chunk& c, int window, int G, int t) {
  const int q0 = t * kRows / G, q1 = min((t * kRows + kRows - 1) / G, c.n - 1);
  const int p0 = c.L - c.n + q0, p1 = c.L - c.n + q1;
  const int wf = window > 0 ? max(p0 - window + 1, 0) : 0;
  Tiles r;
  r.np = (c.pre + kT - 1) / kT;
  r.skip = max(wf / kT - r.np, 0);
  const int last = (max(max(p1 + 1, c.pre), 0) + kT - 1) / kT;
  r.count = max(last - r.skip, 1);
  return r;
}

constexpr int kPlanThreads = 1024;

// Exclusive scan of one int per thread over the CTA; returns the total.
__device__ __forceinline__ int block_scan(int x, int* excl, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *excl = v - x + (warp ? s_warp[warp - 1] : 0);
  const int total = s_warp[kPlanThreads / 32 - 1];
  __syncthreads();
  return total;
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

__global__ void __launch_bounds__(kPlanThreads) prefill_plan_kernel(const PrefillArgs a,
                                                                    const PlanView v, int ranges) {
  __shared__ int s_warp[kPlanThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  int carry = 0;
  for (int base = 0; base < a.batch; base += kPlanThreads) {
    const int b = base + tid;
    int n = 0;
    if (b < a.batch) {
      bool bo, bl;
      const Chunk c = load_chunk(a, b, &bo, &bl);
      if (bo) raise_error(a.err, FP8PA_DEVERR_Q_OFFSETS);
      if (bl) raise_error(a.err, FP8PA_DEVERR_SEQ_LEN);
      // overlapping or repeated offsets cannot add blocks beyond the bound
      n = static_cast<int>((static_cast<long long>(c.n) * a.G + kRows - 1) / kRows);
    }
    int ex;
    const int total = block_scan(n, &ex, s_warp);
    if (b < a.batch) v.rbase[b] = min(carry + ex, v.blocks);
    carry = min(carry + total, v.blocks);
  }
  if (tid == 0) v.rbase[a.batch] = carry;
  __syncthreads();
  const int blocks = carry;
  carry = 0;
  for (int base = 0; base < blocks; base += kPlanThreads) {
    const int i = base + tid;
    int n = 0;
    if (i < blocks) {
      const int b = last_le(v.rbase, a.batch, i);
      bool bo, bl;
      const Chunk c = load_chunk(a, b, &bo, &bl);
      n = block_tiles(c, a.window, a.G, i - v.rbase[b]).count;
      v.rb_b[i] = b;
    }
    int ex;
    const int total = block_scan(n, &ex, s_warp);
    if (i < blocks) v.rb_pre[i] = carry + ex;
    carry += total;
  }
  if (tid == 0) v.rb_pre[blocks] = carry;
  __syncthreads();
  const int U = carry * a.hkv;
  const int upw = max(1, (U + ranges - 1) / ranges);
  if (tid == 0) {
    v.head[0] = U;
    v.head[1] = upw;
  }
  for (int w = tid; w <= ranges; w += kPlanThreads) {
    const long long want = static_cast<long long>(w) * upw;
    int u = want < U ? static_cast<int>(want) : U, it = blocks * a.hkv;
    if (u < U) {
      const int rb = last_le(v.rb_pre, blocks, u / a.hkv);
      const int pre = v.rb_pre[rb], c = v.rb_pre[rb + 1] - pre;
      const int h = (u - pre * a.hkv) / c, f = pre * a.hkv + h * c;
      it = rb * a.hkv + h;
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

// ---------------------------------------------------------------- shared memory
template <int D>
struct Smem {
  static constexpr int kTile = kT * D * 2;  // a 128-row f16 tile
  static constexpr int kQ = 0;              // two row tiles
  static constexpr int kK = 2 * kTile;      // two stages
  static constexpr int kV = 4 * kTile;      // two stages
  static constexpr int kScale = 6 * kTile;  // four stages of [K scales][V scales] f32
  static constexpr int kInfo = kScale + 4 * 2 * kT * 4;  // four stages of StageInfo
  static constexpr int kXch = kInfo + 4 * 64;  // [parity][warp of softmax][lane] f32
  static constexpr int kBars = kXch + 2 * 16 * 32 * 4;
  static constexpr int kMisc = kBars + 320;  // TMEM base, abort flag
  static constexpr int kBytes = kMisc + 16;
};
struct StageInfo {
  uint32_t valid[4];  // tokens whose page exists
  float vmax[4];      // largest V scale of each 32 tokens
};

// Barriers and the arrivals that complete a phase.  Q and P: the eight softmax
// warps of the row tile; scales: the eight conversion jobs of the tile; K and V
// full: four jobs; X (t * 4 + lane quarter): the two softmax warps of the same
// rows; the others: a commit of the tensor cores.
enum { kBarQ = 0, kBarP = 2, kBarScale = 4, kBarKFull = 8, kBarVFull = 10, kBarX = 12,
       kBarKFree = 20, kBarVFree = 22, kBarS = 24, kBarO = 26, kBarDrain = 28, kNumBars = 29 };

// ---------------------------------------------------------------- conversions
// 16 codes -> 16 f16 (two 16-byte core-matrix rows), exactly.
template <int FMT>
__device__ __forceinline__ void codes16_to_f16(const uint4& c, uint4& lo, uint4& hi) {
  codes4_to_f16x2x2<FMT>(c.x, lo.x, lo.y);
  codes4_to_f16x2x2<FMT>(c.y, lo.z, lo.w);
  codes4_to_f16x2x2<FMT>(c.z, hi.x, hi.y);
  codes4_to_f16x2x2<FMT>(c.w, hi.z, hi.w);
}

// Whether any of 16 codes is an infinity or a NaN.
template <int FMT>
__device__ __forceinline__ bool codes_nonfinite(const uint4& c) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (FMT == FP8PA_E4M3) bad |= __vcmpeq4(w[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    if constexpr (FMT == FP8PA_E5M2) bad |= __vcmpeq4(w[i] & 0x7C7C7C7Cu, 0x7C7C7C7Cu);
  }
  return bad != 0;
}

__device__ __forceinline__ uint4 hmul8(const uint4& a, uint32_t f) {
  auto m = [&](uint32_t x) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x),
                              *reinterpret_cast<const __half2*>(&f));
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  return make_uint4(m(a.x), m(a.y), m(a.z), m(a.w));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// Registers that a tcgen05.ld filled: what uses them stays behind the
// tcgen05.wait::ld before this.
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[16]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// A row's bound of z + log2(V scale) from the largest of each (vmax 0: none).
__device__ __forceinline__ float bound_of(float zmax, float vmax) {
  return zmax + static_cast<float>(min(max(exp_above(vmax), -60), 120));
}

// D[tmem] (+)= A[tmem] * B[smem], one thread.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                              bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// The largest of eight bytes.
__device__ __forceinline__ uint32_t max_byte(const uint32_t (&w)[2]) {
  uint32_t m = __vmaxu4(w[0], w[1]);
  m = __vmaxu4(m, m >> 16);
  return max(m & 0xFFu, (m >> 8) & 0xFFu);
}

// Bits t of a 32-token word at token t0 with lo <= t0 + t < hi.
__device__ __forceinline__ uint32_t word_bits(int t0, int lo, int hi) {
  const int a = min(max(lo - t0, 0), 32), b = min(max(hi - t0, 0), 32);
  const uint32_t below_b = b == 32 ? 0xFFFFFFFFu : (1u << b) - 1u;
  const uint32_t below_a = a == 32 ? 0xFFFFFFFFu : (1u << a) - 1u;
  return below_b & ~below_a;
}

// One item of a CTA's range: a row block of a request for one KV head, tiles
// [t0, t1) of its list.
struct Item {
  int b, kvh, row0, rows;  // first row within the request, rows of the block
  Chunk c;
  Tiles tl{0, 0, 0};
  int t0, t1;
};

// Out of line: every role calls it once per item, and the roles' loops have to
// share the instruction caches.
__device__ __noinline__ Item load_item(const PrefillArgs& a, const PlanView& v, int it, int u,
                                       int u1) {
  Item r;
  const int rb = it / a.hkv;
  r.kvh = it - rb * a.hkv;
  r.b = v.rb_b[rb];
  const int pre = v.rb_pre[rb], cnt = v.rb_pre[rb + 1] - pre;
  const int f = pre * a.hkv + r.kvh * cnt;
  bool x, y;
  r.c = load_chunk(a, r.b, &x, &y);
  const int t = rb - v.rbase[r.b];
  r.row0 = t * kRows;
  r.rows = min(kRows, r.c.n * a.G - r.row0);
  r.tl = block_tiles(r.c, a.window, a.G, t);
  r.t0 = u - f;
  r.t1 = min(r.tl.count, u1 - f);
  return r;
}

__device__ __forceinline__ int tile_token(const Item& it, int k) {
  return (k < it.tl.np ? k : k + it.tl.skip) * kT;
}

// ---------------------------------------------------------------- conversion
// The work of one converting warp.  A tile has eight jobs, 32 tokens of K or V
// each (part 0-3: K, 4-7: V), dealt round robin over the converting warps.  A
// lane holds row r8 of four 8-row groups and, of each, the 16-byte chunks c4
// (and c4 + 4): loads take 64 contiguous bytes of 8 rows, stores the 8 rows of a
// core matrix, free of bank conflicts.  A job's codes and scales are loaded as
// soon as the job before it is stored, its block ids one job earlier; kAhead jobs
// earlier it is asked for into L2, which is what keeps HBM busy where a chunk
// has few rows.
template <int D, int FMT>
__device__ __forceinline__ void convert_tiles(const PrefillArgs& a, const PlanView& pv,
                                              uint8_t* sm, int* abort_flag, int it, int u, int u1,
                                              int first, int lane) {
  using SM = Smem<D>;
  constexpr int H = D / 64;  // 16-byte chunks of a row per lane
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SM::kBars);
  StageInfo* infos = reinterpret_cast<StageInfo*>(sm + SM::kInfo);
  const int r8 = lane & 7, c4 = lane >> 3;
  const int lgbs = 31 - __clz(a.bs);  // block sizes are powers of two
  const bool mx = FMT != FP8PA_INT8 && a.mode == FP8PA_SCALE_MX_BLOCK;
  const int nbx = mx ? D / a.gs : 0;

  // the open item: tiles left of it, its block table, the tokens that some row
  // sees ([lo, hi) and [0, pre); others are neither looked up nor read) and
  // those that every row sees
  Tiles tl{0, 0, 0};
  int k = 0, n = 0, kt = 0, kvh = 0, lo = 0, hi = 0, pre = 0, all_lo = 0, all_hi = 0;
  const int32_t* table = nullptr;
  auto token_of = [&](int i) { return (i < tl.np ? i : i + tl.skip) * kT; };
  auto wanted = [&](int j) { return (j < hi && j >= lo) || j < pre; };
  // block ids of a job's two 16-token halves (a half lies in one block); -1
  // where no row sees any of its tokens
  auto load_ids = [&](int i, int part, int (&id)[2]) {
    const int j = token_of(i) + (part & 3) * 32;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int t = j + 16 * x;
      id[x] = (t < hi && t + 16 > lo) || t < pre
                  ? __ldg(table + static_cast<int>(static_cast<uint32_t>(t) >> lgbs))
                  : -1;
    }
  };
  auto row_of = [&](int blk, int t) {
    return (static_cast<uint32_t>(blk) * a.hkv + kvh) * a.bs + (t & (a.bs - 1));
  };

  int ids[2], part = first;  // of this job
  bool have = false;         // ids are loaded
  int pf_blk = -1, pf_t = 0;  // a half-job to ask for into L2
  bool pf_v = false;
  for (uint32_t g = 0;;) {   // g: the job's tile, counted over the range
    while (k >= n) {
      if (u >= u1) return;
      const Item im = load_item(a, pv, it, u, u1);
      ++it;
      pf_blk = -1;
      k -= n;
      n = im.t1 - im.t0;
      kt = im.t0;
      u += n;
      tl = im.tl;
      kvh = im.kvh;
      pre = im.c.pre;
      table = a.block_tables + static_cast<long>(im.b) * a.max_blocks;
      const int pA = im.c.L - im.c.n + im.row0 / a.G;
      const int pB = im.c.L - im.c.n + (im.row0 + im.rows - 1) / a.G;
      lo = a.window > 0 ? max(pA - a.window + 1, 0) : 0;
      hi = pB + 1;
      all_lo = a.window > 0 ? max(pB - a.window + 1, 0) : 0;
      all_hi = pA + 1;
    }
    if (!have) load_ids(kt + k, part, ids);
    const bool V = part >= 4;
    const int dw = part & 3;
    const uint8_t* cache = V ? a.v_cache : a.k_cache;
    const float* gscale = V ? a.v_scale : a.k_scale;
    const int j0 = token_of(kt + k), j = j0 + dw * 32;
    const bool whole = (j0 >= all_lo && j0 + kT <= all_hi) || j0 + kT <= pre;
    uint4 buf[4][H];
    uint32_t okm = 0;  // groups whose row is wanted and exists
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int blk = ids[x >> 1], t = j + x * 8 + r8;
      const bool ok = wanted(t) && blk >= 0 && blk < a.num_blocks;
      if (ok) okm |= 1u << x;
      const uint4* src = reinterpret_cast<const uint4*>(
                             cache + static_cast<size_t>(ok ? row_of(blk, t) : 0u) * D) + c4;
#pragma unroll
      for (int h = 0; h < H; ++h)
        buf[x][h] = ok ? __ldg(src + h * 4) : make_uint4(0u, 0u, 0u, 0u);
    }
    float sc = 1.f;  // scale of token 32 dw + lane
    bool sok;
    uint32_t below[H];  // MX: exponents of the lane's chunks below their rows' largest, by group
    {
      const int blk = lane < 16 ? ids[0] : ids[1], t = j + lane;
      sok = wanted(t) && blk >= 0 && blk < a.num_blocks;
      if (wanted(t) && !sok) raise_error(a.err, FP8PA_DEVERR_BLOCK_RANGE);
      const size_t rw = sok ? row_of(blk, t) : 0u;
      if (a.mode == FP8PA_SCALE_TOKEN_HEAD) {
        if (sok) sc = __ldg(gscale + rw);
      } else if (a.mode == FP8PA_SCALE_SEGMENT) {
        if (sok) sc = __ldg(gscale + static_cast<long>(blk) * a.hp + kvh);
      } else if (mx) {
        // 2, 4 or 8 bytes a row; absent ones read as zero
        auto row_bytes = [&](size_t row, uint32_t (&w)[2]) {
          const uint8_t* e = reinterpret_cast<const uint8_t*>(gscale) + row * nbx;
          w[1] = nbx == 8 ? __ldg(reinterpret_cast<const uint32_t*>(e) + 1) : 0u;
          w[0] = nbx == 2 ? __ldg(reinterpret_cast<const uint16_t*>(e))
                          : __ldg(reinterpret_cast<const uint32_t*>(e));
        };
#pragma unroll
        for (int h = 0; h < H; ++h) below[h] = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (!((okm >> x) & 1)) continue;
          uint32_t w[2];
          row_bytes(row_of(ids[x >> 1], j + x * 8 + r8), w);
          const uint32_t em = max_byte(w);
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const int b = (h * 4 + c4) * 16 / a.gs;
            below[h] |= (em - (((b & 4 ? w[1] : w[0]) >> (8 * (b & 3))) & 0xFF)) << (8 * x);
          }
        }
        if (sok) {
          uint32_t w[2];
          row_bytes(rw, w);
          sc = exp2i(static_cast<int>(max_byte(w)) - 127);
        }
      }
    }
    // ---- the job behind this one
    int nk = k, npart = part + kConvWarps;
    if (npart >= 8) {
      npart -= 8;
      ++nk;
    }
    have = nk < n;
    if (have) load_ids(kt + nk, npart, ids);

    // ---- a job further ahead is asked for into L2 (its block id was loaded one
    // job ago), and the next one's block id; lane x < 2 for half x
    if (pf_blk >= 0 && pf_blk < a.num_blocks) {
      const size_t row = row_of(pf_blk, pf_t);
      prefetch_l2((pf_v ? a.v_cache : a.k_cache) + row * D, 16 * D);
      if (a.mode == FP8PA_SCALE_TOKEN_HEAD) prefetch_l2((pf_v ? a.v_scale : a.k_scale) + row, 64);
      else if (mx)
        prefetch_l2(reinterpret_cast<const uint8_t*>(pf_v ? a.v_scale : a.k_scale) + row * nbx,
                    16 * nbx);
    }
    pf_blk = -1;
    if (lane < 2) {
      const int ahead = part + kAhead * kConvWarps, ak = k + (ahead >> 3);
      if (ak < n) {
        pf_v = (ahead & 7) >= 4;
        pf_t = token_of(kt + ak) + (ahead & 3) * 32 + lane * 16;
        if ((pf_t < hi && pf_t + 16 > lo) || pf_t < pre)
          pf_blk = __ldg(table + static_cast<int>(static_cast<uint32_t>(pf_t) >> lgbs));
      }
    }

    const uint32_t st = g & 1, s4 = g & 3;
    float* ss = reinterpret_cast<float*>(sm + SM::kScale) + s4 * 2 * kT + (V ? kT : 0) + dw * 32;
    // The stage's last reader was the MMA of tile g - 2; the scale stage's the
    // softmax of tile g - 4, whose P was waited for before that MMA.
    if (g >= 2 && !__all_sync(0xffffffffu,
                              tc_wait(bars + (V ? kBarVFree : kBarKFree) + st,
                                      ((g >> 1) - 1) & 1, abort_flag, a.err)))
      return;
    ss[lane] = sc;
    const uint32_t valid = __ballot_sync(0xffffffffu, sok);
    const float vmax = warp_max_f32(sok && sc <= FLT_MAX ? sc : 0.f);
    if (lane == 0) {
      if (V) infos[s4].vmax[dw] = vmax;
      else infos[s4].valid[dw] = valid;
    }
    __syncwarp();
    // Groups to keep; the others become zero.  In a tile that some row does
    // not see whole, a non-finite V code would reach rows that mask its token
    // (0 * NaN): it is zeroed and its token's scale made NaN, for the rows that
    // do see it.
    uint32_t keep = okm;
    if (FMT != FP8PA_INT8 && V && !whole) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        bool nf = false;
#pragma unroll
        for (int h = 0; h < H; ++h) nf = nf || codes_nonfinite<FMT>(buf[x][h]);
        uint32_t any = nf ? 1u : 0u;
        any |= __shfl_xor_sync(0xffffffffu, any, 8);
        any |= __shfl_xor_sync(0xffffffffu, any, 16);
        if (any && ((okm >> x) & 1)) {
          keep &= ~(1u << x);
          if (c4 == 0) ss[x * 8 + r8] = __int_as_float(0x7FC00000);
        }
      }
    }
    // K: core matrices (8 tokens x 8 dims) 128 bytes apart along the tokens,
    // 2048 along the dims; V: D * 16 along the tokens, 128 along the dims
    uint8_t* dst = sm + (V ? SM::kV : SM::kK) + st * SM::kTile + r8 * 16 +
                   (V ? dw * (D * 64) + c4 * 256 : dw * 512 + c4 * 4096);
    const int kG = V ? D * 16 : 128, kC = V ? 4 * 256 : 4 * 4096, kH = V ? 128 : 2048;
    auto store = [&](int x, int h, const uint4& p, const uint4& q) {
      *reinterpret_cast<uint4*>(dst + x * kG + h * kC) = p;
      *reinterpret_cast<uint4*>(dst + x * kG + h * kC + kH) = q;
    };
    if (keep == 0xFu && !mx) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          uint4 p, q;
          codes16_to_f16<FMT>(buf[x][h], p, q);
          store(x, h, p, q);
        }
      }
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool kept = (keep >> x) & 1;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          uint4 p, q;
          codes16_to_f16<FMT>(buf[x][h], p, q);
          if (mx) {
            // the block's power of two relative to the row's largest
            const int e = (below[h] >> (8 * x)) & 0xFF;
            const float f = __int_as_float((127 - min(e, 126)) << 23);
            const __half2 f2 = __floats2half2_rn(f, f);
            const uint32_t fw = *reinterpret_cast<const uint32_t*>(&f2);
            p = hmul8(p, fw);
            q = hmul8(q, fw);
          }
          if (!kept) p = q = make_uint4(0u, 0u, 0u, 0u);
          store(x, h, p, q);
        }
      }
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(bars + kBarScale + s4);
      mbar_arrive(bars + (V ? kBarVFull : kBarKFull) + st);
    }
    g += nk - k;
    k = nk;
    part = npart;
  }
}

// ---------------------------------------------------------------- kernel
// VAR: 0 no score modifier but the masks, 1 distance bias, 2 capped scores
// (with or without a bias).
template <int D, int FMT, int VAR>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const PrefillArgs a,
                                                              const PlanView pv) {
  using SM = Smem<D>;
  // used as it stands, so that its accesses stay in the shared space
  extern __shared__ __align__(128) uint8_t sm[];
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(sm + SM::kMisc);
  int& s_abort = *reinterpret_cast<int*>(sm + SM::kMisc + 4);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SM::kBars);
  float* scales = reinterpret_cast<float*>(sm + SM::kScale);
  StageInfo* infos = reinterpret_cast<StageInfo*>(sm + SM::kInfo);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  griddep_wait();
  griddep_launch_dependents();
  const int u0 = pv.start[blockIdx.x], u1 = pv.start[blockIdx.x + 1];
  if (u0 >= u1) return;
  const int it0 = pv.item[blockIdx.x];

  if (warp == kIssueWarp) tmem_alloc(&s_tmem, 512);
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bars + i, i >= kBarKFree ? 1 : (i >= kBarX ? 2 : (i >= kBarKFull ? 4 : 8)));
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_relinquish();
  const uint32_t tmem = s_tmem;
  int* abort_flag = &s_abort;
  auto wait = [&](int bar, uint32_t parity) {
    return tc_wait(bars + bar, parity, abort_flag, a.err);
  };
  // a wait of a whole warp: one answer for all lanes
  auto wait_warp = [&](int bar, uint32_t parity) {
    return __all_sync(0xffffffffu, tc_wait(bars + bar, parity, abort_flag, a.err)) != 0;
  };

  if (warp == kIssueWarp) {
    // ================================================= MMA issuer
    // S_t of tile k + 1 goes where P_t of tile k was: it is issued behind the
    // P V that reads it, and the tensor cores work through one thread's MMAs in
    // the order of their issue.
    if (lane == 0) {
      const uint32_t idesc_s = tc_idesc(0, 0, 0, 0, 128, kT);  // f16, both K-major
      const uint32_t idesc_o = tc_idesc(0, 0, 0, 1, 128, D);   // A in TMEM, B MN-major
      const uint32_t base = smem_u32(sm);
      const uint64_t dq0 = tc_desc(base + SM::kQ, 2048, 128, 0);
      const uint64_t dk0 = tc_desc(base + SM::kK, 2048, 128, 0);
      const uint64_t dv0 = tc_desc(base + SM::kV, D * 16, 128, 0);
      constexpr uint32_t kNext = SM::kTile >> 4;  // the other row tile or stage
      auto mma_s = [&](int t, uint32_t st) {  // S_t = Q_t K^T
        const uint64_t dq = dq0 + t * kNext, dk = dk0 + st * kNext;
        const uint32_t d = tmem + t * kT;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma_f16(d, dq + k * (4096 >> 4), dk + k * (4096 >> 4), idesc_s, k > 0);
        tc_commit(bars + kBarS + t);
      };
      auto mma_o = [&](int t, uint32_t st, bool first) {  // O_t += P_t V
        const uint64_t dv = dv0 + st * kNext;
        const uint32_t d = tmem + 256 + t * 128, p = tmem + t * kT;
#pragma unroll
        for (int k = 0; k < kT / 16; ++k)  // the halves of P start 64 columns apart
          tc_mma_f16_ts(d, p + (k >> 2) * kHalf + (k & 3) * 8, dv + k * (2 * D * 16 >> 4), idesc_o,
                        !(first && k == 0));
      };
      uint32_t g = 0;              // tiles done by this CTA
      uint32_t nq = 0, np = 0;     // bit t: phase of row tile t's Q and P
      bool ok = true;
      for (int it = it0, u = u0; u < u1 && ok; ++it) {
        const Item im = load_item(a, pv, it, u, u1);
        const int n = im.t1 - im.t0;
        u += n;
        const int two = im.rows > 128 ? 2 : 1;
        // k = -1 issues the first S of the row tiles, k >= 0 P V of tile k and
        // S of tile k + 1
        for (int k = -1; k < n && ok; ++k) {
          const bool more = k + 1 < n;
          const uint32_t g1 = g + (k >= 0 ? 1 : 0);  // tile k + 1
          if (more) ok = wait(kBarKFull + (g1 & 1), (g1 >> 1) & 1);
          if (k >= 0) ok = ok && wait(kBarVFull + (g & 1), (g >> 1) & 1);
#pragma unroll 1
          for (int t = 0; t < two && ok; ++t) {
            const uint32_t phase = k < 0 ? nq : np;
            ok = wait((k < 0 ? kBarQ : kBarP) + t, (phase >> t) & 1);
            if (!ok) break;
            if (k < 0) nq ^= 1u << t;
            else np ^= 1u << t;
            tc_fence_after();
            if (k >= 0) {
              mma_o(t, g & 1, k == 0);
              if (t + 1 == two) tc_commit(bars + kBarVFree + (g & 1));
              if (!more) tc_commit(bars + kBarO + t);
            }
            if (more) mma_s(t, g1 & 1);
          }
          if (more) tc_commit(bars + kBarKFree + (g1 & 1));
          g = g1;
        }
      }
    }
  } else if (warp >= kConvWarp) {
    convert_tiles<D, FMT>(a, pv, sm, abort_flag, it0, u0, u1, warp - kConvWarp, lane);
  } else {
    // ================================================= softmax warps
    const int t = warp >> 3, half = (warp >> 2) & 1;  // row tile, and tokens of its tiles
    const int rl = (warp & 3) * 32 + lane;            // row within it
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + t * kT + half * kHalf + lanes, to = tmem + 256 + t * 128 + lanes;
    float* xch = reinterpret_cast<float*>(sm + SM::kXch) + warp * 32 + lane;
    uint32_t nx = 0;
    // Trade one value per row with the other warp of the rows.  The slots
    // alternate: one is written again only after the other warp's next arrival.
    auto trade = [&](float mine, float& other) {
      float* slot = xch + (nx & 1) * (16 * 32);
      *slot = mine;
      __syncwarp();
      const int bar = kBarX + t * 4 + (warp & 3);
      if (lane == 0) mbar_arrive(bars + bar);
      const bool good = wait_warp(bar, nx & 1);
      ++nx;
      other = slot[half ? -4 * 32 : 4 * 32];
      return good;
    };
    uint32_t g = 0, ns = 0, no = 0;  // tiles of the CTA; tiles and items of this row tile
    bool ok = true;
    for (int it = it0, u = u0; u < u1 && ok; ++it) {
      const Item im = load_item(a, pv, it, u, u1);
      const int n = im.t1 - im.t0;
      u += n;
      if (t == 1 && im.rows <= 128) {  // row tile 1 of a short block idles
        g += n;
        continue;
      }
      const int r = t * 128 + rl;  // row of the block
      const bool live = r < im.rows;
      const int rr = im.row0 + min(r, im.rows - 1);
      const int qi = rr / a.G, h = im.kvh * a.G + rr % a.G;
      const long grow = (static_cast<long>(im.c.qlo) + qi) * a.hq + h;  // row of q and out
      float zs;
      {
        // ---- the row of q, normalised by a power of two, into shared memory
        // (every QK^T of the previous item is done: its last S was read)
        const uint4* src = reinterpret_cast<const uint4*>(a.q + grow * D);
        const float sgn = a.sm_scale < 0.f ? -1.f : 1.f;
        const bool st = a.mode == FP8PA_SCALE_CHANNEL_STATIC;
        const float* kc = a.k_scale + static_cast<long>(im.kvh) * D;
        float amax = 0.f;
        auto get = [&](int x, float (&f)[8]) {
          const uint4 raw = __ldg(src + x);
          const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[2 * e] = __uint_as_float(w[e] << 16) * sgn;
            f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u) * sgn;
          }
          if (st) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= __ldg(kc + x * 8 + e);
          }
        };
#pragma unroll 4
        for (int x = 0; x < D / 8; ++x) {
          float f[8];
          get(x, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
        }
        const int eq = amax > 0.f ? exp_above(amax) : 0;
        const float fq = exp2i(14 - eq);
        uint8_t* dst = sm + SM::kQ + t * SM::kTile + (rl >> 3) * 128 + (rl & 7) * 16;
#pragma unroll 2
        for (int x0 = 0; x0 < D / 16; ++x0) {  // this thread's half, from L1
          const int x = half * (D / 16) + x0;
          float f[8];
          get(x, f);
          const uint4 o = make_uint4(pack_half2(f[0] * fq, f[1] * fq),
                                     pack_half2(f[2] * fq, f[3] * fq),
                                     pack_half2(f[4] * fq, f[5] * fq),
                                     pack_half2(f[6] * fq, f[7] * fq));
          *reinterpret_cast<uint4*>(dst + x * 2048) = o;
        }
        // log2-domain factor of a raw score (capped scores: of 2 z / cap); never
        // zero, so that a masked -inf stays -inf
        zs = fmaxf(fabsf(a.sm_scale) * exp2i(eq - 14) * kLog2e *
                       (VAR == 2 ? 2.f / a.cap : 1.f),
                   1e-37f);
        fence_proxy_async();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + kBarQ + t);
      const int pos = im.c.L - im.c.n + qi;
      const int wf = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
      const int pre = im.c.pre;
      // extremes over the warp's rows (positions rise with the row)
      const int pA = __shfl_sync(0xffffffffu, pos, 0), wB = __shfl_sync(0xffffffffu, wf, 31);
      const float slope = (VAR > 0 && a.slopes) ? __ldg(a.slopes + h) * kLog2e : 0.f;
      const float cap_log2 = VAR == 2 ? a.cap * kLog2e : 0.f;
      float ref = kNegBig, l = 0.f;

      for (int k = 0; k < n; ++k, ++g) {
        const uint32_t s4 = g & 3;
        const int j0 = tile_token(im, im.t0 + k) + half * kHalf;
        if (!wait_warp(kBarScale + s4, (g >> 2) & 1) || !wait_warp(kBarS + t, ns & 1)) {
          ok = false;
          break;
        }
        ++ns;
        tc_fence_after();
        const float* sk = scales + s4 * 2 * kT + half * kHalf;
        const float* sv = sk + kT;
        const uint2 val = *reinterpret_cast<const uint2*>(&infos[s4].valid[half * 2]);
        // whether every row of the warp sees all of the thread's tokens
        const bool whole =
            ((j0 >= wB && j0 + kHalf - 1 <= pA) || (VAR == 0 && j0 + kHalf <= pre)) &&
            (val.x & val.y) == 0xFFFFFFFFu && (VAR < 2 || a.cap <= kCapFast);
        uint2 mw = make_uint2(0xFFFFFFFFu, 0xFFFFFFFFu);  // tokens that the row sees
        const float zf = VAR > 0 ? 1.f : zs;
        float bound;
        // ---- scores times K scales (VAR > 0: final scores) go back to TMEM:
        // reading the scales a second time would cost shared-memory bandwidth
        // that the MMAs' operands need.  And a bound of z + log2(V scale).
        if (whole) {
          const float2 vm = *reinterpret_cast<const float2*>(&infos[s4].vmax[half * 2]);
          const ulonglong2* sk2 = reinterpret_cast<const ulonglong2*>(sk);
          const uint64_t zs2 = f2_pack(zs, zs), step = f2_pack(2.f * slope, 2.f * slope);
          float m4[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) m4[x] = __int_as_float(0xff800000);
#pragma unroll 2
          for (int c = 0; c < 4; ++c) {
            uint32_t raw[16];
            tmem_ld16(ts + c * 16, raw);
            // the bias of tokens 2 i, 2 i + 1 of the chunk: -slope (pos - j)
            const float b0 = VAR > 0 ? slope * static_cast<float>(j0 + c * 16 - pos) : 0.f;
            const uint64_t bias = f2_pack(b0, b0 + slope);
            tmem_ld_wait();
            tmem_landed(raw);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const ulonglong2 f = sk2[c * 4 + i / 2];
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t* r = raw + (i + x) * 2;
                uint64_t z = f2_mul(f2_pack(__uint_as_float(r[0]), __uint_as_float(r[1])),
                                    x ? f.y : f.x);
                float p, q;
                if constexpr (VAR > 0) {
                  const float fi = static_cast<float>(i + x);
                  const uint64_t b = f2_fma(step, f2_pack(fi, fi), bias);
                  if constexpr (VAR == 1) {
                    z = f2_fma(z, zs2, b);
                  } else {  // cap tanh(z / cap) = cap - 2 cap / (2^x + 1)
                    f2_unpack(f2_mul(z, zs2), p, q);
                    z = f2_add(f2_pack(cap_fast(p, cap_log2), cap_fast(q, cap_log2)), b);
                  }
                }
                f2_unpack(z, p, q);
                m4[(i + x) & 3] = max3(m4[(i + x) & 3], p, q);
                r[0] = __float_as_uint(p);
                r[1] = __float_as_uint(q);
              }
            }
            tmem_st16(ts + c * 16, raw);
          }
          bound = bound_of(max3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * zf, fmaxf(vm.x, vm.y));
        } else {
          // some row masks some token: masked scores become -inf, and a row's V
          // bound is that of the tokens it sees
          mw.x = (word_bits(j0, wf, pos + 1) | word_bits(j0, 0, pre)) & val.x;
          mw.y = (word_bits(j0 + 32, wf, pos + 1) | word_bits(j0 + 32, 0, pre)) & val.y;
          float mx = __int_as_float(0xff800000), vmax = 0.f;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t raw[16];
            tmem_ld16(ts + c * 16, raw);
            tmem_ld_wait();
            tmem_landed(raw);
            const uint32_t m = (c < 2 ? mw.x : mw.y) >> (16 * (c & 1));
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float z = __uint_as_float(raw[i]) * sk[c * 16 + i];
              if constexpr (VAR > 0) {
                z *= zs;
                if constexpr (VAR == 2) z = cap_log2 * tanh_f32(z * (0.5f / kLog2e));
                z = fmaf(-slope, fabsf(static_cast<float>(pos - j0 - c * 16 - i)), z);
              }
              const bool see = (m >> i) & 1;
              z = see ? z : __int_as_float(0xff800000);
              mx = fmaxf(mx, z);
              vmax = fmaxf(vmax, see ? sv[c * 16 + i] : 0.f);
              raw[i] = __float_as_uint(z);
            }
            tmem_st16(ts + c * 16, raw);
          }
          bound = bound_of(mx * zf, vmax);
        }
        tmem_st_wait();
        // ---- the reference, shared by the row's two threads: where the bound
        // passed it by 2^kTau it moves, and with it the sums and O
        float other;
        if (!trade(bound, other)) {
          ok = false;
          break;
        }
        bound = fmaxf(bound, other);
        float al = 1.f;
        if (bound > ref + kTau) {
          al = ex2(ref - bound);
          ref = bound;
        }
        if (__any_sync(0xffffffffu, al != 1.f)) {
          l *= al;
          if (k > 0) {  // (P V of the last tile is done: S of this one came behind it)
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              const uint32_t at = to + half * (D / 2) + c * 16;
              uint32_t o[16];
              tmem_ld16(at, o);
              tmem_ld_wait();
              tmem_landed(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
              tmem_st16(at, o);
            }
          }
        }
        // ---- P and its sum
        const float c0 = kShift - ref;
        const uint64_t zf2 = f2_pack(zf, zf), c02 = f2_pack(c0, c0);
        const ulonglong2* sv2 = reinterpret_cast<const ulonglong2*>(sv);
        uint64_t la = 0, lb = 0;  // (0.f, 0.f)
        auto weigh = [&](auto masked) {
#pragma unroll 2
          for (int c = 0; c < 4; ++c) {
            uint32_t raw[16], pw[8];
            tmem_ld16(ts + c * 16, raw);
            tmem_ld_wait();
            tmem_landed(raw);
            const uint32_t m = (c < 2 ? mw.x : mw.y) >> (16 * (c & 1));
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const ulonglong2 v = sv2[c * 4 + i / 2];
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t* r = raw + (i + x) * 2;
                const uint64_t z = f2_pack(__uint_as_float(r[0]), __uint_as_float(r[1]));
                float p, q;
                f2_unpack(VAR > 0 ? f2_add(z, c02) : f2_fma(z, zf2, c02), p, q);
                const uint64_t p2 = f2_pack(ex2(p), ex2(q));
                if (x) lb = f2_add(lb, p2);
                else la = f2_add(la, p2);
                uint64_t v2 = x ? v.y : v.x;
                if constexpr (masked.value) {  // a masked token's scale may be anything
                  f2_unpack(v2, p, q);
                  v2 = f2_pack((m >> (2 * (i + x))) & 1 ? p : 0.f,
                               (m >> (2 * (i + x) + 1)) & 1 ? q : 0.f);
                }
                f2_unpack(f2_mul(p2, v2), p, q);
                pw[i + x] = pack_half2(p, q);
              }
            }
            tmem_st8(ts + c * 8, pw);
          }
        };
        if (whole) weigh(std::false_type{});
        else weigh(std::true_type{});
        float x, y;
        f2_unpack(f2_add(la, lb), x, y);
        l += x + y;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kBarP + t);
      }
      if (!ok) break;

      // ---- the block's result, or this range's piece of it: half the dims each
      float other;
      if (!trade(l, other) || !wait_warp(kBarO + t, no & 1)) {
        ok = false;
        break;
      }
      ++no;
      l += other;
      tc_fence_after();
      const bool piece = im.t0 > 0 || im.t1 < im.tl.count;
      const float inv = piece ? 1.f : (l == 0.f ? 0.f : 1.f / l);
      const int slot = blockIdx.x * 2 + (im.t0 > 0 ? 0 : 1);
      const bool stat = a.mode == FP8PA_SCALE_CHANNEL_STATIC;
      const float* vch = a.v_scale + static_cast<long>(im.kvh) * D;
#pragma unroll 1
      for (int c0 = 0; c0 < D / 32; ++c0) {
        const int c = half * (D / 32) + c0;
        uint32_t o[16];
        tmem_ld16(to + c * 16, o);
        tmem_ld_wait();
        tmem_landed(o);
        if (!live) continue;
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          f[i] = __uint_as_float(o[i]) * inv;
          if (stat) f[i] *= __ldg(vch + c * 16 + i);
        }
        if (piece || a.out_f32) {
          float* dst = piece ? pv.o + (static_cast<long>(slot) * kRows + r) * D + c * 16
                             : reinterpret_cast<float*>(a.out) + grow * D + c * 16;
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(dst + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + grow * D +
                                                c * 16);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const __nv_bfloat162 b2 =
                  __floats2bfloat162_rn(f[8 * i + 2 * x], f[8 * i + 2 * x + 1]);
              w[x] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (piece && live && half == 0) pv.ml[static_cast<long>(slot) * kRows + r] = make_float2(ref, l);
      tc_fence_before();
    }
  }

  // ---- drain and free: no MMA may still be in flight
  __syncwarp();
  if (warp == kIssueWarp && lane == 0) {
    tc_commit(bars + kBarDrain);
    (void)mbar_wait_bounded(bars + kBarDrain, 0, kWaitLimitCycles);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- merge
// CTA (w, part): if cut w + 1 is the first inside its item, fold the pieces of
// 32 of the item's rows: the first ends range w, the others open the ranges
// behind it.
constexpr int kMergeRows = 32;

template <int D>
__global__ void __launch_bounds__(256) prefill_merge_kernel(const PrefillArgs a, const PlanView pv,
                                                            int ranges) {
  griddep_wait();
  griddep_launch_dependents();
  const int w = blockIdx.x;
  const int cut = pv.start[w + 1], U = pv.head[0];
  if (cut >= U) return;
  const int it = pv.item[w + 1], rb = it / a.hkv, kvh = it - rb * a.hkv;
  const int pre = pv.rb_pre[rb], c = pv.rb_pre[rb + 1] - pre;
  const int f = pre * a.hkv + kvh * c;
  // an earlier cut inside the item folds it
  if (cut <= f || pv.start[w] > f) return;
  const int b = pv.rb_b[rb];
  bool x, y;
  const Chunk ch = load_chunk(a, b, &x, &y);
  const int row0 = (rb - pv.rbase[b]) * kRows, rows = min(kRows, ch.n * a.G - row0);
  constexpr int TPR = D / 4;        // threads per row
  constexpr int RPC = 256 / TPR;    // rows at a time
  const int sub = threadIdx.x / TPR, d0 = (threadIdx.x % TPR) * 4;
  for (int r = blockIdx.y * kMergeRows + sub; r < min(rows, (static_cast<int>(blockIdx.y) + 1) * kMergeRows);
       r += RPC) {
    float M = kNegBig, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = w; k < ranges; ++k) {
      if (k > w && pv.start[k] >= f + c) break;
      if (k > w && pv.start[k] == pv.start[k + 1]) continue;  // an empty range
      const long p = (static_cast<long>(2 * k + (k == w ? 1 : 0)) * kRows) + r;
      const float2 ml = pv.ml[p];
      const float4 o = *reinterpret_cast<const float4*>(pv.o + p * D + d0);
      const float mn = fmaxf(M, ml.x);
      const float s0 = ex2(M - mn), s1 = ex2(ml.x - mn);
      L = L * s0 + ml.y * s1;
      acc.x = acc.x * s0 + o.x * s1;
      acc.y = acc.y * s0 + o.y * s1;
      acc.z = acc.z * s0 + o.z * s1;
      acc.w = acc.w * s0 + o.w * s1;
      M = mn;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int rr = row0 + r;
    const long grow = (static_cast<long>(ch.qlo) + rr / a.G) * a.hq + kvh * a.G + rr % a.G;
    if (a.out_f32) {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + grow * D + d0) =
          make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    } else {
      __nv_bfloat162 o[2] = {__floats2bfloat162_rn(acc.x * inv, acc.y * inv),
                             __floats2bfloat162_rn(acc.z * inv, acc.w * inv)};
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + grow * D + d0) =
          *reinterpret_cast<const uint2*>(o);
    }
  }
}

// ---------------------------------------------------------------- host side
using PrefillFn = void (*)(const PrefillArgs, const PlanView);

template <int D, int FMT>
PrefillFn pick_var(int var) {
  return var == 0 ? prefill_kernel<D, FMT, 0>
                  : (var == 1 ? prefill_kernel<D, FMT, 1> : prefill_kernel<D, FMT, 2>);
}
template <int D>
PrefillFn pick_fmt(int fmt, int var) {
  return fmt == FP8PA_E4M3   ? pick_var<D, FP8PA_E4M3>(var)
         : fmt == FP8PA_E5M2 ? pick_var<D, FP8PA_E5M2>(var)
                             : pick_var<D, FP8PA_INT8>(var);
}

}  // namespace

size_t prefill_workspace_bytes(int total_q, int batch, int hq, int hkv, int d, int device) {
  return plan_layout(nullptr, total_q, batch, hq / hkv, d, sm_count(device), nullptr);
}

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int ranges = sm_count(dev);
  PlanView pv;
  plan_layout(static_cast<char*>(a.workspace), a.total_q, a.batch, a.G, a.d, ranges, &pv);
  const int var = a.cap > 0.f ? 2 : (a.slopes ? 1 : 0);
  const PrefillFn fn = a.d == 128 ? pick_fmt<128>(a.fmt, var) : pick_fmt<64>(a.fmt, var);
  const int smem = a.d == 128 ? Smem<128>::kBytes : Smem<64>::kBytes;
  if ((e = ensure_smem_attr(reinterpret_cast<const void*>(fn), smem)) != cudaSuccess) return e;

  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreads);
  if ((e = cudaLaunchKernelEx(&cfg, prefill_plan_kernel, a, pv, ranges)) != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(ranges));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  if ((e = cudaLaunchKernelEx(&cfg, fn, a, pv)) != cudaSuccess) return e;
  if (ranges < 2) return cudaSuccess;
  cfg.gridDim = dim3(static_cast<unsigned>(ranges - 1), kRows / kMergeRows);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return a.d == 128 ? cudaLaunchKernelEx(&cfg, prefill_merge_kernel<128>, a, pv, ranges)
                    : cudaLaunchKernelEx(&cfg, prefill_merge_kernel<64>, a, pv, ranges);
}

}  // namespace fp8pa
