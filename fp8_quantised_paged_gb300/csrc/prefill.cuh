// prefill.cuh -- attention of ragged query chunks over the paged cache, causal
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
// Each K or V code is read and converted once for 256 rows, or, where a request
// has many row blocks, once for all of them (ready tiles, below).
//
// Work is the flat list of (row block, KV head, token tile) units.  A planner
// kernel counts the tiles that each row block can see and cuts the list into
// one contiguous range per SM; where a cut falls inside an item (it is moved
// to an item's edge when that is a few tiles away) the pieces leave partial
// results that a merge kernel folds with the log-sum-exp rule.  A long chunk
// and a few rows over a long context are balanced alike.
//
// Numerics.  The converters give K^ and V^ as f16: a code times its token's scale
// relative to the largest of its 32 tokens (a power of two 2^e that stays
// outside), rounded once (2^-11; exact for MX blocks and static scales).  The
// largest is put as high as f16 allows, so that a token whose scale is 2^r below
// it (which some rows may mask) is off by no more than 2^(r - 32) beside that
// rounding; E5M2's codes fill f16's exponents by themselves: 2^(r - 25).  The
// exponent of V has a floor (kLowV), which holds the sums of rows within fp32; as P
// carries that exponent, a weight is lost to the sum where it and the exponents apart
// make 2^-126, past 2^100 between the scales of V.  Scaling
// the fp32 scores and P instead would keep the scales exact, but costs every
// score two multiplications and two broadcast loads beside MMAs that fill the
// shared-memory bandwidth: 1.45 ms against 1.30 ms for 2048 queries over 16384
// tokens (before the ready tiles).  q is exact in f16 after a power-of-two normaliser per row
// (CHANNEL_STATIC folds the K scales into it and rounds once, 2^-11).  P enters
// the second product as f16 (2^-11).  The running reference of a row is a bound
// of max(z + e), e the exponent of the V^ group, so P stays inside f16 whatever
// the scales; it moves only when passed by 2^kTau, which is exact, as sums and O
// carry the same reference.
//
// Roles: warps 0-7 and 8-15 the softmax of row tiles 0 and 1, two threads per
// row, each with half of a step's tokens (four warps per scheduler hide one
// another's waits; the two agree on the row's reference through shared memory);
// then seven warps that convert codes into shared memory, or two that load ready
// tiles (a thread each); the last issues the MMAs (one thread).  While the tensor
// cores work on one row tile, the other's softmax runs.  Every wait is bounded.
//
// Measured, head_dim 128, 64 heads over 8: 2048 queries over 16384 tokens 910-920
// us, 1.12 PFLOP/s (58% of a large library product's rate); before the ready tiles
// 1260 us.  Per 128-token tile of 256 rows that is 4200 cycles, 2800 of them with
// MMAs under way (2048 at their own rate: the shared memory that feeds both
// operands of S also takes the tiles in), the rest the softmax's own chain.
#pragma once

#include <float.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "score_mods.cuh"
#include "tc.cuh"

namespace fp8pa {

// ---------------------------------------------------------------- plan
// Workspace: header, block prefix of the requests, then per row block its
// request and the prefix of its tiles, then the ranges' first units, then the
// partial pieces.
struct PlanView {
  int* head;     // [0] units, [1] units per range (before cuts move)
  int* rbase;    // [batch + 1] first row block of a request
  int4* rb;      // [blocks][3] a row block: see RowBlock
  int* rb_pre;   // [blocks + 1] tiles before a row block (of one KV head)
  int* start;    // [ranges + 1] first unit of a range
  int* item;     // [ranges + 1] the item that holds it
  float2* ml;    // [2 * ranges][kRows] reference and sum of a piece
  float* o;      // [2 * ranges][kRows][d]
  uint8_t* tiles;  // ready tiles: [batch][KV heads][tpr][K^, V^] in their shared-memory form
  uint8_t* info;   // ... and the StageInfo of each
  int blocks;    // bound of the row blocks
  int tpr;       // tiles of a request
};

using PrefillFn = void (*)(const PrefillArgs, const PlanView);
// The instances for a format, MX scales and score variant (prefill_d64.cu,
// prefill_d128.cu).  ready: the kernel over ready tiles, and the one that makes
// them.
struct PrefillKernels {
  PrefillFn attend, make;
  int smem, threads;
};
PrefillKernels pick_prefill_d64(int fmt, int var, bool mx, bool ready);
PrefillKernels pick_prefill_d128(int fmt, int var, bool mx, bool ready);

namespace {

constexpr int kRows = 256;   // rows of a block: two tiles of 128
constexpr int kT = 128;      // tokens per tile
constexpr int kAhead = 3;    // jobs that a converting warp asks L2 for ahead
constexpr int kConvWarp = 16, kConvWarps = 7;  // or a K and a V loader over ready tiles
// Tokens scored at a time.  Over ready tiles the MMAs are what is waited for, and a
// step of 64 costs S nearly what one of 128 does (93 cycles against 87 for each 16
// dims): 2048 queries over 16384 tokens take 1362 us by 64, 910-920 us by 128.  Without
// them chunks are short, mostly of one row tile, and two steps of 64 in columns of
// their own let S of one run beside the softmax of the other.  That paid while the
// scores went through TMEM again (386 us by 64, 453 by 128, for 8 chunks of 64 rows over
// 32768 tokens).  With scores in registers it no longer does: 370 and 366 us there (MX
// scales, bias), 320 and 305 with token scales alone, 114 and 103 for two row tiles (512
// rows over 16384 tokens).
template <bool READY>
constexpr int kStep = READY ? 128 : 64;
template <bool READY>
constexpr int kIssueWarp = kConvWarp + (READY ? 2 : kConvWarps);
template <bool READY>
constexpr int kThreads = (kIssueWarp<READY> + 1) * 32;
constexpr int kSnap = 4;     // a cut this near an item's edge moves to it
constexpr float kShift = 12.f;  // P = 2^(z - ref + 12): at most 2^15 with the lazy bound
constexpr float kTau = 3.f;     // the reference may lag by 2^3
constexpr float kNegBig = -1e30f;
// The smallest exponents that K^ and V^ leave out.  A row's sum holds 2^(z - ref + 12)
// of each token, and ref is at least max(z + e) - kTau: a token adds at
// most 2^(15 - e), 2^95 here, so that 2^31 tokens whose V is next to nothing stay
// within fp32.  Values of V below 2^-94 lose bits in V^ for it (half of 2^-104).
constexpr int kLowK = -107, kLowV = -80;

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

// A row block, as the planner writes it: its request and chunk, its rows, and
// the token tiles that it can see: tiles [0, np) of the prefix, then from tile np
// + skip on, `count` in all (at least one, so that rows that see nothing are
// written); the positions of its first and last query.
struct RowBlock {
  int b, qlo, n, L;
  int pre, row0, rows, np;
  int skip, count, pA, pB;
};
__device__ __forceinline__ RowBlock make_row_block(const Chunk& c, int b, int window, int G,
                                                   int t) {
  RowBlock r;
  r.b = b;
  r.qlo = c.qlo;
  r.n = c.n;
  r.L = c.L;
  r.pre = c.pre;
  r.row0 = t * kRows;
  r.rows = min(kRows, c.n * G - r.row0);
  r.pA = c.L - c.n + r.row0 / G;
  r.pB = c.L - c.n + (r.row0 + r.rows - 1) / G;
  const int wf = window_first(window, r.pA);
  r.np = (c.pre + kT - 1) / kT;
  r.skip = max(wf / kT - r.np, 0);
  const int last = (max(max(r.pB + 1, c.pre), 0) + kT - 1) / kT;
  r.count = max(last - r.skip, 1);
  return r;
}
__device__ __forceinline__ RowBlock load_row_block(const int4* p) {
  const int4 a = p[0], b = p[1], c = p[2];
  return RowBlock{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
}

// ---------------------------------------------------------------- shared memory
// Of a tile's four groups of 32 tokens: the exponents that K^ and V^ leave out,
// the tokens whose page exists, and those whose V is not finite (zeroed in V^
// where some row masks them; rows that see one are NaN).
struct StageInfo {
  int ek[4], ev[4];
  uint32_t valid[4], bad[4];
};

template <int D>
struct Smem {
  static constexpr int kTile = kT * D * 2;  // a 128-row f16 tile
  static constexpr int kQ = 0;              // two row tiles
  static constexpr int kK = 2 * kTile;      // two stages
  static constexpr int kV = 4 * kTile;      // two stages
  static constexpr int kInfo = 6 * kTile;   // four stages of StageInfo
  static constexpr int kXch = kInfo + 4 * sizeof(StageInfo);  // [parity][warp of softmax][lane] f32
  static constexpr int kBars = kXch + 2 * 16 * 32 * 4;
  static constexpr int kMisc = kBars + 320;  // TMEM base, abort flag
  static constexpr int kBytes = kMisc + 16;
};
// Barriers and the arrivals that complete a phase.  Q (by row tile t) and P (t * 2
// + step): the eight softmax warps of the row tile; scales: the eight conversion
// jobs of the tile; K and V full: four jobs (over ready tiles, one thread and its
// bytes for each of these); X (t * 4 + lane quarter): the two softmax warps of the
// same rows; the others, S and O by t * 2 + step: a commit of the tensor cores.
enum { kBarQ = 0, kBarP = 2, kBarScale = 6, kBarKFull = 10, kBarVFull = 12, kBarX = 14,
       kBarKFree = 22, kBarVFree = 24, kBarS = 26, kBarO = 30, kBarDrain = 34, kNumBars = 35 };

// ---------------------------------------------------------------- conversions
// 16 codes -> 16 f16 (two 16-byte core-matrix rows), exactly.
template <int FMT>
__device__ __forceinline__ void codes16_to_f16(const uint4& c, uint4& lo, uint4& hi) {
  codes4_to_f16x2x2<FMT>(c.x, lo.x, lo.y);
  codes4_to_f16x2x2<FMT>(c.y, lo.z, lo.w);
  codes4_to_f16x2x2<FMT>(c.z, hi.x, hi.y);
  codes4_to_f16x2x2<FMT>(c.w, hi.z, hi.w);
}

// 16 code bytes that one CTA reads once: they are kept out of L1, which is small
// beside this kernel's shared memory.
__device__ __forceinline__ uint4 ld_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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

__device__ __forceinline__ __half2 h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t h2_bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
// Eight f16 codes times a scale hi + lo, rounded once.
__device__ __forceinline__ uint4 scale8(const uint4& a, __half2 hi, __half2 lo) {
  auto m = [&](uint32_t x) { return h2_bits(__hfma2(h2(x), hi, __hmul2(h2(x), lo))); };
  return make_uint4(m(a.x), m(a.y), m(a.z), m(a.w));
}
__device__ __forceinline__ uint4 scale8(const uint4& a, __half2 f) {
  auto m = [&](uint32_t x) { return h2_bits(__hmul2(h2(x), f)); };
  return make_uint4(m(a.x), m(a.y), m(a.z), m(a.w));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// Registers that a tcgen05.ld filled: what uses them stays behind the
// tcgen05.wait::ld before this.
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[8]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]));
}
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

// One item of a CTA's range: a row block for one KV head, tiles [t0, t1) of its
// list.  Out of line: every role calls it once per item, and the roles' loops
// have to share the instruction caches.
struct Item {
  RowBlock r;
  int kvh, t0, t1;
};
__device__ __noinline__ Item load_item(const PrefillArgs& a, const PlanView& v, int it, int u,
                                       int u1) {
  Item m;
  const int rb = it / a.hkv;
  m.kvh = it - rb * a.hkv;
  const int pre = v.rb_pre[rb];
  m.r = load_row_block(v.rb + 3 * rb);
  const int f = pre * a.hkv + m.kvh * m.r.count;
  m.t0 = u - f;
  m.t1 = min(m.r.count, u1 - f);
  return m;
}

// ---------------------------------------------------------------- conversion
// A job: 32 tokens of K or V of a tile (parts 0-3: K, 4-7: V) and one KV head, by
// one warp.  A lane holds row r8 of four 8-row groups and, of each, the 16-byte
// chunks c4 (and c4 + 4): loads take 64 contiguous bytes of 8 rows, stores the 8
// rows of a core matrix, free of bank conflicts.
template <int D>
struct Job {
  uint4 buf[4][D / 64];  // the lane's codes
  uint32_t okm;          // groups whose row is wanted and exists
  float sc;              // scale of token `lane`
  bool sok;              // ... which is wanted and exists
  uint32_t ex[D / 64];   // MX: exponents of the lane's chunks, by group
  int em;                // ... and of the token's largest block
};
// The tokens that some row sees: [lo, hi) and [0, pre).  Others are neither
// looked up nor read.
struct Seen {
  int lo, hi, pre;
  __device__ __forceinline__ bool operator()(int j) const { return (j < hi && j >= lo) || j < pre; }
};
// Block ids of the two 16-token halves of a job at token j (a half lies in one
// block); -1 where no row sees any of its tokens.
__device__ __forceinline__ void job_blocks(const int32_t* table, int lgbs, const Seen& seen, int j,
                                           int (&id)[2]) {
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int t = j + 16 * x;
    id[x] = (t < seen.hi && t + 16 > seen.lo) || t < seen.pre
                ? __ldg(table + static_cast<int>(static_cast<uint32_t>(t) >> lgbs))
                : -1;
  }
}
__device__ __forceinline__ uint32_t cache_row(const PrefillArgs& a, int kvh, int blk, int t) {
  return (static_cast<uint32_t>(blk) * a.hkv + kvh) * a.bs + (t & (a.bs - 1));
}

template <int D, bool MX>
__device__ __forceinline__ void load_job(const PrefillArgs& a, bool V, int kvh, const int (&ids)[2],
                                         int j, const Seen& seen, int lane, Job<D>& job) {
  constexpr int H = D / 64;
  const int r8 = lane & 7, c4 = lane >> 3;
  const uint8_t* cache = V ? a.v_cache : a.k_cache;
  const float* gscale = V ? a.v_scale : a.k_scale;
  job.okm = 0;
  const int nbx = MX ? D / a.gs : 0;
  // code rows of the two halves' first tokens
  const bool blk_ok[2] = {ids[0] >= 0 && ids[0] < a.num_blocks,
                          ids[1] >= 0 && ids[1] < a.num_blocks};
  const uint32_t row[2] = {blk_ok[0] ? cache_row(a, kvh, ids[0], j) : 0u,
                           blk_ok[1] ? cache_row(a, kvh, ids[1], j + 16) : 0u};
  const uint32_t lane_at = r8 * D + c4 * 16;
  if (((j >= seen.lo && j + 32 <= seen.hi) || j + 32 <= seen.pre) && blk_ok[0] && blk_ok[1]) {
    job.okm = 0xFu;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint8_t* src =
          cache + static_cast<size_t>(row[x >> 1]) * D + lane_at + (x & 1) * 8 * D;
#pragma unroll
      for (int h = 0; h < H; ++h) job.buf[x][h] = ld_codes(src + h * 64);
    }
  } else {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const bool ok = seen(j + x * 8 + r8) && blk_ok[x >> 1];
      if (ok) job.okm |= 1u << x;
      const uint8_t* src =
          cache + static_cast<size_t>(row[x >> 1]) * D + lane_at + (x & 1) * 8 * D;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        job.buf[x][h] = make_uint4(0u, 0u, 0u, 0u);
        if (ok) job.buf[x][h] = ld_codes(src + h * 64);
      }
    }
  }
  job.sc = 1.f;
  job.em = 0;
  {
    const bool want = seen(j + lane);
    job.sok = want && (lane < 16 ? blk_ok[0] : blk_ok[1]);
    if (want && !job.sok) raise_error(a.err, FP8PA_DEVERR_BLOCK_RANGE);
    const size_t rw = (lane < 16 ? row[0] : row[1]) + (lane & 15);
    if (a.mode == FP8PA_SCALE_TOKEN_HEAD) {
      if (job.sok) job.sc = __ldg(gscale + rw);
    } else if (a.mode == FP8PA_SCALE_SEGMENT) {
      if (job.sok) job.sc = __ldg(gscale + static_cast<long>(lane < 16 ? ids[0] : ids[1]) * a.hp + kvh);
    } else if constexpr (MX) {
      // 2, 4 or 8 bytes a row (a missing block's rows read as block 0's: not
      // used)
      const uint8_t* exps = reinterpret_cast<const uint8_t*>(gscale);
      uint32_t w[2];
      w[1] = nbx == 8 ? __ldg(reinterpret_cast<const uint32_t*>(exps + rw * 8) + 1) : 0u;
      w[0] = nbx == 2 ? __ldg(reinterpret_cast<const uint16_t*>(exps + rw * 2))
                      : __ldg(reinterpret_cast<const uint32_t*>(exps + rw * nbx));
      job.em = job.sok ? static_cast<int>(max_byte(w)) : 0;
      // the lane's rows' blocks from the lanes that hold them
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int b = (h * 4 + c4) * 16 / a.gs;
        job.ex[h] = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t lo4 = __shfl_sync(0xffffffffu, w[0], x * 8 + r8);
          const uint32_t hi4 = __shfl_sync(0xffffffffu, w[1], x * 8 + r8);
          job.ex[h] |= (((b & 4 ? hi4 : lo4) >> (8 * (b & 3))) & 0xFFu) << (8 * x);
        }
      }
    }
  }
}

// The job's part of a 128-token tile of f16, and of its info.  whole: every row
// sees the whole tile.
template <int D, int FMT, bool MX>
__device__ __forceinline__ void finish_job(const PrefillArgs& a, Job<D>& job, bool V, int dw,
                                           bool whole, uint8_t* tile, StageInfo* info, int lane) {
  constexpr int H = D / 64;
  constexpr int kRoom = FMT == FP8PA_E5M2 ? 0 : 7;  // codes of at most 448 leave f16 this much
  const int r8 = lane & 7, c4 = lane >> 3;
  const uint32_t valid = __ballot_sync(0xffffffffu, job.sok);
  // The group's exponent, kRoom below the one above its largest finite scale, and the
  // scales relative to it.  A scale counts as finite where its largest code is, in fp32
  // (append writes no others): the relative scales of these stay below 2^kRoom, so that
  // V^ is finite, and a larger one does not cost its group the precision.
  const bool finite = MX ? job.em <= 254 - (FMT == FP8PA_E5M2 ? 15 : 8)
                         : job.sc <= FLT_MAX / code_max<FMT>();  // (not for a NaN)
  const int low = V ? kLowV : kLowK;
  int e;
  if constexpr (MX) {
    e = max(__reduce_max_sync(0xffffffffu, finite ? job.em : 0) - 127 - kRoom, low);
  } else {
    e = max(exp_above(warp_max_f32(job.sok && finite ? job.sc : 0.f)) - kRoom, low);
    if (a.mode == FP8PA_SCALE_CHANNEL_STATIC) e = 0;
    job.sc *= exp2i(-e);
  }
  // Groups to keep; the others become zero.  In a tile that some row does
  // not see whole, a V that is not finite would reach rows that mask its token
  // (0 * NaN): it is zeroed and its token marked, for the rows that do see it.
  uint32_t keep = job.okm, bad = 0;
  if (V && !whole) {
    uint32_t nf = 0;  // bit x: this lane's chunks of group x
    if constexpr (FMT != FP8PA_INT8) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        bool f = false;
#pragma unroll
        for (int h = 0; h < H; ++h) f = f || codes_nonfinite<FMT>(job.buf[x][h]);
        nf |= f ? 1u << x : 0u;
      }
      nf |= __shfl_xor_sync(0xffffffffu, nf, 8);
      nf |= __shfl_xor_sync(0xffffffffu, nf, 16);
    }
    const uint32_t nfs = __ballot_sync(0xffffffffu, job.sok && !finite);  // by token
#pragma unroll
    for (int x = 0; x < 4; ++x) nf |= ((nfs >> (x * 8 + r8)) & 1u) << x;
    nf &= job.okm;
    keep &= ~nf;
#pragma unroll
    for (int x = 0; x < 4; ++x)  // lanes 0-7 hold the rows in order
      bad |= (__ballot_sync(0xffffffffu, (nf >> x) & 1u) & 0xFFu) << (8 * x);
  }
  if (lane == 0) {
    if (V) {
      info->ev[dw] = e;
      info->bad[dw] = bad;
    } else {
      info->ek[dw] = e;
      info->valid[dw] = valid;
    }
  }
  // K: core matrices (8 tokens x 8 dims) 128 bytes apart along the tokens,
  // 2048 along the dims; V: D * 16 along the tokens, 128 along the dims
  uint8_t* dst =
      tile + r8 * 16 + (V ? dw * (D * 64) + c4 * 256 : dw * 512 + c4 * 4096);
  const int kG = V ? D * 16 : 128, kC = V ? 4 * 256 : 4 * 4096, kH = V ? 128 : 2048;
  auto store = [&](int x, int h, const uint4& p, const uint4& q) {
    *reinterpret_cast<uint4*>(dst + x * kG + h * kC) = p;
    *reinterpret_cast<uint4*>(dst + x * kG + h * kC + kH) = q;
  };
  const bool plain = a.mode == FP8PA_SCALE_CHANNEL_STATIC;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    __half2 hi, lo;
    if constexpr (!MX) {
      const float f = __shfl_sync(0xffffffffu, job.sc, x * 8 + r8);
      const __half fh = __float2half_rn(f);
      hi = __half2half2(fh);
      lo = __half2half2(__float2half_rn(f - __half2float(fh)));
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      uint4 p, q;
      codes16_to_f16<FMT>(job.buf[x][h], p, q);
      if constexpr (MX) {
        // the block's power of two relative to the group's largest finite one (beyond
        // it, infinite)
        const int be = static_cast<int>((job.ex[h] >> (8 * x)) & 0xFFu) - 127 - e;
        const float f = __int_as_float((be > kRoom ? 255 : max(be, -126) + 127) << 23);
        const __half2 f2 = __floats2half2_rn(f, f);
        p = scale8(p, f2);
        q = scale8(q, f2);
      } else if (!plain) {
        p = scale8(p, hi, lo);
        q = scale8(q, hi, lo);
      }
      if (keep != 0xFu && ((keep >> x) & 1) == 0) p = q = make_uint4(0u, 0u, 0u, 0u);
      store(x, h, p, q);
    }
  }
}

// The work of one converting warp: jobs are dealt round robin over the warps.  A
// job's codes and scales are loaded as soon as the job before it is stored, its
// block ids one job earlier; kAhead jobs earlier it is asked for into L2, which
// is what keeps HBM busy where a chunk has few rows.
template <int D, int FMT, bool MX>
__device__ __forceinline__ void convert_tiles(const PrefillArgs& a, const PlanView& pv,
                                              uint8_t* sm, int* abort_flag, int it, int u, int u1,
                                              int first, int lane) {
  using SM = Smem<D>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SM::kBars);
  StageInfo* infos = reinterpret_cast<StageInfo*>(sm + SM::kInfo);
  const int lgbs = 31 - __clz(a.bs);  // block sizes are powers of two
  const int nbx = MX ? D / a.gs : 0;

  // the open item: tiles left of it, its block table, the tokens that some row
  // sees and those that every row sees
  int np = 0, skip = 0, k = 0, n = 0, kt = 0, kvh = 0, all_lo = 0, all_hi = 0;
  Seen seen{0, 0, 0};
  const int32_t* table = nullptr;
  auto token_of = [&](int i) { return (i < np ? i : i + skip) * kT; };
  auto load_ids = [&](int i, int part, int (&id)[2]) {
    job_blocks(table, lgbs, seen, token_of(i) + (part & 3) * 32, id);
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
      np = im.r.np;
      skip = im.r.skip;
      kvh = im.kvh;
      seen.pre = im.r.pre;
      table = a.block_tables + static_cast<long>(im.r.b) * a.max_blocks;
      seen.lo = window_first(a.window, im.r.pA);
      seen.hi = im.r.pB + 1;
      all_lo = window_first(a.window, im.r.pB);
      all_hi = im.r.pA + 1;
    }
    if (!have) load_ids(kt + k, part, ids);
    const bool V = part >= 4;
    const int dw = part & 3;
    const int j0 = token_of(kt + k), j = j0 + dw * 32;
    const bool whole = (j0 >= all_lo && j0 + kT <= all_hi) || j0 + kT <= seen.pre;
    Job<D> job;
    load_job<D, MX>(a, V, kvh, ids, j, seen, lane, job);
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
      const size_t row = cache_row(a, kvh, pf_blk, pf_t);
      prefetch_l2((pf_v ? a.v_cache : a.k_cache) + row * D, 16 * D);
      if (a.mode == FP8PA_SCALE_TOKEN_HEAD) prefetch_l2((pf_v ? a.v_scale : a.k_scale) + row, 64);
      else if (MX)
        prefetch_l2(reinterpret_cast<const uint8_t*>(pf_v ? a.v_scale : a.k_scale) + row * nbx,
                    16 * nbx);
    }
    pf_blk = -1;
    if (lane < 2) {
      const int ahead = part + kAhead * kConvWarps, ak = k + (ahead >> 3);
      if (ak < n) {
        pf_v = (ahead & 7) >= 4;
        pf_t = token_of(kt + ak) + (ahead & 3) * 32 + lane * 16;
        if ((pf_t < seen.hi && pf_t + 16 > seen.lo) || pf_t < seen.pre)
          pf_blk = __ldg(table + static_cast<int>(static_cast<uint32_t>(pf_t) >> lgbs));
      }
    }

    const uint32_t st = g & 1, s4 = g & 3;
    // The stage's last reader was the MMA of tile g - 2; the info stage's the
    // softmax of tile g - 4, whose P was waited for before that MMA.
    if (g >= 2 && !__all_sync(0xffffffffu,
                              tc_wait(bars + (V ? kBarVFree : kBarKFree) + st,
                                      ((g >> 1) - 1) & 1, abort_flag, a.err)))
      return;
    finish_job<D, FMT, MX>(a, job, V, dw, whole, sm + (V ? SM::kV : SM::kK) + st * SM::kTile,
                           infos + s4, lane);
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

// ---------------------------------------------------------------- ready tiles
// A chunk of many row blocks converts each tile once for all of them: one CTA per
// tile of a request and KV head, one warp per job, writes the tile as it lies in
// shared memory.  V that is not finite is marked in every tile, as each may be
// masked for some row.
template <int D, int FMT, bool MX>
__global__ void __launch_bounds__(256) ready_kernel(const __grid_constant__ PrefillArgs a,
                                                    const __grid_constant__ PlanView pv) {
  griddep_wait();
  griddep_launch_dependents();
  const int bh = blockIdx.x / pv.tpr, tile = blockIdx.x - bh * pv.tpr;
  const int b = bh / a.hkv, kvh = bh - b * a.hkv;
  bool bad_off, bad_len;
  const Chunk c = load_chunk(a, b, &bad_off, &bad_len);
  const Seen seen{window_first(a.window, c.L - c.n), c.L, c.pre};
  // the tiles of the request's row blocks (tile 0 for rows that see nothing)
  if (c.n == 0 || (tile * kT >= seen.pre && (tile < seen.lo / kT || tile * kT >= max(c.L, 1))))
    return;
  const int part = threadIdx.x >> 5, lane = threadIdx.x & 31, dw = part & 3;
  const bool V = part >= 4;
  const int j = tile * kT + dw * 32;
  int ids[2];
  job_blocks(a.block_tables + static_cast<long>(b) * a.max_blocks, 31 - __clz(a.bs), seen, j, ids);
  Job<D> job;
  load_job<D, MX>(a, V, kvh, ids, j, seen, lane, job);
  constexpr int kTile = Smem<D>::kTile;
  finish_job<D, FMT, MX>(a, job, V, dw, false,
                         pv.tiles + (static_cast<size_t>(blockIdx.x) * 2 + (V ? 1 : 0)) * kTile,
                         reinterpret_cast<StageInfo*>(pv.info) + blockIdx.x, lane);
}

// One thread's work: the K^ tiles of a CTA's range and their infos, or the V^
// tiles.  Its last copies are waited for, so that none is in flight at its end.
template <int D>
__device__ __forceinline__ void load_tiles(const PrefillArgs& a, const PlanView& pv, uint8_t* sm,
                                           int* abort_flag, int it, int u, int u1, bool V) {
  using SM = Smem<D>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SM::kBars);
  uint64_t* full = bars + (V ? kBarVFull : kBarKFull);
  uint64_t* free = bars + (V ? kBarVFree : kBarKFree);
  // the tiles were written by ordinary stores, before griddep_wait
  asm volatile("fence.proxy.async.global;" ::: "memory");
  uint32_t g = 0;
  bool ok = true;
  for (; u < u1 && ok; ++it) {
    const Item im = load_item(a, pv, it, u, u1);
    u += im.t1 - im.t0;
    const size_t base = static_cast<size_t>(im.r.b * a.hkv + im.kvh) * pv.tpr;
    for (int k = im.t0; k < im.t1; ++k, ++g) {
      const uint32_t st = g & 1, s4 = g & 3;
      // (an info's last reader: the softmax of tile g - 4, as in finish_job's order)
      ok = g < 2 || tc_wait(free + st, ((g >> 1) - 1) & 1, abort_flag, a.err);
      if (!ok) break;
      const size_t at = base + (k < im.r.np ? k : k + im.r.skip);
      if (!V) {
        mbar_arrive_expect_tx(bars + kBarScale + s4, sizeof(StageInfo));
        bulk_load(sm + SM::kInfo + s4 * sizeof(StageInfo), pv.info + at * sizeof(StageInfo),
                  sizeof(StageInfo), bars + kBarScale + s4);
      }
      mbar_arrive_expect_tx(full + st, SM::kTile);
      bulk_load(sm + (V ? SM::kV : SM::kK) + st * SM::kTile,
                pv.tiles + (at * 2 + (V ? 1 : 0)) * SM::kTile, SM::kTile, full + st);
    }
  }
  for (uint32_t x = g > 4 ? g - 4 : 0; x < g; ++x) {
    if (!V) (void)mbar_wait_bounded(bars + kBarScale + (x & 3), (x >> 2) & 1, kWaitLimitCycles);
    if (x + 2 >= g) (void)mbar_wait_bounded(full + (x & 1), (x >> 1) & 1, kWaitLimitCycles);
  }
}

// ---------------------------------------------------------------- kernel
// VAR: 0 no score modifier but the masks, 1 distance bias, 2 capped scores
// (with or without a bias).  MX: scales are exponents of MX blocks.  READY: over
// ready tiles, whatever the format.
template <int D, int FMT, int VAR, bool MX, bool READY>
__global__ void __launch_bounds__(kThreads<READY>, 1)
    prefill_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ PlanView pv) {
  using SM = Smem<D>;
  // used as it stands, so that its accesses stay in the shared space
  extern __shared__ __align__(128) uint8_t sm[];
  constexpr int kS = kStep<READY>, kSteps = kT / kS;
  constexpr int kHalf = kS / 2;    // tokens of a step that a softmax thread has,
  constexpr int kGroups = kHalf / 32;  // in groups of 32
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(sm + SM::kMisc);
  int& s_abort = *reinterpret_cast<int*>(sm + SM::kMisc + 4);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SM::kBars);
  StageInfo* infos = reinterpret_cast<StageInfo*>(sm + SM::kInfo);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  griddep_wait();
  griddep_launch_dependents();
  const int u0 = pv.start[blockIdx.x], u1 = pv.start[blockIdx.x + 1];
  if (u0 >= u1) return;
  const int it0 = pv.item[blockIdx.x];

  if (warp == kIssueWarp<READY>) tmem_alloc(&s_tmem, 512);
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bars + i, i >= kBarKFree                             ? 1
                          : i >= kBarX                               ? 2
                          : READY && i >= kBarScale                  ? 1
                          : i >= kBarKFull                           ? 4
                                                                     : 8);
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp<READY>) tmem_relinquish();
  const uint32_t tmem = s_tmem;
  int* abort_flag = &s_abort;
  auto wait = [&](int bar, uint32_t parity) {
    return tc_wait(bars + bar, parity, abort_flag, a.err);
  };
  // a wait of a whole warp: one answer for all lanes
  auto wait_warp = [&](int bar, uint32_t parity) {
    return __all_sync(0xffffffffu, tc_wait(bars + bar, parity, abort_flag, a.err)) != 0;
  };

  if (warp == kIssueWarp<READY>) {
    // ================================================= MMA issuer
    // S_t of a step goes where P_t was, kSteps steps before: it is issued behind
    // the P V that reads it, and the tensor cores work through one thread's MMAs in
    // the order of their issue.
    if (lane == 0) {
      const uint32_t idesc_s = tc_idesc(0, 0, 0, 0, 128, kS);  // f16, both K-major
      const uint32_t idesc_o = tc_idesc(0, 0, 0, 1, 128, D);      // A in TMEM, B MN-major
      const uint32_t base = smem_u32(sm);
      const uint64_t dq0 = tc_desc(base + SM::kQ, 2048, 128, 0);
      const uint64_t dk0 = tc_desc(base + SM::kK, 2048, 128, 0);
      const uint64_t dv0 = tc_desc(base + SM::kV, D * 16, 128, 0);
      constexpr uint32_t kNext = SM::kTile >> 4;  // the other row tile or stage
      auto mma_s = [&](int t, int step, uint32_t st) {  // S_t = Q_t K^T
        const uint64_t dq = dq0 + t * kNext, dk = dk0 + st * kNext + step * (kS * 16 >> 4);
        const uint32_t d = tmem + t * kT + step * kS;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma_f16(d, dq + k * (4096 >> 4), dk + k * (4096 >> 4), idesc_s, k > 0);
        tc_commit(bars + kBarS + t * 2 + step);
      };
      auto mma_o = [&](int t, int step, uint32_t st, bool first) {  // O_t += P_t V
        const uint64_t dv = dv0 + st * kNext + step * (kS / 8 * D * 16 >> 4);
        const uint32_t d = tmem + 256 + t * 128, p = tmem + t * kT + step * kS;
#pragma unroll
        for (int k = 0; k < kS / 16; ++k)  // the halves of P start kHalf columns apart
          tc_mma_f16_ts(d, p + k / (kS / 32) * kHalf + k % (kS / 32) * 8, dv + k * (2 * D * 16 >> 4), idesc_o,
                        !(first && k == 0));
        tc_commit(bars + kBarO + t * 2 + step);
      };
      uint32_t g = 0;           // tiles done by this CTA
      uint32_t nq = 0, np = 0;  // bit t: phase of row tile t's Q and P
      bool ok = true;
      for (int it = it0, u = u0; u < u1 && ok; ++it) {
        const Item im = load_item(a, pv, it, u, u1);
        const int n = im.t1 - im.t0;
        u += n;
        const int two = im.r.rows > 128 ? 2 : 1;
        ok = wait(kBarKFull + (g & 1), (g >> 1) & 1);
#pragma unroll 1
        for (int t = 0; t < two && ok; ++t) {  // the first tile's scores
          ok = wait(kBarQ + t, (nq >> t) & 1);
          if (!ok) break;
          nq ^= 1u << t;
          tc_fence_after();
          for (int step = 0; step < kSteps; ++step) mma_s(t, step, g & 1);
        }
        tc_commit(bars + kBarKFree + (g & 1));
        for (int k = 0; k < n && ok; ++k, ++g) {
          const bool more = k + 1 < n;
          ok = wait(kBarVFull + (g & 1), (g >> 1) & 1) &&
               (!more || wait(kBarKFull + ((g + 1) & 1), ((g + 1) >> 1) & 1));
#pragma unroll 1
          for (int x = 0; x < 2 * kSteps && ok; ++x) {
            const int step = x >> 1, t = x & 1;
            if (t >= two) continue;
            ok = wait(kBarP + t * 2 + step, (np >> t) & 1);
            if (!ok) break;
            if (step == kSteps - 1) np ^= 1u << t;
            tc_fence_after();
            mma_o(t, step, g & 1, k == 0 && step == 0);
            if (more) mma_s(t, step, (g + 1) & 1);
          }
          tc_commit(bars + kBarVFree + (g & 1));
          if (more) tc_commit(bars + kBarKFree + ((g + 1) & 1));
        }
      }
    }
  } else if (warp >= kConvWarp) {
    if constexpr (READY) {
      if (lane == 0) load_tiles<D>(a, pv, sm, abort_flag, it0, u0, u1, warp != kConvWarp);
    } else {
      convert_tiles<D, FMT, MX>(a, pv, sm, abort_flag, it0, u0, u1, warp - kConvWarp, lane);
    }
  } else {
    // ================================================= softmax warps
    const int t = warp >> 3, half = (warp >> 2) & 1;  // row tile, and half of a step's tokens
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
    uint32_t g = 0, ns = 0;  // tiles of the CTA, and of this row tile
    bool ok = true;
    for (int it = it0, u = u0; u < u1 && ok; ++it) {
      const Item im = load_item(a, pv, it, u, u1);
      const int n = im.t1 - im.t0;
      u += n;
      if (t == 1 && im.r.rows <= 128) {  // row tile 1 of a short block idles
        g += n;
        continue;
      }
      const int r = t * 128 + rl;  // row of the block
      const bool live = r < im.r.rows;
      // query and head of a row of the block (rows past its end: the last one's)
      auto query_of = [&](int row, int& qi, int& h) {
        const int rr = im.r.row0 + min(row, im.r.rows - 1);
        qi = rr / a.G;
        h = im.kvh * a.G + rr - qi * a.G;
      };
      int qi, h;
      query_of(r, qi, h);
      const long grow = (static_cast<long>(im.r.qlo) + qi) * a.hq + h;  // row of q and out
      float zs;
      {
        // ---- the rows of q, each normalised by a power of two, into shared
        // memory (every QK^T of the previous item is done: its last S was read).
        // A warp takes 16 of its 32 rows: 8 rows x 64 bytes per load, all loads
        // in flight at once, core matrices written free of bank conflicts.
        const float sgn = a.sm_scale < 0.f ? -1.f : 1.f;
        const bool st = a.mode == FP8PA_SCALE_CHANNEL_STATIC;
        const float* kc = a.k_scale + static_cast<long>(im.kvh) * D;
        const int r8 = lane & 7, c4 = lane >> 3;
        uint4 raw[2][D / 32];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          int qy, hy;
          query_of(t * 128 + (warp & 3) * 32 + (half * 2 + y) * 8 + r8, qy, hy);
          const uint4* src = reinterpret_cast<const uint4*>(
                                 a.q + ((static_cast<long>(im.r.qlo) + qy) * a.hq + hy) * D) + c4;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) raw[y][x] = __ldg(src + x * 4);
        }
        int eq[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          auto get = [&](int x, float (&f)[8]) {
            const uint32_t w[4] = {raw[y][x].x, raw[y][x].y, raw[y][x].z, raw[y][x].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[2 * e] = __uint_as_float(w[e] << 16) * sgn;
              f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u) * sgn;
            }
            if (st) {
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] *= __ldg(kc + (x * 4 + c4) * 8 + e);
            }
          };
          float amax = 0.f;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            float f[8];
            get(x, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
          }
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
          eq[y] = amax > 0.f ? exp_above(amax) : 0;
          const float fq = exp2i(14 - eq[y]);
          uint8_t* dst = sm + SM::kQ + t * SM::kTile + ((warp & 3) * 4 + half * 2 + y) * 128 +
                         r8 * 16 + c4 * 2048;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            float f[8];
            get(x, f);
            *reinterpret_cast<uint4*>(dst + x * 4 * 2048) =
                make_uint4(pack_half2(f[0] * fq, f[1] * fq), pack_half2(f[2] * fq, f[3] * fq),
                           pack_half2(f[4] * fq, f[5] * fq), pack_half2(f[6] * fq, f[7] * fq));
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kBarQ + t);
        // this lane's row: group lane / 8 of four, in this warp's half or the
        // other's
        float mine = static_cast<float>((lane >> 3) & 1 ? eq[1] : eq[0]), theirs;
        if (!trade(mine, theirs)) {
          ok = false;
          break;
        }
        const int er = static_cast<int>((lane >> 4) == half ? mine : theirs);
        // log2-domain factor of a raw score (capped scores: see cap_in)
        zs = fabsf(a.sm_scale) * exp2i(er - 14) * (VAR == 2 ? a.cap_in : kLog2e);
      }
      const int pos = im.r.L - im.r.n + qi;
      const int wf = window_first(a.window, pos);
      const int pre = im.r.pre;
      // extremes over the warp's rows (positions rise with the row)
      const int pA = __shfl_sync(0xffffffffu, pos, 0), wB = __shfl_sync(0xffffffffu, wf, 31);
      const float slope = (VAR > 0 && a.slopes) ? __ldg(a.slopes + h) * kLog2e : 0.f;
      const float cap_log2 = VAR == 2 ? a.cap * kLog2e : 0.f;
      float ref = kNegBig, l = 0.f;

      // An item's first scores are waited for before its first info: a row tile that
      // sat out the items before may be several phases of that barrier ahead, and a
      // parity tells only two apart.  Once the issuer is here, every earlier phase is
      // over, and the one after this waits for this row tile's P.
      ok = wait_warp(kBarS + t * 2, ns & 1);
      for (int x = 0; x < kSteps * n && ok; ++x) {
        const int step = x % kSteps, kt = im.t0 + x / kSteps;
        const uint32_t s4 = g & 3;
        const uint32_t sc = ts + step * kS;  // the thread's scores, then P
        const int j0 = (kt < im.r.np ? kt : kt + im.r.skip) * kT + step * kS + half * kHalf;
        if (step == 0 && !wait_warp(kBarScale + s4, (g >> 2) & 1)) {
          ok = false;
          break;
        }
        // the groups' factors, exponents and the tokens that the row sees
        const StageInfo& info = infos[s4];
        const int first = (step * kS + half * kHalf) / 32;
        float zw[kGroups], ev[kGroups];
        uint32_t m[kGroups], all = 0xFFFFFFFFu, nan = 0;
#pragma unroll
        for (int w = 0; w < kGroups; ++w) {
          ev[w] = static_cast<float>(info.ev[first + w]);
          // (VAR 0 multiplies a masked -inf by the factor: not zero)
          zw[w] = zs * exp2i(info.ek[first + w]);
          if (VAR == 0) zw[w] = fmaxf(zw[w], 1e-37f);
          m[w] = info.valid[first + w];
          all &= m[w];
        }
        // whether every row of the warp sees all of the thread's tokens
        const bool whole =
            ((j0 >= wB && j0 + kHalf - 1 <= pA) || (VAR == 0 && j0 + kHalf <= pre)) &&
            all == 0xFFFFFFFFu && (VAR < 2 || a.cap <= kCapFast);
#pragma unroll
        for (int w = 0; w < kGroups; ++w) {
          if (!whole)
            m[w] &= word_bits(j0 + w * 32, wf, pos + 1) | word_bits(j0 + w * 32, 0, pre);
          nan |= m[w] & info.bad[first + w];
        }
        if (nan) l = __int_as_float(0x7FC00000);
        if (!wait_warp(kBarS + t * 2 + step, ns & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // ---- a bound of z + e over the row's tokens.  The first group's scores stay
        // in registers (VAR > 0: as final scores), the second's in TMEM.
        uint32_t raw[2][16];
        float bound = __int_as_float(0xff800000);
        auto find = [&](auto masked, int w) {
          tmem_ld16(sc + w * 32, raw[0]);
          tmem_ld16(sc + w * 32 + 16, raw[1]);
          tmem_ld_wait();
          tmem_landed(raw[0]);
          tmem_landed(raw[1]);
          const int jw = j0 + w * 32;
          float m4[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) m4[y] = __int_as_float(0xff800000);
          // the bias of tokens 2 i, 2 i + 1 of the group: -slope (pos - j)
          // (VAR 2: and the cap, less what the tanh leaves of it)
          const float b0 = VAR > 0 ? fmaf(slope, static_cast<float>(jw - pos), cap_log2) : 0.f;
          const uint64_t zw2 = f2_pack(zw[w], zw[w]), bias = f2_pack(b0, b0 + slope);
          const uint64_t by2 = f2_pack(2.f * slope, 2.f * slope);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint32_t* r = &raw[i / 8][(i % 8) * 2];
            float y[2] = {__uint_as_float(r[0]), __uint_as_float(r[1])};
            if constexpr (VAR > 0) {
              if constexpr (masked.value) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                  y[v] *= zw[w];
                  if constexpr (VAR == 2) y[v] = a.cap * tanh_f32(y[v] * a.tanh_in) * kLog2e;
                  y[v] = fmaf(-slope, fabsf(static_cast<float>(pos - jw - 2 * i - v)), y[v]);
                }
              } else {
                const float fi = static_cast<float>(i);
                const uint64_t b = f2_fma(by2, f2_pack(fi, fi), bias);
                uint64_t z = f2_pack(y[0], y[1]);
                if constexpr (VAR == 1) {
                  z = f2_fma(z, zw2, b);
                } else {  // cap tanh(z / cap) = cap - 2 cap / (2^x + 1), cap in the bias
                  f2_unpack(f2_mul(z, zw2), y[0], y[1]);
                  f2_unpack(f2_add(f2_pack(ex2(y[0]), ex2(y[1])), f2_pack(1.f, 1.f)), y[0], y[1]);
                  z = f2_fma(f2_pack(rcp_fast(y[0]), rcp_fast(y[1])),
                             f2_pack(-2.f * cap_log2, -2.f * cap_log2), b);
                }
                f2_unpack(z, y[0], y[1]);
              }
            }
            if constexpr (masked.value) {
              y[0] = (m[w] >> (2 * i)) & 1 ? y[0] : __int_as_float(0xff800000);
              y[1] = (m[w] >> (2 * i + 1)) & 1 ? y[1] : __int_as_float(0xff800000);
            }
            m4[i & 3] = max3(m4[i & 3], y[0], y[1]);
            if constexpr (VAR > 0 || masked.value) {
              r[0] = __float_as_uint(y[0]);
              r[1] = __float_as_uint(y[1]);
            }
          }
          if ((VAR > 0 || masked.value) && w > 0) {
            tmem_st16(sc + w * 32, raw[0]);
            tmem_st16(sc + w * 32 + 16, raw[1]);
          }
          const float mx = max3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
          bound = fmaxf(bound, fmaf(mx, VAR > 0 ? 1.f : zw[w], ev[w]));
        };
#pragma unroll
        for (int w = kGroups - 1; w >= 0; --w) {
          if (whole) find(std::false_type{}, w);
          else find(std::true_type{}, w);
        }
        if (kGroups > 1 && (VAR > 0 || !whole)) tmem_st_wait();
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
          if (x > 0) {
            // behind P V of the step before: in the same columns, S of this step came
            // after it
            if (kSteps > 1 && !wait_warp(kBarO + t * 2 + (step ^ 1), (ns - (step ^ 1)) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              const uint32_t at = to + half * (D / 2) + c * 8;
              uint32_t o[8];
              tmem_ld8(at, o);
              tmem_ld_wait();
              tmem_landed(o);
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
              tmem_st8(at, o);
            }
          }
        }
        // ---- P (with the V^ group's exponent in it) and its sum (without)
#pragma unroll
        for (int w = 0; w < kGroups; ++w) {
          if (w > 0) {
            tmem_ld16(sc + w * 32, raw[0]);
            tmem_ld16(sc + w * 32 + 16, raw[1]);
            tmem_ld_wait();
            tmem_landed(raw[0]);
            tmem_landed(raw[1]);
          }
          const float c0 = kShift - ref + ev[w], f = VAR > 0 ? 1.f : zw[w];
          const uint64_t f2 = f2_pack(f, f), c02 = f2_pack(c0, c0);
          uint64_t la = 0, lb = 0;  // (0.f, 0.f)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint64_t z =
                  f2_pack(__uint_as_float(raw[c][2 * i]), __uint_as_float(raw[c][2 * i + 1]));
              float p, q;
              f2_unpack(VAR > 0 ? f2_add(z, c02) : f2_fma(z, f2, c02), p, q);
              p = ex2(p);
              q = ex2(q);
              if (i & 1) lb = f2_add(lb, f2_pack(p, q));
              else la = f2_add(la, f2_pack(p, q));
              pw[i] = pack_half2(p, q);
            }
            tmem_st8(sc + (w * 2 + c) * 8, pw);
          }
          float y, z;
          f2_unpack(f2_add(la, lb), y, z);
          l = fmaf(y + z, ex2(-ev[w]), l);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kBarP + t * 2 + step);
        if (step == kSteps - 1) {
          ++ns;
          ++g;
        }
      }
      if (!ok) break;

      // ---- the block's result, or this range's piece of it: half the dims each
      float other;
      if (!trade(l, other) || !wait_warp(kBarO + t * 2 + kSteps - 1, (ns - 1) & 1)) {
        ok = false;
        break;
      }
      l += other;
      tc_fence_after();
      const bool piece = im.t0 > 0 || im.t1 < im.r.count;
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
  if (warp == kIssueWarp<READY> && lane == 0) {
    tc_commit(bars + kBarDrain);
    (void)mbar_wait_bounded(bars + kBarDrain, 0, kWaitLimitCycles);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp<READY>) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- instances
template <int D, int FMT, bool MX, bool READY>
PrefillFn pick_var(int var) {
  return var == 0 ? prefill_kernel<D, FMT, 0, MX, READY>
                  : (var == 1 ? prefill_kernel<D, FMT, 1, MX, READY>
                              : prefill_kernel<D, FMT, 2, MX, READY>);
}
template <int D, int FMT, bool MX>
PrefillKernels pick_mx(int var, bool ready) {
  // over ready tiles the format no longer matters: one instance for all
  return {ready ? pick_var<D, FP8PA_E4M3, false, true>(var) : pick_var<D, FMT, MX, false>(var),
          ready ? ready_kernel<D, FMT, MX> : nullptr, Smem<D>::kBytes, ready ? kThreads<true> : kThreads<false>};
}
template <int D>
PrefillKernels pick_fmt(int fmt, int var, bool mx, bool ready) {
  if (fmt == FP8PA_INT8) return pick_mx<D, FP8PA_INT8, false>(var, ready);
  if (fmt == FP8PA_E4M3)
    return mx ? pick_mx<D, FP8PA_E4M3, true>(var, ready) : pick_mx<D, FP8PA_E4M3, false>(var, ready);
  return mx ? pick_mx<D, FP8PA_E5M2, true>(var, ready) : pick_mx<D, FP8PA_E5M2, false>(var, ready);
}

}  // namespace

}  // namespace fp8pa
