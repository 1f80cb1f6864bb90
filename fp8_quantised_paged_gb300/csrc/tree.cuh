// tree.cuh -- attention for trees of drafted tokens over the paged cache, on the
// fifth-generation tensor cores.
//
//   z_j = sm_scale q_i . k^_j;  z_j = cap tanh(z_j / cap);  z_j -= slope (pos_i - pos_j)
//   out_i = sum_j softmax(z)_j v^_j  over the tokens ahead of the tree (as the window and
//   the prefix leave them) and the nodes on i's line, itself among them
//
// Rows and work.  The (node, head) pairs of a request and KV head are rows, a TMEM lane
// each, in blocks of 128 (RAW false: 256); (row block, KV head, 128-token tile) units are cut
// into one range per SM, and cut items leave pieces, as in the prefill (ranges.cuh,
// prefill.cu).  A tree has few rows over a long context, so the cache's bytes bound it, and
// three things keep the tensor cores and the softmax out of their way:
//  - A block runs as two streams, one on the even tiles and one on the odd ones, with
//    scores, weights, sums and O of their own.
//  - A stream takes a tile by halves: while its softmax is at one half, the tensor cores
//    multiply the other half's weights and make the next tile's scores in its place.
//  - A block of at most 64 (or 32) rows stands twice (four times) in the lanes: each of the
//    copies weighs its share of a tile's tokens, with zeros for the others'.  The products
//    are the same, the softmax is half (a quarter).
// The partial results (1 to 8 a row) are added up at the block's end.  A block of more than
// 128 rows gives each stream 128 of its own, and every tile: what is converted serves twice
// the rows (64 nodes x 4 heads of 8 x 32K tokens, MX: 538-543 us; 559 where blocks of 128
// rows took 788).
// FP8 codes gain less by it, since K needs no converting and the second q takes the place of
// two of the four K tiles (12 x 16K, 64 nodes: 448 us against 498; a ragged batch of 64, 64
// nodes: 278 against 254; one request of 16K: 88 against 76), and keep to 128 rows.
//
// Measured (layer of 64 query and 8 KV heads of 128 dims, E4M3, a scale per token): 12 x 16K
// tokens and 16 nodes 146 us a call, 2.9 TB/s of the cache; one request of 700 tokens 28-31 us,
// which is the host's time (17.6 on the device, three dependent launches).  What bounds it is
// neither DRAM (44 % of its cycles at 12 x 16K) nor the tensor pipe (34 %) but the softmax, at
// half of the issue slots (51 %): its warps find S ready, and take 2650 cycles for half a tile
// (190 for a wait that is over, 1100 for the bound, 110 for the reference, 950 for P), so that
// an SM takes that for a tile of one of its two streams.  An item beside its tiles costs 17000
// cycles (q in two terms): 5000 until q stands in shared memory, 2000 until the first P, 8000
// for the sums.
// A suspend hint in the waits, scores held in registers between the passes (196-204 us, for
// spills) and two threads a lane (195 us) were no faster.
//
// Products.  S = Q K^T on FP8 tensor cores: the K codes as TMA lands them, q as two E4M3
// terms hi + lo (exact for bf16 but for elements 2^-9 below the row's largest), the token's
// scale multiplied to the fp32 score.  Static channel scales go into q, whose products with
// them have more bits: a third term keeps these to 2^-14 (two terms to 2^-9, where the f16 of
// other formats holds 2^-11).  O += P V on f16: V's codes are exact in f16, their
// scale goes into P in fp32 before its one rounding (2^-11).  So no code is rounded, and a
// K tile needs no converting.  INT8 codes and MX blocks (RAW false) are converted for both
// products: INT8 exactly, an MX block's codes times its power of two relative to the
// token's largest.
//
// References and sums as in the prefill: a row's reference is a bound of max(z + e), e the
// exponent of the token group's V scales, and moves only when passed by 2^kTau.
//
// Roles: warps 0-3 and 4-7 the softmax of streams 0 and 1, a thread a lane; four warps
// that convert V (RAW false: and four for K), one that issues MMAs for each stream, and
// (RAW) one that copies K's pages by TMA and lays out their scales, and one for V's.  RAW
// has 512 threads of 128 registers and spills 8 bytes at most; 576 of 96 spill some in the
// softmax, but six converting warps of 128 registers, 32-token jobs dealt among them, took 1735
// us where eight took 788.  Every wait is bounded.
#pragma once

#include "prefill.cuh"

namespace fp8pa {

// What the tree attention needs beside the prefill's arguments.
struct TreeView {
  const uint32_t* line;  // [total_q][8] the nodes on a node's line, as the window leaves them
  const int32_t* depth;  // [total_q]
  FastDiv div_g;         // by the heads of a KV head
};

using TreeFn = void (*)(const PrefillArgs, const PlanView, const TreeView, const CUtensorMap,
                        const CUtensorMap);
struct TreeKernel {
  TreeFn fn;
  int smem, threads;
};
// raw: FP8 codes with a scale per token, segment or channel (st).
TreeKernel pick_tree_d64(bool raw, bool st, int var);
TreeKernel pick_tree_d128(bool raw, bool st, int var);

namespace {

constexpr int kMaxTree = FP8PA_MAX_TREE;
constexpr int kLineWords = kMaxTree / 32;

constexpr int kTreeConv = 8;  // first converting warp
template <bool RAW>
constexpr int kTreeIssue = kTreeConv + (RAW ? 4 : 8);
template <bool RAW>
constexpr int kTreeThreads = (kTreeIssue<RAW> + (RAW ? 4 : 2)) * 32;

// Of a tile: its tokens' scales (V's relative to the 2^ev of their group of 32) and their
// positions behind the tokens ahead of the tree (for a distance bias), the groups'
// exponents, the tokens whose page exists (held: as V's copies say it), those whose V's
// scale is not finite, and, written with V in f16, those with codes that are not, where some
// row does not see the whole tile; the groups that every row sees whole; the first token,
// and what masks it.
struct TileInfo {
  float ks[kT], vs[kT], pos[kT];
  float ev[4];
  uint32_t valid[4], bad[4], held[4], cbad[4], seen[4];
  int j0, ctx, pre;
  uint32_t whole;
};
constexpr uint32_t kInfos = 8;  // stages
// Of a row: where its window begins, and its node's line.
struct RowMask {
  int wf, node;
};

template <int D, bool RAW>
struct TreeSmem {
  static constexpr int kHalf = 2 * kT * D;         // a 128-row f16 tile, or both terms of q
  static constexpr int kCodes = kT * D;            // a tile of codes
  static constexpr int kQ = 0;                     // q (RAW false: two tiles); between items, sums of O
  static constexpr int kV = (RAW ? 1 : 2) * kHalf;  // two tiles of V in f16
  static constexpr int kK = kV + 2 * kHalf;             // K: tiles of codes, or of f16
  static constexpr int kKTile = RAW ? kCodes : kHalf;
  // (an even number: a stage then serves one stream within an item)
  static constexpr int kKStages = RAW ? 4 : 2;
  static constexpr int kVCodes = kK + kKStages * kKTile;  // RAW: two tiles of V codes
  static constexpr int kInfo = kVCodes + (RAW ? 2 * kCodes : 0);
  static constexpr int kMl = kInfo + static_cast<int>(kInfos * sizeof(TileInfo));
  static constexpr int kRow = kMl + 2 * 128 * 8;   // [lane] RowMask (kMl: [stream][lane] float2)
  static constexpr int kExp = kRow + 256 * static_cast<int>(sizeof(RowMask));  // [lane] of q
  static constexpr int kBars = kExp + 256 * 4;
  static constexpr int kMisc = kBars + 320;        // TMEM base, abort flag
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kQ3 = (kBytes + 1023) / 1024 * 1024;  // the third term of q, if any
  static constexpr int kBytesThree = kQ3 + kCodes;
  static_assert((RAW ? kBytesThree : kBytes) <= 227 * 1024);
};
// Barriers and the arrivals that complete a phase: Q the eight softmax warps and the two
// issuers; P (stream * 2 + half) the stream's four; Info the copying warps (RAW) or the
// converting ones; K full one thread and its bytes (RAW) or four warps; V codes full a thread
// and its bytes, free the four converting warps; V full four warps; All the eight softmax
// warps; K and V free two commits of the tensor cores, one for each stream; S and O (stream *
// 2 + half) and Drain (by stream) one.
enum { kTQ = 0, kTP = 1, kTInfo = 5, kTKFull = 13, kTVCFull = 17, kTVCFree = 19, kTVFull = 21,
       kTAll = 23, kTKFree = 24, kTVFree = 28, kTS = 30, kTO = 34, kTDrain = 38, kTreeBars = 40 };
template <bool RAW>
__device__ __forceinline__ int tree_bar_count(int i) {
  return i < kTP        ? 10
         : i < kTInfo   ? 4
         : i < kTKFull  ? (RAW ? 2 : 8)
         : i < kTVCFull ? (RAW ? 1 : 4)
         : i < kTVCFree ? 1
         : i < kTAll    ? 4
         : i < kTKFree  ? 8
         : i < kTS      ? 2
                        : 1;
}

// The lanes of a share of a block's tokens (256: of both streams).
__device__ __forceinline__ int share_lanes(const RowBlock& r) {
  return r.rows <= 32 ? 32 : (r.rows <= 64 ? 64 : (r.rows <= 128 ? 128 : 256));
}

// Byte of chunk c (16 bytes) of row r in a tile of D-byte rows, as TMA's swizzle over D
// bytes places it.
template <int D>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// First token of tile x of a row block's list.  The list is walked from its end: with a
// distance bias the newest tokens weigh most, and a reference that starts there stays
// (rescaling O with every tile took 1700 cycles of 13000).
__device__ __forceinline__ int first_token(int np, int skip, int x) {
  return (x < np ? x : x + skip) * kT;
}

// What a converting warp's open item says of its tokens.
struct OpenItem {
  int np, skip, last, kvh, ctx, L, qlo, all_lo;
  Seen seen;
  const int32_t* table;
  __device__ __forceinline__ void open(const PrefillArgs& a, const Item& im) {
    np = im.r.np;
    skip = im.r.skip;
    last = im.r.count - 1;
    kvh = im.kvh;
    ctx = im.r.pA;
    L = im.r.L;
    qlo = im.r.qlo;
    all_lo = window_first(a.window, L - 1);
    seen = Seen{window_first(a.window, ctx), L, im.r.pre};
    table = a.block_tables + static_cast<long>(im.r.b) * a.max_blocks;
  }
  __device__ __forceinline__ int token_of(int tile) const { return first_token(np, skip, last - tile); }
  // whether every row sees the group of 32 tokens at jw, the whole tile at token j0
  __device__ __forceinline__ bool sees(int jw) const {
    return (jw >= all_lo && jw + 32 <= ctx) || jw + 32 <= seen.pre;
  }
  __device__ __forceinline__ bool whole(int j0) const {
    return (j0 >= all_lo && j0 + kT <= ctx) || j0 + kT <= seen.pre;
  }
};

// ---------------------------------------------------------------- copies (RAW)
// The scales of a tile, lane x those of tokens 4 x .. 4 x + 3 (of one page).
struct TileScales {
  float4 s;
  uint32_t ok;  // bits of the four: wanted, and their page exists
};
// pages: lane x holds the tile's page x.  whole: every row sees the whole tile.
template <bool V>
__device__ __forceinline__ TileScales load_scales(const PrefillArgs& a, const OpenItem& o,
                                                  int pages, int j0, bool whole, int lgbs,
                                                  int lane) {
  TileScales r;
  const int id = __shfl_sync(0xffffffffu, pages, (lane * 4) >> lgbs), j = j0 + lane * 4;
  const bool there = id >= 0 && id < a.num_blocks;
  uint32_t want = 0xFu;
  if (!whole) {
    want = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) want |= o.seen(j + i) ? 1u << i : 0u;
  }
  if (!V && want != 0 && !there) raise_error(a.err, FP8PA_DEVERR_BLOCK_RANGE);
  r.ok = there ? want : 0u;
  r.s = make_float4(1.f, 1.f, 1.f, 1.f);
  const float* scale = V ? a.v_scale : a.k_scale;
  if (there && a.mode == FP8PA_SCALE_TOKEN_HEAD) {
    r.s = __ldg(reinterpret_cast<const float4*>(scale + cache_row(a, o.kvh, id, j)));
  } else if (there && a.mode == FP8PA_SCALE_SEGMENT) {
    const float x = __ldg(scale + static_cast<size_t>(id) * a.hp + o.kvh);
    r.s = make_float4(x, x, x, x);
  }
  return r;
}
// Bits of 32 tokens from four of each of eight lanes, the same word in all eight.
__device__ __forceinline__ uint32_t group_bits(uint32_t four, int lane) {
  uint32_t w = four << (4 * (lane & 7));
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, s);
  return w;
}

// One warp for K or V: the pages of a CTA's tiles into its stages (lane x copies page x;
// pages that no row sees are not read), and its part of the tiles' infos.  Scales are
// loaded a tile ahead, block ids two.  (An info's last reader, the softmax of the stream's
// tile after g - 8, is over once S of tile g - 4 is, or the product with V of tile g - 6.)
template <int D, bool V>
__device__ __forceinline__ void copy_tiles(const PrefillArgs& a, const PlanView& pv,
                                           const TreeView& tv, uint8_t* sm, int* abort_flag,
                                           const CUtensorMap* map, int it, int u, int u1, int lane,
                                           bool bias) {
  using SM = TreeSmem<D, true>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SM::kBars);
  TileInfo* infos = reinterpret_cast<TileInfo*>(sm + SM::kInfo);
  constexpr uint32_t kS = V ? 2 : SM::kKStages;
  constexpr int kFull = V ? kTVCFull : kTKFull, kFree = V ? kTVCFree : kTKFree;
  const int per = kT / a.bs, lgbs = 31 - __clz(a.bs);
  const uint32_t bytes = a.bs * D;
  const float top = FLT_MAX / (a.fmt == FP8PA_E4M3 ? code_max<FP8PA_E4M3>()
                                                   : code_max<FP8PA_E5M2>());
  uint32_t g = 0;
  OpenItem o;
  bool ok = true;
  while (u < u1 && ok) {
    const Item im = load_item(a, pv, it, u, u1);
    ++it;
    u += im.t1 - im.t0;
    o.open(a, im);
    auto page_of = [&](int tile) {
      const int t = o.token_of(tile) + lane * a.bs;
      const bool want = tile < im.t1 && lane < per &&
                        ((t < o.seen.hi && t + a.bs > o.seen.lo) || t < o.seen.pre);
      return want ? __ldg(o.table + (t >> lgbs)) : -1;
    };
    int id = page_of(im.t0), id1 = page_of(im.t0 + 1);
    TileScales s = load_scales<V>(a, o, id, o.token_of(im.t0), o.whole(o.token_of(im.t0)), lgbs,
                                  lane);
    bool whole = o.whole(o.token_of(im.t0));
    for (int k = im.t0; k < im.t1; ++k, ++g) {
      const int j0 = o.token_of(k), here = id;
      const TileScales now = s;
      const bool all_rows = whole;
      id = id1;
      if (k + 1 < im.t1) {
        const int next = o.token_of(k + 1);
        whole = o.whole(next);
        s = load_scales<V>(a, o, id, next, whole, lgbs, lane);
      }
      id1 = page_of(k + 2);
      const bool have = here >= 0 && here < a.num_blocks;
      const uint32_t count = __popc(__ballot_sync(0xffffffffu, have)), st = g % kS;
      TileInfo* info = infos + g % kInfos;
      if (g >= kS &&
          !__all_sync(0xffffffffu, tc_wait(bars + kFree + st, (g / kS - 1) & 1, abort_flag, a.err))) {
        ok = false;
        break;
      }
      // the word of a lane's group, written by the first of its eight lanes
      const int grp = lane >> 3;
      const bool lead = (lane & 7) == 0;
      uint32_t held = 0xFFFFFFFFu;
      if (!__all_sync(0xffffffffu, now.ok == 0xFu)) held = group_bits(now.ok, lane);
      if (V) {  // what the converting warps need comes with the codes
        if (lead) info->held[grp] = held;
        if (lane == 0) info->whole = all_rows;
        __syncwarp();
      }
      if (lane == 0) mbar_arrive_expect_tx(bars + kFull + st, count * bytes);
      __syncwarp();
      if (have)
        tma_load_2d(sm + (V ? SM::kVCodes : SM::kK) + st * SM::kCodes + lane * bytes, map, 0,
                    (here * a.hkv + o.kvh) * a.bs, bars + kFull + st);
      const float x[4] = {now.s.x, now.s.y, now.s.z, now.s.w};
      float y[4];
      if constexpr (V) {
        // a scale counts as finite where its largest code is (append writes no others)
        uint32_t fin = 0;
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool f = x[i] <= top;  // (not for a NaN)
          fin |= f ? 1u << i : 0u;
          y[i] = f && (now.ok >> i) & 1u ? x[i] : 0.f;
          m = fmaxf(m, y[i]);
        }
#pragma unroll
        for (int i = 1; i < 8; i <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
        const int e = max(exp_above(m), kLowV);
        const float f = exp2i(-e);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] *= f;
        uint32_t bad = 0;
        if (__any_sync(0xffffffffu, (now.ok & ~fin) != 0)) bad = group_bits(now.ok & ~fin, lane);
        if (lead) {
          info->ev[grp] = static_cast<float>(e);
          info->bad[grp] = bad;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (now.ok >> i) & 1u ? x[i] : 0.f;
        if (bias) {
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = j0 + lane * 4 + i;
            p[i] = static_cast<float>(j < o.ctx || j >= o.L ? j - o.ctx
                                                            : __ldg(tv.depth + o.qlo + j - o.ctx));
          }
          reinterpret_cast<float4*>(info->pos)[lane] = make_float4(p[0], p[1], p[2], p[3]);
        }
        if (lead) {
          info->valid[grp] = held;
          info->seen[grp] = held == 0xFFFFFFFFu && (all_rows || o.sees(j0 + grp * 32));
        }
        if (lane == 0) {
          info->j0 = j0;
          info->ctx = o.ctx;
          info->pre = o.seen.pre;
        }
      }
      reinterpret_cast<float4*>(V ? info->vs : info->ks)[lane] = make_float4(y[0], y[1], y[2], y[3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + kTInfo + g % kInfos);
    }
  }
  if (lane == 0) {  // no copy is in flight at the end
    for (uint32_t x = g > kS ? g - kS : 0; x < g; ++x)
      (void)mbar_wait_bounded(bars + kFull + x % kS, (x / kS) & 1, kWaitLimitCycles);
  }
  __syncwarp();
}

// ---------------------------------------------------------------- conversions
// 2^e for e >= -149.
__device__ __forceinline__ float pow2_any(int e) {
  return __int_as_float(e >= -126 ? (e + 127) << 23 : (e >= -149 ? 1 << (e + 149) : 0));
}

// K's part of a tile's info, for the 32 tokens at j of group dw (a lane each).
__device__ __forceinline__ void put_k_info(const TreeView& tv, const OpenItem& o, TileInfo* info,
                                           int dw, int j, int lane, float scale, bool ok,
                                           bool bias) {
  const uint32_t valid = __ballot_sync(0xffffffffu, ok);
  info->ks[dw * 32 + lane] = scale;
  if (bias) {
    const int p = j + lane;
    info->pos[dw * 32 + lane] = static_cast<float>(
        p < o.ctx || p >= o.L ? p - o.ctx : __ldg(tv.depth + o.qlo + p - o.ctx));
  }
  if (lane == 0) {
    info->valid[dw] = valid;
    info->seen[dw] = o.sees(j) && valid == 0xFFFFFFFFu;
    if (dw == 0) {
      info->j0 = j;
      info->ctx = o.ctx;
      info->pre = o.seen.pre;
    }
  }
}
// V's part; bad: bits of the tokens whose codes are not finite.  A scale counts as finite
// where its largest code is (append writes no others).
template <int FMT>
__device__ __forceinline__ void put_v_info(TileInfo* info, int dw, int lane, float scale, bool ok,
                                           uint32_t bad) {
  const bool finite = scale <= FLT_MAX / code_max<FMT>();  // (not for a NaN)
  const int e = max(exp_above(warp_max_f32(ok && finite ? scale : 0.f)), kLowV);
  info->vs[dw * 32 + lane] = ok && finite ? scale * exp2i(-e) : 0.f;
  bad |= __ballot_sync(0xffffffffu, ok && !finite);
  if (lane == 0) {
    info->ev[dw] = static_cast<float>(e);
    info->bad[dw] = bad;
  }
}

// 32 tokens of a tile and KV head, by one warp: a lane holds row r8 = lane % 8 of four
// 8-row groups and, of each, the 16-byte chunks lane / 8 (and 4 more), as the prefill's
// Job, but has the exponents of its rows from memory and not from other lanes.
template <int D>
struct Codes {
  uint4 buf[4][D / 64];
  uint32_t okm;    // groups whose row is wanted and exists
  uint2 ex[4];     // MX: the exponents of the rows' blocks
  float sc;        // scale of token `lane`
  bool sok;        // ... which is wanted and exists
};
template <int D, bool MX>
__device__ __forceinline__ void load_codes(const PrefillArgs& a, const OpenItem& o, bool V,
                                           const int (&ids)[2], int j, int lane, Codes<D>& c) {
  const int r8 = lane & 7, c4 = lane >> 3;
  const uint8_t* cache = V ? a.v_cache : a.k_cache;
  const float* scale = V ? a.v_scale : a.k_scale;
  const bool there[2] = {ids[0] >= 0 && ids[0] < a.num_blocks,
                         ids[1] >= 0 && ids[1] < a.num_blocks};
  // (a missing block's rows read as block 0's: not used)
  const uint32_t row[2] = {there[0] ? cache_row(a, o.kvh, ids[0], j) : 0u,
                           there[1] ? cache_row(a, o.kvh, ids[1], j + 16) : 0u};
  c.okm = 0;
  const int nbx = MX ? D / a.gs : 0;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint32_t rw = row[x >> 1] + (x & 1) * 8 + r8;
    const uint8_t* src = cache + static_cast<size_t>(rw) * D + c4 * 16;
#pragma unroll
    for (int h = 0; h < D / 64; ++h) c.buf[x][h] = ld_codes(src + h * 64);
    if (o.seen(j + x * 8 + r8) && there[x >> 1]) c.okm |= 1u << x;
    if constexpr (MX) {
      const uint8_t* e = reinterpret_cast<const uint8_t*>(scale) + static_cast<size_t>(rw) * nbx;
      c.ex[x] = make_uint2(0u, 0u);
      if (nbx == 8) c.ex[x] = __ldg(reinterpret_cast<const uint2*>(e));
      else if (nbx == 4) c.ex[x].x = __ldg(reinterpret_cast<const uint32_t*>(e));
      else c.ex[x].x = __ldg(reinterpret_cast<const uint16_t*>(e));
    }
  }
  const bool want = o.seen(j + lane);
  c.sok = want && (lane < 16 ? there[0] : there[1]);
  if (!V && want && !c.sok) raise_error(a.err, FP8PA_DEVERR_BLOCK_RANGE);
  c.sc = 1.f;
  if (a.mode == FP8PA_SCALE_TOKEN_HEAD)
    c.sc = __ldg(scale + (lane < 16 ? row[0] : row[1]) + (lane & 15));
  else if (a.mode == FP8PA_SCALE_SEGMENT && c.sok)
    c.sc = __ldg(scale + static_cast<size_t>(lane < 16 ? ids[0] : ids[1]) * a.hp + o.kvh);
}

// The tokens of a job of V whose codes are not all finite (bits of the 32); their rows are
// taken out of job.okm.
template <int D, int FMT>
__device__ __forceinline__ uint32_t drop_nonfinite(Codes<D>& job, int lane) {
  if constexpr (FMT == FP8PA_INT8) return 0;
  uint32_t nf = 0, bad = 0;  // bit x of nf: this lane's chunks of row group x
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    bool f = false;
#pragma unroll
    for (int h = 0; h < D / 64; ++h) f = f || codes_nonfinite<FMT>(job.buf[x][h]);
    nf |= f ? 1u << x : 0u;
  }
  nf |= __shfl_xor_sync(0xffffffffu, nf, 8);
  nf |= __shfl_xor_sync(0xffffffffu, nf, 16);
  nf &= job.okm;
  job.okm &= ~nf;
#pragma unroll
  for (int x = 0; x < 4; ++x)  // lanes 0-7 hold the rows in order
    bad |= (__ballot_sync(0xffffffffu, (nf >> x) & 1u) & 0xFFu) << (8 * x);
  return bad;
}

// A job's codes as f16 into a tile; rows of V that are not in job.okm are zero.
template <int D, int FMT, bool MX>
__device__ __forceinline__ void put_tile(const Codes<D>& job, bool V, int dw, int gs,
                                         uint8_t* tile, int lane) {
  constexpr int H = D / 64;
  constexpr int kRoom = FMT == FP8PA_E5M2 ? 0 : 7;
  const int r8 = lane & 7, c4 = lane >> 3;
  // core matrices as in the prefill's tiles
  uint8_t* dst =
      tile + r8 * 16 + (V ? dw * (D * 64) + c4 * 256 : dw * 512 + c4 * 4096);
  const int kG = V ? D * 16 : 128, kC = V ? 4 * 256 : 4 * 4096, kH = V ? 128 : 2048;
  const bool drop = V && !__all_sync(0xffffffffu, job.okm == 0xFu);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    int top = 0;  // the row's largest exponent
    if constexpr (MX) top = static_cast<int>(max_byte(reinterpret_cast<const uint32_t(&)[2]>(job.ex[x])));
#pragma unroll
    for (int h = 0; h < H; ++h) {
      uint4 p, q;
      codes16_to_f16<FMT>(job.buf[x][h], p, q);
      if constexpr (MX) {
        const int b = (h * 4 + c4) * 16 / gs;
        const uint32_t e = (b & 4 ? job.ex[x].y : job.ex[x].x) >> (8 * (b & 3)) & 0xFFu;
        const float f = exp2i(static_cast<int>(e) - top + kRoom);
        const __half2 f2 = __floats2half2_rn(f, f);
        p = scale8(p, f2);
        q = scale8(q, f2);
      }
      if (drop && ((job.okm >> x) & 1) == 0) p = q = make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(dst + x * kG + h * kC) = p;
      *reinterpret_cast<uint4*>(dst + x * kG + h * kC + kH) = q;
    }
  }
}

// RAW: a warp's 32 tokens of each of n tiles, V's codes from the copied stage into the f16
// tile.
template <int D, int FMT>
__device__ __forceinline__ void convert_raw(const PrefillArgs& a, uint8_t* sm, int* abort_flag,
                                            uint32_t n, int dw, int lane) {
  using SM = TreeSmem<D, true>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SM::kBars);
  TileInfo* infos = reinterpret_cast<TileInfo*>(sm + SM::kInfo);
  const int r8 = lane & 7, c4 = lane >> 3;
  for (uint32_t g = 0; g < n; ++g) {
    const uint32_t st = g & 1;
    if (!__all_sync(0xffffffffu, tc_wait(bars + kTVCFull + st, (g >> 1) & 1, abort_flag, a.err)))
      return;
    Codes<D> job;
    const uint8_t* src = sm + SM::kVCodes + st * SM::kCodes;
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        job.buf[x][h] = *reinterpret_cast<const uint4*>(
            src + swizzled<D>(dw * 32 + x * 8 + r8, c4 + h * 4));
    TileInfo* info = infos + g % kInfos;
    const uint32_t held = info->held[dw];
    const bool whole = info->whole;
    // the codes are in registers before the next copy may land on them: without the fence
    // copies from L2 overtook these loads (in every call of 8 trees over 2500 tokens)
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + kTVCFree + st);
    job.okm = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) job.okm |= ((held >> (x * 8 + r8)) & 1u) << x;
    const uint32_t bad = whole ? 0u : drop_nonfinite<D, FMT>(job, lane);
    if (g >= 2 && !__all_sync(0xffffffffu, tc_wait(bars + kTVFree + st, ((g >> 1) - 1) & 1,
                                                   abort_flag, a.err)))
      return;
    put_tile<D, FMT, false>(job, true, dw, 0, sm + SM::kV + st * SM::kHalf, lane);
    if (lane == 0) info->cbad[dw] = bad;
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + kTVFull + st);
  }
}

// RAW false: a warp's 32 tokens of K or of V of every tile, from the cache into the f16
// tile; a tile kAhead on is asked for into L2.
template <int D, int FMT, bool MX>
__device__ __forceinline__ void convert_loaded(const PrefillArgs& a, const PlanView& pv,
                                               const TreeView& tv, uint8_t* sm, int* abort_flag,
                                               int it, int u, int u1, int part, int lane,
                                               bool bias) {
  using SM = TreeSmem<D, false>;
  constexpr int kRoom = FMT == FP8PA_E5M2 ? 0 : 7;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SM::kBars);
  TileInfo* infos = reinterpret_cast<TileInfo*>(sm + SM::kInfo);
  const int lgbs = 31 - __clz(a.bs), dw = part & 3, nbx = MX ? D / a.gs : 0;
  const bool V = part >= 4;
  uint32_t g = 0;
  OpenItem o;
  while (u < u1) {
    const Item im = load_item(a, pv, it, u, u1);
    ++it;
    u += im.t1 - im.t0;
    o.open(a, im);
    int ids[2];
    job_blocks(o.table, lgbs, o.seen, o.token_of(im.t0) + dw * 32, ids);
    for (int k = im.t0; k < im.t1; ++k, ++g) {
      const uint32_t st = g & 1, si = g % kInfos;
      const int j0 = o.token_of(k), j = j0 + dw * 32;
      Codes<D> job;
      load_codes<D, MX>(a, o, V, ids, j, lane, job);
      if (k + 1 < im.t1) job_blocks(o.table, lgbs, o.seen, o.token_of(k + 1) + dw * 32, ids);
      if (lane < 2 && k + kAhead < im.t1) {
        const int t = o.token_of(k + kAhead) + dw * 32 + lane * 16;
        const int id = (t < o.seen.hi && t + 16 > o.seen.lo) || t < o.seen.pre
                           ? __ldg(o.table + (t >> lgbs)) : -1;
        if (id >= 0 && id < a.num_blocks) {
          const size_t row = cache_row(a, o.kvh, id, t);
          prefetch_l2((V ? a.v_cache : a.k_cache) + row * D, 16 * D);
          if (a.mode == FP8PA_SCALE_TOKEN_HEAD) prefetch_l2((V ? a.v_scale : a.k_scale) + row, 64);
          else if (MX)
            prefetch_l2(reinterpret_cast<const uint8_t*>(V ? a.v_scale : a.k_scale) + row * nbx,
                        16 * nbx);
        }
      }
      float scale = job.sc;
      if constexpr (MX) {  // of token `lane`: this lane's row of group c4
        const uint2 e = lane < 16 ? (lane < 8 ? job.ex[0] : job.ex[1])
                                  : (lane < 24 ? job.ex[2] : job.ex[3]);
        const int top = static_cast<int>(max_byte(reinterpret_cast<const uint32_t(&)[2]>(e)));
        scale = top == 255 ? __int_as_float(0x7FC00000) : pow2_any(top - 127 - kRoom);
      }
      // V's info goes first, as S waits for it.  (An info's last reader, the softmax of the
      // stream's tile after g - 8, came before the waits of tiles before.)
      TileInfo* info = infos + si;
      if (V) {
        const uint32_t bad = o.whole(j0) ? 0u : drop_nonfinite<D, FMT>(job, lane);
        put_v_info<FMT>(info, dw, lane, scale, job.sok, bad);
        if (lane == 0) info->cbad[dw] = 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kTInfo + si);
      }
      if (g >= 2 && !__all_sync(0xffffffffu, tc_wait(bars + (V ? kTVFree : kTKFree) + st,
                                                     ((g >> 1) - 1) & 1, abort_flag, a.err)))
        return;
      put_tile<D, FMT, MX>(job, V, dw, a.gs, sm + (V ? SM::kV : SM::kK) + st * SM::kHalf, lane);
      if (!V) put_k_info(tv, o, info, dw, j, lane, scale, job.sok, bias);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        if (!V) mbar_arrive(bars + kTInfo + si);
        mbar_arrive(bars + (V ? kTVFull : kTKFull) + st);
      }
    }
  }
}

// The tokens of group w of a tile that a row sees: the window and the prefix ahead of the
// tree, and the nodes on its line.  Out of line, with all that it needs in shared memory:
// few groups are not seen whole, and registers are short.
__device__ __noinline__ uint32_t seen_bits(const TileInfo* info, int w, const RowMask* row,
                                           const uint32_t* lines) {
  const int jw = info->j0 + w * 32, ctx = info->ctx;
  uint32_t see = word_bits(jw, row->wf, ctx) | word_bits(jw, 0, info->pre);
  const int o = jw - ctx;  // the first token as a node
  if (o > -32) {
    const uint32_t* line = lines + static_cast<long>(row->node) * kLineWords;
    const int w0 = max(o, 0) >> 5;
    if (o < 0) see |= __ldg(line) << (-o);
    else if (w0 < kLineWords)
      see |= __funnelshift_r(__ldg(line + w0), w0 + 1 < kLineWords ? __ldg(line + w0 + 1) : 0u,
                             o & 31);
  }
  return see & info->valid[w];
}
// Whether a row saw, among the groups of a set, codes of V that are not finite.
__device__ __noinline__ bool saw_nan(const TileInfo* info, uint32_t groups, const RowMask* row,
                                     const uint32_t* lines) {
  uint32_t bad = 0;
  for (int w = 0; w < 4; ++w)
    if (((groups >> w) & 1u) != 0 && info->cbad[w] != 0)
      bad |= info->cbad[w] & seen_bits(info, w, row, lines);
  return bad != 0;
}

// 32 registers that a tcgen05.ld filled: what uses them stays behind the wait before this.
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[32]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]));
  asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

__device__ __forceinline__ uint64_t u2_pack(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}

// One lane of a whole warp, the same each time.  Under a branch on it the operands of an MMA
// stay in uniform registers; under one on the lane's number each costs a move, and eight
// MMAs take 930 cycles to issue beside busy warps.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// ---------------------------------------------------------------- kernel
// VAR: 0 no score modifier but the masks, 1 distance bias, 2 capped scores (with or
// without a bias).  THREE: q in three terms, for static channel scales (RAW), 4-5 % slower
// than two (12 x 16K, E4M3: 153 us, 147; ragged 64, E5M2: 206, 199), so an instance of its own: a
// branch on the mode cost calls with token scales 2 % as well (ragged 64, E4M3: 232 us, 227).
template <int D, bool RAW, int VAR, bool THREE>
__global__ void __launch_bounds__(kTreeThreads<RAW>, 1)
    tree_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ PlanView pv,
                const __grid_constant__ TreeView tv, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv) {
  using SM = TreeSmem<D, RAW>;
  // (the swizzled tiles start at multiples of 1024 bytes)
  extern __shared__ __align__(1024) uint8_t tree_sm[];
  uint8_t* const sm = tree_sm;
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(sm + SM::kMisc);
  int& s_abort = *reinterpret_cast<int*>(sm + SM::kMisc + 4);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SM::kBars);
  TileInfo* infos = reinterpret_cast<TileInfo*>(sm + SM::kInfo);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kIssue = kTreeIssue<RAW>;

  griddep_wait();
  griddep_launch_dependents();
  const int u0 = pv.start[blockIdx.x], u1 = pv.start[blockIdx.x + 1];
  if (u0 >= u1) return;
  const int it0 = pv.item[blockIdx.x];

  if (warp == kIssue) tmem_alloc(&s_tmem, 512);
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < kTreeBars; ++i) mbar_init(bars + i, tree_bar_count<RAW>(i));
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssue) tmem_relinquish();
  const uint32_t tmem = s_tmem;
  int* abort_flag = &s_abort;
  // a wait of a whole warp: one answer for all lanes
  auto wait_warp = [&](int bar, uint32_t parity) {
    return __all_sync(0xffffffffu, tc_wait(bars + bar, parity, abort_flag, a.err)) != 0;
  };

  if (warp >= kIssue && warp < kIssue + 2) {
    // ================================================= MMA issuers
    // A warp for each stream, so that neither waits behind the other's barriers.  TMEM: S at
    // 0 and 128, O at 256 and 384; a half of a tile has 64 columns of S, and its P lies in
    // them, so that the next S waits for the product with V: products of different kinds
    // and accumulators keep no order of their own.
    const int t = __shfl_sync(0xffffffffu, warp - kIssue, 0);
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(sm), 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t idesc_s = RAW ? tc_idesc(0, a.fmt == FP8PA_E5M2 ? 1 : 0, 0, 0, 128, kT / 2)
                                 : tc_idesc(0, 0, 0, 0, 128, kT / 2);
    const uint32_t idesc_o = tc_idesc(0, 0, 0, 1, 128, D);  // A in TMEM, B MN-major
    const uint64_t dv0 = tc_desc(base + SM::kV, D * 16, 128, 0);
    const uint64_t dq0 = RAW ? tc_desc(base + SM::kQ, 16, D * 8, D == 128 ? 2 : 4)
                             : tc_desc(base + SM::kQ, 2048, 128, 0);
    const uint64_t dk0 = RAW ? tc_desc(base + SM::kK, 16, D * 8, D == 128 ? 2 : 4)
                             : tc_desc(base + SM::kK, 2048, 128, 0);
    const uint32_t ds0 = tm + t * kT, d_o = tm + 256 + t * 128;
    uint32_t g = 0, nq = 0, np = 0;  // tiles before the item; items; tiles of the stream
    bool ok = true;
    int wide = 0;
    auto free_stage = [&](int bar) {  // a stream that has the tile to itself speaks for both
      tc_commit(bars + bar);
      if (!wide) tc_commit(bars + bar);
    };
    auto mma_s = [&](uint32_t st, int h) {
      const uint64_t dq = dq0 + (wide ? t * (SM::kHalf >> 4) : 0);
      const uint64_t dk = dk0 + st * (SM::kKTile >> 4) + h * (RAW ? kT / 2 * D >> 4 : 1024 >> 4);
      const uint32_t ds = ds0 + h * (kT / 2);
      if (elect_one()) {
        if constexpr (RAW) {
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              tc_mma_f8(ds, dq + term * (SM::kCodes >> 4) + k * 2, dk + k * 2, idesc_s,
                        (term | k) != 0);
          if constexpr (THREE) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              tc_mma_f8(ds, dq + ((SM::kQ3 - SM::kQ) >> 4) + k * 2, dk + k * 2, idesc_s, true);
          }
        } else {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc_mma_f16(ds, dq + k * (4096 >> 4), dk + k * (4096 >> 4), idesc_s, k > 0);
        }
        tc_commit(bars + kTS + t * 2 + h);
        if (h == 1) free_stage(kTKFree + st);
      }
      __syncwarp();
    };
    auto mma_o = [&](uint32_t st, int h, bool first) {
      const uint64_t dv = dv0 + st * (SM::kHalf >> 4) + h * (kT / 2 * D * 2 >> 4);
      const uint32_t p = ds0 + h * (kT / 2);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kT / 32; ++k)  // the groups of P start 32 columns apart
          tc_mma_f16_ts(d_o, p + (k >> 1) * 32 + (k & 1) * 8, dv + k * (2 * D * 16 >> 4), idesc_o,
                        !(first && k == 0));
        tc_commit(bars + kTO + t * 2 + h);
        if (h == 1) free_stage(kTVFree + st);
      }
      __syncwarp();
    };
    auto wait_s = [&](uint32_t x) {  // what S of tile x needs
      return wait_warp(kTKFull + x % SM::kKStages, (x / SM::kKStages) & 1) &&
             wait_warp(kTInfo + x % kInfos, (x / kInfos) & 1);
    };
    for (int it = it0, u = u0; u < u1 && ok; ++it) {
      const Item im = load_item(a, pv, it, u, u1);
      const int n = __shfl_sync(0xffffffffu, im.t1 - im.t0, 0);
      u += n;
      // q first, and every item's: once it is there, every tile before the item is over, and
      // a parity of the barriers below can mean no phase but its own (later ones follow its
      // own, as the stages are even in number).  The issuer arrives there itself: one that
      // has no tile in some items would otherwise hold none of them back, and q of two more
      // could pass it by.
      if (elect_one()) mbar_arrive(bars + kTQ);
      __syncwarp();
      ok = wait_warp(kTQ, nq & 1);
      ++nq;
      wide = __shfl_sync(0xffffffffu, !RAW && im.r.rows > 128, 0);
      const int k0 = wide ? 0 : t, step = wide ? 1 : 2;
      if (ok && k0 < n) {
        ok = wait_s(g + k0);
        if (!ok) break;
        tc_fence_after();
        mma_s((g + k0) % SM::kKStages, 0);
        mma_s((g + k0) % SM::kKStages, 1);
      }
      for (int k = k0; k < n && ok; k += step, ++np) {
        const uint32_t gk = g + k, gn = gk + step;
        const bool more = k + step < n;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          if (h == 0) ok = wait_warp(kTVFull + (gk & 1), (gk >> 1) & 1);
          ok = ok && wait_warp(kTP + t * 2 + h, np & 1);
          if (!ok) break;
          tc_fence_after();
          mma_o(gk & 1, h, k == k0 && h == 0);
          if (!more) continue;
          if (h == 0) ok = wait_s(gn);
          ok = ok && wait_warp(kTO + t * 2 + h, np & 1);
          if (!ok) break;
          tc_fence_after();
          mma_s(gn % SM::kKStages, h);
        }
      }
      g += n;
    }
  } else if (RAW && warp >= kIssue + 2) {
    if constexpr (RAW) {
      constexpr bool bias = VAR > 0;
      if (warp == kIssue + 2)
        copy_tiles<D, false>(a, pv, tv, sm, abort_flag, &mk, it0, u0, u1, lane, bias);
      else
        copy_tiles<D, true>(a, pv, tv, sm, abort_flag, &mv, it0, u0, u1, lane, bias);
    }
  } else if (warp >= kTreeConv) {
    const int part = warp - kTreeConv;
    if constexpr (RAW) {
      if (a.fmt == FP8PA_E4M3)
        convert_raw<D, FP8PA_E4M3>(a, sm, abort_flag, u1 - u0, part, lane);
      else
        convert_raw<D, FP8PA_E5M2>(a, sm, abort_flag, u1 - u0, part, lane);
    } else {
      constexpr bool bias = VAR > 0;
      if (a.fmt == FP8PA_INT8)
        convert_loaded<D, FP8PA_INT8, false>(a, pv, tv, sm, abort_flag, it0, u0, u1, part, lane,
                                             bias);
      else if (a.fmt == FP8PA_E4M3)
        convert_loaded<D, FP8PA_E4M3, true>(a, pv, tv, sm, abort_flag, it0, u0, u1, part, lane,
                                            bias);
      else
        convert_loaded<D, FP8PA_E5M2, true>(a, pv, tv, sm, abort_flag, it0, u0, u1, part, lane,
                                            bias);
    }
  } else {
    // ================================================= softmax warps
    const int t = warp >> 2;                // stream
    const int rl = (warp & 3) * 32 + lane;  // lane of the tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + t * kT + lanes, to = tmem + 256 + t * 128 + lanes;
    float2* ml = reinterpret_cast<float2*>(sm + SM::kMl);
    int* exps = reinterpret_cast<int*>(sm + SM::kExp);
    const bool cap_quick = a.cap <= kCapFast;
    constexpr int kTop = RAW ? 8 : 14;  // exponent of a normalised row of q
    uint32_t na = 0;
    auto sync_all = [&]() {  // all softmax warps
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + kTAll);
      const bool good = wait_warp(kTAll, na & 1);
      ++na;
      return good;
    };
    uint32_t g = 0, ns = 0;  // tiles of the CTA, and of this stream
    bool ok = true;
    for (int it = it0, u = u0; u < u1 && ok; ++it) {
      const Item im = load_item(a, pv, it, u, u1);
      const int n = im.t1 - im.t0;
      u += n;
      const int sl = share_lanes(im.r);
      // rows of two tiles of lanes: each stream has its own, and every token tile
      const bool wide = !RAW && sl == 256;
      const int mine = wide ? n : (n + 1 - t) >> 1;  // tiles of this stream
      const uint32_t g0 = wide ? g : g + t, step = wide ? 1 : 2;
      const int bl = wide ? t * 128 + rl : rl;  // lane of the block
      RowMask* const row = reinterpret_cast<RowMask*>(sm + SM::kRow) + bl;
      // query and head of a lane's row (lanes past the block's end: its last row)
      auto query_of = [&](int l, int& qi, int& h) {
        const int rr = im.r.row0 + min(l & (sl - 1), im.r.rows - 1);
        qi = static_cast<int>(fast_div(static_cast<uint32_t>(rr), tv.div_g));
        h = im.kvh * a.G + rr - qi * a.G;
      };
      {
        // ---- the rows of q, each normalised by a power of two, into shared memory (every S
        // of the item before was read), 8 rows x 64 bytes of a warp a load
        const float sgn = a.sm_scale < 0.f ? -1.f : 1.f;
        const bool st = a.mode == FP8PA_SCALE_CHANNEL_STATIC;
        const float* kc = a.k_scale + static_cast<long>(im.kvh) * D;
        const int r8 = lane & 7, c4 = lane >> 3;
        // (a turn at a time: rows asked for a turn ahead, or two turns laid out, were slower, 203
        // and 200 us against 197 for the ragged 64)
#pragma unroll 1
        for (int y = 0; y < (wide ? 4 : 2); ++y) {
          const int of_block = (warp * (wide ? 4 : 2) + y) * 8 + r8, to_row = of_block & 127;
          uint8_t* dst = sm + SM::kQ + (of_block >> 7) * SM::kHalf;
          int qy, hy;
          query_of(of_block, qy, hy);
          const uint4* src = reinterpret_cast<const uint4*>(
                                 a.q + ((static_cast<long>(im.r.qlo) + qy) * a.hq + hy) * D) + c4;
          uint4 raw[D / 32];
#pragma unroll
          for (int x = 0; x < D / 32; ++x) raw[x] = __ldg(src + x * 4);
          float f[D / 32][8], amax = 0.f;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[x][2 * e] = __uint_as_float(w[e] << 16) * sgn;
              f[x][2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u) * sgn;
            }
            if (st) {
              const float4* k8 = reinterpret_cast<const float4*>(kc + (x * 4 + c4) * 8);
              const float4 k0 = __ldg(k8), k1 = __ldg(k8 + 1);
              const float k[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) f[x][e] *= k[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[x][e]));
          }
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
          // (129 for an infinity: such a row is NaN)
          const int eq = amax > 0.f ? exp_above(amax) : 0;
          if (c4 == 0) exps[of_block] = eq;
          const float fq = exp2i(kTop - eq);
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[x][e] *= fq;
            if constexpr (RAW) {  // hi, lo = what hi leaves, and (THREE) what both leave
              uint32_t hi[4], lo[4];
              // the codes of f[x], which is left as what they do not hold
              auto term = [&](uint32_t (&code)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  code[e] = f32x2_to_codes2<FP8PA_E4M3>(f[x][2 * e], f[x][2 * e + 1]);
                  const float2 b = __half22float2(h2(codes2_to_f16x2<FP8PA_E4M3>(code[e])));
                  f[x][2 * e] -= b.x;
                  f[x][2 * e + 1] -= b.y;
                }
              };
              term(hi);
              term(lo);
              const int c8 = x * 4 + c4;  // 8 dims: half a 16-byte chunk
              uint8_t* p = dst + swizzled<D>(to_row, c8 >> 1) + (c8 & 1) * 8;
              *reinterpret_cast<uint2*>(p) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
              *reinterpret_cast<uint2*>(p + SM::kCodes) =
                  make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
              if constexpr (THREE) {
                term(lo);
                *reinterpret_cast<uint2*>(p + (SM::kQ3 - SM::kQ)) =
                    make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
              }
            } else {
              *reinterpret_cast<uint4*>(dst + (to_row >> 3) * 128 + r8 * 16 +
                                        (x * 4 + c4) * 2048) =
                  make_uint4(pack_half2(f[x][0], f[x][1]), pack_half2(f[x][2], f[x][3]),
                             pack_half2(f[x][4], f[x][5]), pack_half2(f[x][6], f[x][7]));
            }
          }
        }
      }
      int qi, h;
      query_of(bl, qi, h);
      const int qrow = im.r.qlo + qi;
      const int depth = __ldg(tv.depth + qrow);
      if (wide || t == 0) *row = RowMask{window_first(a.window, im.r.pA + depth), qrow};
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + kTQ);
      const float slope = (VAR > 0 && a.slopes) ? __ldg(a.slopes + h) * kLog2e : 0.f;
      const float cap_log2 = VAR == 2 ? a.cap * kLog2e : 0.f;
      // the bias of a token is slope pos + b0 (and the cap, where its tanh is taken from 1)
      const float b0 = (cap_quick ? cap_log2 : 0.f) - slope * static_cast<float>(depth);
      // the thread's groups of 32 tokens
      const int part = rl / sl;
      const uint32_t groups = sl >= 128 ? 0xFu : (sl == 64 ? 5u << part : 1u << part);
      float ref = kNegBig, l = 0.f, zs = 0.f;
      // makes the row NaN where it saw codes of tile gt that are not finite
      auto late_nan = [&](uint32_t gt) {
        const TileInfo* info = infos + gt % kInfos;
        const uint4 c = *reinterpret_cast<const uint4*>(info->cbad);
        if ((c.x | c.y | c.z | c.w) != 0 && saw_nan(info, groups, row, tv.line))
          l = __int_as_float(0x7FC00000);
      };
      uint32_t ra[32];  // a group's scores
      uint4 sc[8];      // and their scales, loaded beside them
      for (int x = 0; x < 2 * mine; ++x) {  // halves of the stream's tiles
        const int half = x & 1;
        const uint32_t gt = g0 + (x >> 1) * step;
        // (S is issued once the tile's info is complete)
        if (!wait_warp(kTS + t * 2 + half, ns & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (x == 0) {
          // log2-domain factor of a raw score (capped scores: see cap_in)
          const int er = exps[bl];
          zs = fabsf(a.sm_scale) * exp2i(er - kTop) * (VAR == 2 ? a.cap_in : kLog2e);
          if (VAR == 0) zs = max_nan(zs, 1e-37f);  // (it multiplies a masked -inf: not zero)
          if (er > 128) zs = __int_as_float(0x7FC00000);
        } else if (half == 0) {
          late_nan(gt - step);  // (what the tile before brought that is not finite is known by now)
        }
        const TileInfo& info = infos[gt % kInfos];
        auto load = [&](int w, const float* scale) {
          tmem_ld32(ts + w * 32, ra);
          const uint32_t at = smem_u32(scale + w * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i) sc[i] = lds128(at + i * 16);
          tmem_ld_wait();
          tmem_landed(ra);
        };
        // ---- a bound of z + e over the row's tokens; the scores go back to TMEM
        const int w0 = half * 2;
        const float2 ev = *reinterpret_cast<const float2*>(info.ev + w0);
        const uint2 seen = *reinterpret_cast<const uint2*>(info.seen + w0);
        const uint2 bads = *reinterpret_cast<const uint2*>(info.bad + w0);
        float bound = __int_as_float(0xff800000);
        // (both groups laid out: MX, 64 nodes of 8 x 32K 542 us, in a loop 565; FP8 codes, the
        // ragged 64 209 us, in a loop 197)
#pragma unroll (RAW ? 1 : 2)
        for (int y = 0; y < 2; ++y) {
          const int w = w0 + y;
          if (((groups >> w) & 1u) == 0) continue;
          const uint32_t whole = y ? seen.y : seen.x, bad = y ? bads.y : bads.x;
          load(w, info.ks);
          const uint64_t zs2 = f2_pack(zs, zs), sl2 = f2_pack(slope, slope);
          const uint64_t b02 = f2_pack(b0, b0);
#pragma unroll
          for (int i4 = 0; i4 < 8; ++i4) {
            float4 p4;
            if constexpr (VAR > 0) p4 = reinterpret_cast<const float4*>(info.pos + w * 32)[i4];
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2) {
              uint32_t* v = ra + i4 * 4 + i2 * 2;
              uint64_t z = f2_mul(u2_pack(v[0], v[1]),
                                  i2 ? u2_pack(sc[i4].z, sc[i4].w) : u2_pack(sc[i4].x, sc[i4].y));
              float y0, y1;
              if constexpr (VAR > 0) {
                const uint64_t b =
                    f2_fma(sl2, i2 ? f2_pack(p4.z, p4.w) : f2_pack(p4.x, p4.y), b02);
                if constexpr (VAR == 1) {
                  z = f2_fma(z, zs2, b);
                } else if (cap_quick) {  // cap tanh(z / cap) = cap - 2 cap / (2^x + 1)
                  f2_unpack(f2_mul(z, zs2), y0, y1);
                  f2_unpack(f2_add(f2_pack(ex2(y0), ex2(y1)), f2_pack(1.f, 1.f)), y0, y1);
                  z = f2_fma(f2_pack(rcp_fast(y0), rcp_fast(y1)),
                             f2_pack(-2.f * cap_log2, -2.f * cap_log2), b);
                } else {
                  f2_unpack(f2_mul(z, zs2), y0, y1);
                  y0 = a.cap * tanh_f32(y0 * a.tanh_in) * kLog2e;
                  y1 = a.cap * tanh_f32(y1 * a.tanh_in) * kLog2e;
                  z = f2_add(f2_pack(y0, y1), b);
                }
              }
              f2_unpack(z, y0, y1);
              v[0] = __float_as_uint(y0);
              v[1] = __float_as_uint(y1);
            }
          }
          if (!whole || bad) {
            const uint32_t m = seen_bits(&info, w, row, tv.line);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (((m >> i) & 1) == 0) ra[i] = 0xff800000u;
            if (m & bad) l = __int_as_float(0x7FC00000);
          }
          float m4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = __int_as_float(0xff800000);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            m4[i & 3] = max3(m4[i & 3], __uint_as_float(ra[2 * i]), __uint_as_float(ra[2 * i + 1]));
          tmem_st32(ts + w * 32, ra);
          const float mx = max3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
          bound = fmaxf(bound, fmaf(mx, VAR > 0 ? 1.f : zs, y ? ev.y : ev.x));
        }
        tmem_st_wait();
        // ---- the reference: where the bound passed it by 2^kTau it moves, and with it the
        // sums and O
        float al = 1.f;
        if (bound > ref + kTau) {
          al = ex2(ref - bound);
          ref = bound;
        }
        if (__any_sync(0xffffffffu, al != 1.f)) {
          l *= al;
          if (x > 0) {  // behind the product of the half before
            if (!wait_warp(kTO + t * 2 + (half ^ 1), (ns - (half ^ 1)) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              tmem_ld32(to + c * 32, ra);
              tmem_ld_wait();
              tmem_landed(ra);
#pragma unroll
              for (int i = 0; i < 32; ++i) ra[i] = __float_as_uint(__uint_as_float(ra[i]) * al);
              tmem_st32(to + c * 32, ra);
            }
          }
        }
        // ---- P times V's scale, and the sum of P; zeros for the other shares' tokens
#pragma unroll 1
        for (int y = 0; y < 2; ++y) {
          const int w = w0 + y;
          uint32_t pw[16];
          if (((groups >> w) & 1u) == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) pw[i] = 0;
            tmem_st16(ts + w * 32, pw);
            continue;
          }
          const float e = y ? ev.y : ev.x;
          load(w, info.vs);
          const float c0 = kShift - ref + e, f = VAR > 0 ? 1.f : zs;
          const uint64_t f2 = f2_pack(f, f), c02 = f2_pack(c0, c0);
          uint64_t la = 0, lb = 0;  // (0.f, 0.f)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint4 v4 = sc[i >> 1];
            const uint64_t z = u2_pack(ra[2 * i], ra[2 * i + 1]);
            float p, q;
            f2_unpack(VAR > 0 ? f2_add(z, c02) : f2_fma(z, f2, c02), p, q);
            const uint64_t e2 = f2_pack(ex2(p), ex2(q));
            if (i & 1) lb = f2_add(lb, e2);
            else la = f2_add(la, e2);
            f2_unpack(f2_mul(e2, i & 1 ? u2_pack(v4.z, v4.w) : u2_pack(v4.x, v4.y)), p, q);
            pw[i] = pack_half2(p, q);
          }
          tmem_st16(ts + w * 32, pw);
          float sa, sb;
          f2_unpack(f2_add(la, lb), sa, sb);
          l = fmaf(sa + sb, ex2(-e), l);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kTP + t * 2 + half);
        ns += half;
      }
      if (!ok) break;
      if (mine > 0) {  // the last product
        if (!wait_warp(kTO + t * 2 + 1, (ns - 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        late_nan(g0 + step * (mine - 1));
      }
      g += n;

      // ---- the block's result, or this range's piece of it, from the row's partial
      // results: of both streams, and of the shares of the lanes
      const bool piece = im.t0 > 0 || im.t1 < im.r.count;
      const bool stat = a.mode == FP8PA_SCALE_CHANNEL_STATIC;
      const float* vch = a.v_scale + static_cast<long>(im.kvh) * D;
      const long slot = (static_cast<long>(blockIdx.x) * 2 + (im.t0 > 0 ? 0 : 1)) * kRows;
      const int partials = n > 1 || wide ? 256 : 128;  // lanes of the streams that had a tile
      ml[t * 128 + rl] = make_float2(ref, l);
      if (!sync_all()) {
        ok = false;
        break;
      }
      float M = kNegBig, sum = 0.f;
      {
        float2 part[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          part[k] = k * sl < 256 ? ml[(bl & (sl - 1)) + k * sl] : make_float2(kNegBig, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) M = fmaxf(M, part[k].x);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k * sl < 256) sum += part[k].y * ex2(part[k].x - M);
      }
      const float scale = ex2(ref - M) * (piece ? 1.f : (sum == 0.f ? 0.f : 1.f / sum));
      if (piece && (wide || t == 0) && bl < im.r.rows && bl < sl) pv.ml[slot + bl] = make_float2(M, sum);
      // a quarter of the dims at a time: every lane leaves its part, in q's place, then all
      // threads add them up, four dims of a row each.  Chunk c (4 dims) of lane y's part,
      // free of bank conflicts:
      constexpr int kChunks = D / 16;
      auto at = [&](int y, int c) {
        return reinterpret_cast<float4*>(sm + SM::kQ + y * (kChunks * 16) +
                                         ((c ^ y) & (kChunks - 1)) * 16);
      };
#pragma unroll 1
      for (int dq = 0; dq < 4 && ok; ++dq) {
        // a thread adds up chunk c of lanes r, r + 32, ...: all are asked for at once
        const int c = tid % kChunks, r = tid / kChunks, d0 = dq * (D / 4) + c * 4;
        float4 ch = make_float4(1.f, 1.f, 1.f, 1.f);
        if (stat) ch = __ldg(reinterpret_cast<const float4*>(vch + d0));
        if (t * 128 < partials) {
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            uint32_t o[16];
            tmem_ld16(to + dq * (D / 4) + x * 16, o);
            tmem_ld_wait();
            tmem_landed(o);
            float f[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(o[i]) * scale;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *at(t * 128 + rl, x * 4 + i) =
                  make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
          }
        }
        if (!sync_all()) {
          ok = false;
          break;
        }
        if (r < 32 && r < im.r.rows) {
          float4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            v[k] = k * 32 < partials ? *at(r + k * 32, c) : make_float4(0.f, 0.f, 0.f, 0.f);
          auto fold = [&](int k, int from) {
            v[k].x += v[from].x;
            v[k].y += v[from].y;
            v[k].z += v[from].z;
            v[k].w += v[from].w;
          };
          if (sl <= 128) {
#pragma unroll
            for (int k = 0; k < 4; ++k) fold(k, k + 4);
          }
          if (sl <= 64) {
            fold(0, 2);
            fold(1, 3);
          }
          if (sl <= 32) fold(0, 1);
#pragma unroll
          for (int k = 0; k < (RAW ? 4 : 8); ++k) {
            const int row = r + k * 32;
            if (k * 32 >= sl || row >= im.r.rows) continue;
            float4 o = v[k];
            o.x *= ch.x;
            o.y *= ch.y;
            o.z *= ch.z;
            o.w *= ch.w;
            if (piece) {
              *reinterpret_cast<float4*>(pv.o + (slot + row) * D + d0) = o;
              continue;
            }
            int qy, hy;
            query_of(row, qy, hy);
            const long to_row = ((static_cast<long>(im.r.qlo) + qy) * a.hq + hy) * D + d0;
            if (a.out_f32) {
              *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + to_row) = o;
            } else {
              const __nv_bfloat162 b[2] = {__floats2bfloat162_rn(o.x, o.y),
                                           __floats2bfloat162_rn(o.z, o.w)};
              *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + to_row) =
                  *reinterpret_cast<const uint2*>(b);
            }
          }
        }
        if (!sync_all()) ok = false;  // (also: the next item's q goes there)
      }
      tc_fence_before();
    }
  }

  // ---- drain and free: no MMA may still be in flight
  __syncwarp();
  if (warp >= kIssue && warp < kIssue + 2) {
    if (elect_one()) tc_commit(bars + kTDrain + warp - kIssue);
    __syncwarp();
    (void)mbar_wait_bounded(bars + kTDrain + warp - kIssue, 0, kWaitLimitCycles);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssue) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- instances
template <int D, bool RAW, bool THREE>
TreeKernel pick_tree(int var) {
  return {var == 0 ? tree_kernel<D, RAW, 0, THREE>
                   : (var == 1 ? tree_kernel<D, RAW, 1, THREE> : tree_kernel<D, RAW, 2, THREE>),
          THREE ? TreeSmem<D, RAW>::kBytesThree : TreeSmem<D, RAW>::kBytes, kTreeThreads<RAW>};
}
template <int D>
TreeKernel pick_tree(bool raw, bool st, int var) {
  return !raw ? pick_tree<D, false, false>(var)
              : (st ? pick_tree<D, true, true>(var) : pick_tree<D, true, false>(var));
}

}  // namespace

}  // namespace fp8pa
