// append_rope.cu -- the append with rotary positions: q and k rows are turned
// by their token's angles; K and V are scaled, rounded and scattered into the
// paged cache as by append.cu; q goes out as bf16.
//
// Mathematics: a pair (a, b) of dims at angle (c, s) becomes
// (a c - b s, b c + a s), each fp32 product and sum rounded on its own
// (__fmul_rn and so on: no contraction), so the scales and codes are those of
// the written formula bit for bit.  The turned K is quantised straight from
// fp32: rounding it to bf16 first would add an error of 2^-9 to the code's
// 2^-4 for nothing.  Unlike the bf16 rows of append.cu, whose finite set of
// quotients was checked against a corrected product, these take the IEEE
// division.
//
// GB300 design.  A sub-group of LPR lanes holds one row, each lane one
// 16-byte chunk of 8 dims (three at head_dim 576).  Neighbouring pairs lie in
// one lane; paired halves swap their packed words by a shuffle.  Where whole
// rows of paired halves turn (the usual case), a lane takes chunk i of both
// halves instead and no word moves.  A warp works on rows of ONE token, so its
// lanes load their angles once and keep them in registers for all of the warp's
// rows.
//
// Bound by HBM where there are many tokens: 16384 tokens of 64 + 8 + 8 rows of 128
// dims move 647 MB in 127 us, 5.1 TB/s (76% of a plain copy's rate; 218 us with
// neighbours in one lane and the words swapped by shuffles).  A decode step's 12
// tokens take 2.2 us on the GPU, a launch's own time.
#include <float.h>

#include "common.cuh"
#include "internal.h"

namespace fp8pa {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Sums of two packed products, the second taken times sign (1 or -1).  The sums
// are scalar on purpose: a packed sum was contracted with its products.
__device__ __forceinline__ void turn2(uint64_t x, uint64_t y, float sign, float& lo, float& hi) {
  float x0, x1, y0, y1;
  f2_unpack(x, x0, x1);
  f2_unpack(y, y0, y1);
  lo = sign > 0.f ? __fadd_rn(x0, y0) : __fsub_rn(x0, y0);
  hi = sign > 0.f ? __fadd_rn(x1, y1) : __fsub_rn(x1, y1);
}

// Where a row of the call lives: `row` counts a token's q rows, then its K
// rows, then its V rows.
struct RowRef {
  const uint16_t* src;
  int kind;  // 0 q, 1 k, 2 v, -1 none
  int head;
};

__device__ __forceinline__ RowRef row_ref(const RopeArgs& a, long t, int row) {
  RowRef r;
  if (row < a.hq) {
    r.kind = 0;
    r.head = row;
    r.src = a.q + t * a.q_stride + static_cast<long>(row) * a.d;
  } else if (row < a.hq + a.hkv) {
    r.kind = 1;
    r.head = row - a.hq;
    r.src = a.k + t * a.k_stride + static_cast<long>(r.head) * a.d;
  } else if (row < a.rows) {
    r.kind = 2;
    r.head = row - a.hq - a.hkv;
    r.src = a.v + t * a.v_stride + static_cast<long>(r.head) * a.d;
  } else {
    r.kind = -1;
    r.head = 0;
    r.src = nullptr;
  }
  return r;
}

// One K or V row: scale, codes, scatter.  The whole warp calls it (the absmax
// shuffles), `live` lanes store.
template <int FMT, int MODE, int LPR, int R>
__device__ __forceinline__ void store_codes(const RopeArgs& a, const float (&v)[R][8], bool second,
                                            int head, long blk, int off, bool live, int sl) {
  constexpr float kFmax = code_max<FMT>();
  constexpr int kEmax = FMT == FP8PA_E4M3 ? 8 : 15;  // exponent of the largest normal
  const int nch = a.d / 8;
  const long crow = live ? (blk * a.hkv + head) * a.bs + off : 0;
  float* scl = second ? a.scale[1] : a.scale[0];
  float cmax[R], s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    cmax[r] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) cmax[r] = fmaxf(cmax[r], fabsf(v[r][e]));
  }
  if constexpr (MODE == FP8PA_SCALE_TOKEN_HEAD) {
    float m = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) m = fmaxf(m, cmax[r]);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float sc = fmaxf(__fdiv_rn(m, kFmax), 1e-12f);
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = sc;
    if (live && sl == 0) scl[crow] = sc;
  } else if constexpr (MODE == FP8PA_SCALE_TOKEN_GROUP || MODE == FP8PA_SCALE_MX_BLOCK) {
    const int lpg = a.gs / 8;  // lanes per group: a power of two <= LPR
    const int ngroups = a.d / a.gs;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float m = cmax[r];
      for (int o = 1; o < lpg; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const int ci = sl + LPR * r;
      const bool writes = live && ci < nch && (sl & (lpg - 1)) == 0;
      const long at = crow * ngroups + (ci * 8) / a.gs;
      if constexpr (MODE == FP8PA_SCALE_TOKEN_GROUP) {
        s[r] = fmaxf(__fdiv_rn(m, kFmax), 1e-12f);
        if (writes) scl[at] = s[r];
      } else {
        // the block's power of two 2^e, read off the exponent field (a zero or
        // subnormal absmax gives the floor); s is the exact multiplier 2^-e
        const int ef = (__float_as_int(m) >> 23) & 0xFF;
        const int e = ef == 0 ? -127 : min(127, max(-127, ef - 127 - kEmax));
        s[r] = exp2i(-e);
        if (writes) reinterpret_cast<uint8_t*>(scl)[at] = static_cast<uint8_t>(e + 127);
      }
    }
  }
  if (!live) return;
  uint8_t* dst = (second ? a.cache[1] : a.cache[0]) + crow * a.d;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int ci = sl + LPR * r;
    if (ci >= nch) continue;
    float q[8];
    if constexpr (MODE == FP8PA_SCALE_CHANNEL_STATIC) {
      const float4* sp =
          reinterpret_cast<const float4*>(scl + static_cast<long>(head) * a.d + ci * 8);
      const float4 s0 = __ldg(sp), s1 = __ldg(sp + 1);
      const float sc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = __fdiv_rn(v[r][e], sc[e]);
    } else if constexpr (MODE == FP8PA_SCALE_MX_BLOCK) {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = v[r][e] * s[r];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = __fdiv_rn(v[r][e], s[r]);
    }
    uint2 pk;
    pk.x = f32x2_to_codes2<FMT>(q[0], q[1]) | (f32x2_to_codes2<FMT>(q[2], q[3]) << 16);
    pk.y = f32x2_to_codes2<FMT>(q[4], q[5]) | (f32x2_to_codes2<FMT>(q[6], q[7]) << 16);
    *reinterpret_cast<uint2*>(dst + ci * 8) = pk;
  }
}

// STEPS steps of 32 / LPR rows per warp, their loads issued together.  PAIR: a
// lane's two chunks are the halves of its pairs (rot_dim = head_dim = 16 LPR).
template <int FMT, int MODE, int LPR, int R, int STEPS, bool PAIR>
__global__ void __launch_bounds__(kWarps * 32, STEPS > 1 && R < 3 ? 4 : 1)
    append_rope_kernel(const RopeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int SG = 32 / LPR;
  const int lane = threadIdx.x & 31, sg = lane / LPR, sl = lane % LPR;
  const uint32_t wid = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const uint32_t t32 = fast_div(wid, a.div_warps);
  if (t32 >= static_cast<uint32_t>(a.num_tokens)) return;  // warp-uniform
  const long t = t32;
  const int row0 = static_cast<int>(wid - t32 * a.warps_per_token) * (STEPS * SG) + sg;
  const int nch = a.d / 8;

  const int pos = __ldg(a.positions + t), slot = __ldg(a.slot_mapping + t);
  RowRef ref[STEPS];
  uint4 w[STEPS][R];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    ref[i] = row_ref(a, t, row0 + i * SG);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int ci = sl + LPR * r;
      w[i][r] = (ref[i].kind >= 0 && ci < nch)
                    ? __ldcs(reinterpret_cast<const uint4*>(ref[i].src + ci * 8))
                    : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (pos < 0 || pos >= a.max_position) {
    if (slot >= 0 && lane == 0) raise_error(a.err, FP8PA_DEVERR_POSITION);
    return;
  }
  const uint32_t bq = slot < 0 ? 0u : fast_div(static_cast<uint32_t>(slot), a.div_bs);
  const long blk = static_cast<long>(bq);
  const int off = slot < 0 ? 0 : slot - static_cast<int>(bq) * a.bs;
  const bool in_pool = slot >= 0 && blk < a.num_blocks;
  if (slot >= 0 && !in_pool && lane == 0) raise_error(a.err, FP8PA_DEVERR_SLOT_RANGE);

  // This lane's angles: chunk r_rot of the lane is the one that may turn (the
  // range lies in one 256-dim span where rows have more than one chunk a lane;
  // PAIR: both turn, by the same angles).
  const int half = a.rot_dim / 2, hch = half / 8;
  const int r_rot = PAIR ? 0 : a.rot_offset / (8 * LPR);
  const int rc = PAIR ? sl : sl + LPR * r_rot - a.rot_offset / 8;  // chunk within the range
  const bool turns = PAIR || (rc >= 0 && rc < a.rot_dim / 8);
  const bool hi = !PAIR && rc >= hch;  // second half of the range (paired halves)
  // cosines, and the sines with the sign that they enter with: the pair's first
  // dim becomes a c + b (-s), its second b c + a s
  uint64_t cs[4], sn[4];
  if (turns) {
    const float* row = a.cos_sin + static_cast<long>(pos) * a.rot_dim;
    if (!PAIR && a.interleaved) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + rc * 4));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + rc * 4));
      cs[0] = f2_pack(c.x, c.x);
      cs[1] = f2_pack(c.y, c.y);
      cs[2] = f2_pack(c.z, c.z);
      cs[3] = f2_pack(c.w, c.w);
      sn[0] = f2_pack(-s.x, s.x);
      sn[1] = f2_pack(-s.y, s.y);
      sn[2] = f2_pack(-s.z, s.z);
      sn[3] = f2_pack(-s.w, s.w);
    } else {
      const int at = (hi ? rc - hch : rc) * 8;
      const float4* cp = reinterpret_cast<const float4*>(row + at);
      const float4* sp = reinterpret_cast<const float4*>(row + half + at);
      const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
      const float m = hi ? 1.f : -1.f;
      cs[0] = f2_pack(c0.x, c0.y);
      cs[1] = f2_pack(c0.z, c0.w);
      cs[2] = f2_pack(c1.x, c1.y);
      cs[3] = f2_pack(c1.z, c1.w);
      sn[0] = f2_pack(m * s0.x, m * s0.y);
      sn[1] = f2_pack(m * s0.z, m * s0.w);
      sn[2] = f2_pack(m * s1.x, m * s1.y);
      sn[3] = f2_pack(m * s1.z, m * s1.w);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = sn[e] = 0;
  }
  // lane holding the other half's chunk
  const int psl = turns ? (hi ? sl - hch : sl + hch) : sl;
  const int plane = sg * LPR + psl;

#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int kind = ref[i].kind;
    float v[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r) unpack8(w[i][r], v[r]);
    if constexpr (PAIR) {
      if (kind < 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t x = f2_pack(v[0][2 * e], v[0][2 * e + 1]);
          const uint64_t y = f2_pack(v[1][2 * e], v[1][2 * e + 1]);
          // (sn: - s)
          turn2(f2_mul(x, cs[e]), f2_mul(y, sn[e]), 1.f, v[0][2 * e], v[0][2 * e + 1]);
          turn2(f2_mul(y, cs[e]), f2_mul(x, sn[e]), -1.f, v[1][2 * e], v[1][2 * e + 1]);
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (R > 1 && r != r_rot) continue;  // warp-uniform
        float p[8];
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = v[r][e ^ 1];
        } else {
          uint4 o;
          o.x = __shfl_sync(0xffffffffu, w[i][r].x, plane);
          o.y = __shfl_sync(0xffffffffu, w[i][r].y, plane);
          o.z = __shfl_sync(0xffffffffu, w[i][r].z, plane);
          o.w = __shfl_sync(0xffffffffu, w[i][r].w, plane);
          unpack8(o, p);
        }
        if (turns && kind < 2) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            turn2(f2_mul(f2_pack(v[r][2 * e], v[r][2 * e + 1]), cs[e]),
                  f2_mul(f2_pack(p[2 * e], p[2 * e + 1]), sn[e]), 1.f, v[r][2 * e],
                  v[r][2 * e + 1]);
        }
      }
    }
    if (kind == 0) {
      uint16_t* dst = a.q_out + t * a.q_out_stride + static_cast<long>(ref[i].head) * a.d;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int ci = sl + LPR * r;
        if (ci < nch) {
          const uint4 o = make_uint4(pack_bf16(v[r][0], v[r][1]), pack_bf16(v[r][2], v[r][3]),
                                     pack_bf16(v[r][4], v[r][5]), pack_bf16(v[r][6], v[r][7]));
          *reinterpret_cast<uint4*>(dst + ci * 8) = o;
        }
      }
    }
    // a warp whose rows are all queries has no scale to find
    if (__any_sync(0xffffffffu, kind > 0))
      store_codes<FMT, MODE, LPR, R>(a, v, kind == 2, ref[i].head, blk, off, kind > 0 && in_pool,
                                     sl);
  }
}

// Rows per call from which a warp takes several steps of rows (the angles loaded
// once for all of them) instead of one.  Tokens of 80 rows of 128 dims, one step
// against several: 2.2 and 3.1 us for 960 rows, 3.4 and 4.2 for 20480, 4.9 and 5.1
// for 40960, 7.7 and 7.6 for 81920, 39 and 31 for 327680.
constexpr long kBulkRows = 65536;

template <int FMT, int MODE, int LPR, int R, bool PAIR>
cudaError_t launch_shape(RopeArgs a, cudaStream_t stream) {
  constexpr int SG = 32 / LPR, BULK = PAIR ? 2 : 3;
  const bool bulk = static_cast<long>(a.num_tokens) * a.rows >= kBulkRows;
  const int per_warp = (bulk ? BULK : 1) * SG;
  a.warps_per_token = static_cast<uint32_t>((a.rows + per_warp - 1) / per_warp);
  a.div_warps = make_fast_div(a.warps_per_token);
  const long warps = static_cast<long>(a.num_tokens) * a.warps_per_token;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  if (bulk) return cudaLaunchKernelEx(&cfg, append_rope_kernel<FMT, MODE, LPR, R, BULK, PAIR>, a);
  return cudaLaunchKernelEx(&cfg, append_rope_kernel<FMT, MODE, LPR, R, 1, PAIR>, a);
}

template <int FMT, int MODE>
cudaError_t launch_lanes(const RopeArgs& a, cudaStream_t stream) {
  // whole rows of paired halves; a scale group lies within a half
  const bool grouped = MODE == FP8PA_SCALE_TOKEN_GROUP || MODE == FP8PA_SCALE_MX_BLOCK;
  if (!a.interleaved && a.rot_dim == a.d && !(grouped && a.gs > a.d / 2)) {
    if (a.d == 64) return launch_shape<FMT, MODE, 4, 2, true>(a, stream);
    if (a.d == 128) return launch_shape<FMT, MODE, 8, 2, true>(a, stream);
  }
  const int nch = a.d / 8;
  if (nch <= 8) return launch_shape<FMT, MODE, 8, 1, false>(a, stream);
  if (nch <= 16) return launch_shape<FMT, MODE, 16, 1, false>(a, stream);
  if (nch <= 32) return launch_shape<FMT, MODE, 32, 1, false>(a, stream);
  return launch_shape<FMT, MODE, 32, 3, false>(a, stream);
}

template <int FMT>
cudaError_t launch_mode(const RopeArgs& a, int mode, cudaStream_t stream) {
  switch (mode) {
    case FP8PA_SCALE_TOKEN_HEAD: return launch_lanes<FMT, FP8PA_SCALE_TOKEN_HEAD>(a, stream);
    case FP8PA_SCALE_CHANNEL_STATIC:
      return launch_lanes<FMT, FP8PA_SCALE_CHANNEL_STATIC>(a, stream);
    case FP8PA_SCALE_TOKEN_GROUP: return launch_lanes<FMT, FP8PA_SCALE_TOKEN_GROUP>(a, stream);
    default:  // MX blocks: FP8 only (rejected for INT8 by the caller)
      if constexpr (FMT != FP8PA_INT8) return launch_lanes<FMT, FP8PA_SCALE_MX_BLOCK>(a, stream);
      return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_append_rope(const RopeArgs& a, int fmt, int mode, cudaStream_t stream) {
  switch (fmt) {
    case FP8PA_E4M3: return launch_mode<FP8PA_E4M3>(a, mode, stream);
    case FP8PA_E5M2: return launch_mode<FP8PA_E5M2>(a, mode, stream);
    default: return launch_mode<FP8PA_INT8>(a, mode, stream);
  }
}

}  // namespace fp8pa
