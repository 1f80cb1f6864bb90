// prefill.cu -- attention of ragged query chunks over the paged cache, causal
// with score modifiers.
//
//   z_j = sm_scale q_i . k^_j;  z_j = cap tanh(z_j / cap);  z_j -= slope |i - j|
//   out_i = sum_j softmax(z)_j v^_j over j < prefix or i - window < j <= i
//
// One warp per (query, head) walks its visible tokens 32 at a time: a lane
// scores one token, then the lanes share the dims of the weighted sum.  FP32
// throughout, online softmax in the log2 domain.
#include <float.h>

#include "common.cuh"
#include "internal.h"
#include "score_mods.cuh"

namespace fp8pa {

namespace {

constexpr int kWarps = 4;

template <int FMT>
__device__ __forceinline__ void codes4_to_f32(uint32_t w, float (&f)[4]) {
  uint32_t lo, hi;
  codes4_to_f16x2x2<FMT>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

// Scale of dim d of cached row `row` = (block * hkv + kvh) * bs + offset.
__device__ __forceinline__ float row_scale(const PrefillArgs& a, const float* sc, long row,
                                           long blk, int kvh, int d) {
  switch (a.mode) {
    case FP8PA_SCALE_TOKEN_HEAD: return __ldg(sc + row);
    case FP8PA_SCALE_CHANNEL_STATIC: return __ldg(sc + kvh * a.d + d);
    case FP8PA_SCALE_SEGMENT: return __ldg(sc + blk * a.hp + kvh);
    default: {
      const int e = __ldg(reinterpret_cast<const uint8_t*>(sc) + row * (a.d / a.gs) + d / a.gs);
      return e == 0 ? __int_as_float(1 << 22) : __int_as_float(e << 23);
    }
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) prefill_kernel(const PrefillArgs a) {
  __shared__ float s_q[kWarps][D];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long row = static_cast<long>(blockIdx.x) * kWarps + warp;
  if (row >= static_cast<long>(a.total_q) * a.hq) return;
  const int t = static_cast<int>(row / a.hq), h = static_cast<int>(row % a.hq);
  const int kvh = h / a.G;
  // the request whose chunk holds row t
  int b = -1, qlo = 0, qn = 0;
  for (int base = 0; base < a.batch && b < 0; base += 32) {
    const int k = base + lane;
    bool in = false;
    if (k < a.batch) {
      const int lo = __ldg(a.q_offsets + k), hi = __ldg(a.q_offsets + k + 1);
      if (lo < 0 || hi < lo || hi > a.total_q) {
        if (row == 0) raise_error(a.err, FP8PA_DEVERR_Q_OFFSETS);
      } else {
        in = lo <= t && t < hi;
      }
    }
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (m) {
      b = base + __ffs(m) - 1;
      qlo = __ldg(a.q_offsets + b);
      qn = __ldg(a.q_offsets + b + 1) - qlo;
    }
  }
  if (b < 0) return;
  const int cap = a.max_blocks * a.bs;
  int L = __ldg(a.seq_lens + b);
  if ((L < 0 || L > cap || L < qn) && lane == 0) raise_error(a.err, FP8PA_DEVERR_SEQ_LEN);
  L = min(max(L, 0), cap);
  const ScoreMods mods{a.prefix_lens, a.slopes, a.cap, a.window};
  const int pos = L - qn + (t - qlo);
  const int wf = window_first(mods, pos), pre = prefix_len(mods, b, L);
  const int last = max(pos + 1, pre);  // keys [0, last) hold every visible one
  const float slope = a.slopes ? __ldg(a.slopes + h) * kLog2e : 0.f;

  for (int d = lane; d < D; d += 32) {
    float x = __uint_as_float(static_cast<uint32_t>(a.q[row * D + d]) << 16);
    if (a.mode == FP8PA_SCALE_CHANNEL_STATIC) x *= __ldg(a.k_scale + kvh * D + d);
    s_q[warp][d] = x;
  }
  __syncwarp();
  constexpr int PER = D / 32;
  float m = -FLT_MAX, l = 0.f, o[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.f;

  for (int j0 = 0; j0 < last; j0 += 32) {
    const int j = j0 + lane;
    bool vis = (j <= pos && j >= wf) || j < pre;
    if (!__any_sync(0xffffffffu, vis)) continue;
    long krow = 0, blk = 0;
    if (vis) {
      blk = __ldg(a.block_tables + static_cast<long>(b) * a.max_blocks + j / a.bs);
      if (blk < 0 || blk >= a.num_blocks) {
        raise_error(a.err, FP8PA_DEVERR_BLOCK_RANGE);
        vis = false;
      } else {
        krow = (blk * a.hkv + kvh) * a.bs + j % a.bs;
      }
    }
    float z = __int_as_float(0xff800000);
    if (vis) {
      float acc = 0.f;
      const uint4* src = reinterpret_cast<const uint4*>(a.k_cache + krow * D);
      for (int c = 0; c < D / 16; ++c) {
        const uint4 u = __ldg(src + c);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[4];
          codes4_to_f32<FMT>(w[i], f);
#pragma unroll
          for (int e = 0; e < 4; ++e) part = fmaf(f[e], s_q[warp][c * 16 + 4 * i + e], part);
        }
        if (a.mode == FP8PA_SCALE_MX_BLOCK) part *= row_scale(a, a.k_scale, krow, blk, kvh, c * 16);
        acc += part;
      }
      if (a.mode == FP8PA_SCALE_TOKEN_HEAD || a.mode == FP8PA_SCALE_SEGMENT)
        acc *= row_scale(a, a.k_scale, krow, blk, kvh, 0);
      z = acc * a.sm_scale;
      if (a.cap > 0.f) z = a.cap * tanh_f32(z / a.cap);
      z = fmaf(-slope, fabsf(static_cast<float>(pos - j)), z * kLog2e);
    }
    float mx = z;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    const float mn = fmaxf(m, mx);
    const float al = ex2(m - mn);
    const float p = vis ? ex2(z - mn) : 0.f;
    float sum = p;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    l = l * al + sum;
    m = mn;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] *= al;
    const unsigned seen = __ballot_sync(0xffffffffu, vis);
    for (unsigned rest = seen; rest; rest &= rest - 1) {
      const int k = __ffs(rest) - 1;
      const float pk = __shfl_sync(0xffffffffu, p, k);
      const long r = __shfl_sync(0xffffffffu, krow, k), bk = __shfl_sync(0xffffffffu, blk, k);
      float f[4];
      const uint8_t* src = a.v_cache + r * D + lane * PER;
      const uint32_t w = PER == 4 ? __ldg(reinterpret_cast<const uint32_t*>(src))
                                  : __ldg(reinterpret_cast<const uint16_t*>(src));
      codes4_to_f32<FMT>(w, f);
#pragma unroll
      for (int e = 0; e < PER; ++e)
        o[e] = fmaf(pk * row_scale(a, a.v_scale, r, bk, kvh, lane * PER + e), f[e], o[e]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const float v = o[e] * inv;
    const long at = row * D + lane * PER + e;
    if (a.out_f32)
      reinterpret_cast<float*>(a.out)[at] = v;
    else
      reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
  }
}

template <int D>
auto pick_prefill(int fmt) {
  return fmt == FP8PA_E4M3   ? prefill_kernel<D, FP8PA_E4M3>
         : fmt == FP8PA_E5M2 ? prefill_kernel<D, FP8PA_E5M2>
                             : prefill_kernel<D, FP8PA_INT8>;
}

}  // namespace

size_t prefill_workspace_bytes(int, int, int, int, int, int) { return 256; }

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const long rows = static_cast<long>(a.total_q) * a.hq;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, a.d == 128 ? pick_prefill<128>(a.fmt) : pick_prefill<64>(a.fmt),
                            a);
}

}  // namespace fp8pa
