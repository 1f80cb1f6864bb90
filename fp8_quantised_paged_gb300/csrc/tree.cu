// tree.cu -- attention for trees of drafted tokens over the paged cache.
//
//   z_j = sm_scale q_i . k^_j;  z_j = cap tanh(z_j / cap);  z_j -= slope (pos_i - pos_j)
//   out_i = sum_j softmax(z)_j v^_j  over the tokens ahead of the tree (as the window and
//   the prefix leave them) and the nodes on i's line, itself among them
//
// The plain kernel: a warp per (node, query head) walks its visible tokens one at a time,
// a lane holding head_dim / 32 dims, with the running maximum and sum of the softmax.
#include "common.cuh"
#include "internal.h"
#include "score_mods.cuh"

namespace fp8pa {

namespace {

constexpr int kMaxTree = FP8PA_MAX_TREE;

__device__ __forceinline__ float code_value(int fmt, uint8_t c) {
  uint32_t r;
  if (fmt == FP8PA_INT8) return static_cast<float>(c) - 128.f;
  if (fmt == FP8PA_E4M3) r = codes2_to_f16x2<FP8PA_E4M3>(c);
  else r = codes2_to_f16x2<FP8PA_E5M2>(c);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(r & 0xFFFFu)));
}

template <int D>
__global__ void __launch_bounds__(128) tree_plain_kernel(const PrefillArgs a,
                                                         const int32_t* parents) {
  constexpr int N = D / 32;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long wid = static_cast<long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int row = static_cast<int>(wid / a.hq), h = static_cast<int>(wid % a.hq);
  if (row >= a.total_q) return;
  // the request: the last one whose rows hold this one
  int b = -1, lo = 0, hi = 0;
  for (int i = 0; i < a.batch; ++i) {
    lo = __ldg(a.q_offsets + i);
    hi = __ldg(a.q_offsets + i + 1);
    if (lo < 0 || hi < lo || hi > a.total_q) {
      if (wid == 0 && lane == 0) raise_error(a.err, FP8PA_DEVERR_Q_OFFSETS);
      continue;
    }
    if (row >= lo && row < hi) {
      b = i;
      if (wid != 0) break;
    }
  }
  if (b < 0) return;
  lo = __ldg(a.q_offsets + b);
  hi = __ldg(a.q_offsets + b + 1);
  const int n = hi - lo, L = __ldg(a.seq_lens + b);
  if (n > kMaxTree) {
    if (lane == 0) raise_error(a.err, FP8PA_DEVERR_TREE);
    return;
  }
  if (L < n || L > a.max_blocks * a.bs) {
    if (lane == 0) raise_error(a.err, FP8PA_DEVERR_SEQ_LEN);
    return;
  }
  const int ctx = L - n, kvh = h / a.G;
  const int32_t* par = parents + lo;
  auto parent = [&](int i) {
    const int p = __ldg(par + i);
    if (p >= -1 && p < i) return p;
    if (lane == 0) raise_error(a.err, FP8PA_DEVERR_TREE);
    return -1;
  };
  int depth = 0;
  for (int i = parent(row - lo); i >= 0; i = parent(i)) ++depth;
  const int pos = ctx + depth;
  const ScoreMods mods{a.prefix_lens, a.slopes, a.cap, a.window};
  const int pre = prefix_len(mods, b, ctx), wf = window_first(a.window, pos);
  const float slope = a.slopes ? __ldg(a.slopes + h) * kLog2e : 0.f;
  float q[N], kcs[N], vcs[N], o[N], m = -1e30f, l = 0.f;
#pragma unroll
  for (int x = 0; x < N; ++x) {
    const int d = lane * N + x;
    q[x] = __uint_as_float(static_cast<uint32_t>(
               __ldg(a.q + (static_cast<long>(row) * a.hq + h) * D + d)) << 16);
    const bool st = a.mode == FP8PA_SCALE_CHANNEL_STATIC;
    kcs[x] = st ? __ldg(a.k_scale + static_cast<long>(kvh) * D + d) : 1.f;
    vcs[x] = st ? __ldg(a.v_scale + static_cast<long>(kvh) * D + d) : 1.f;
    o[x] = 0.f;
  }
  const int32_t* table = a.block_tables + static_cast<long>(b) * a.max_blocks;
  auto see = [&](int j, int pj) {  // cached token j, at position pj
    const int page = __ldg(table + j / a.bs);
    if (page < 0 || page >= a.num_blocks) {
      if (lane == 0) raise_error(a.err, FP8PA_DEVERR_BLOCK_RANGE);
      return;
    }
    const size_t r = (static_cast<size_t>(page) * a.hkv + kvh) * a.bs + j % a.bs;
    auto scale = [&](const float* s, int d) {
      if (a.mode == FP8PA_SCALE_TOKEN_HEAD) return __ldg(s + r);
      if (a.mode == FP8PA_SCALE_SEGMENT) return __ldg(s + static_cast<size_t>(page) * a.hp + kvh);
      if (a.mode == FP8PA_SCALE_CHANNEL_STATIC) return 1.f;
      const int e = __ldg(reinterpret_cast<const uint8_t*>(s) + r * (D / a.gs) + d / a.gs);
      return e == 255 ? __int_as_float(0x7FC00000)
                      : (e == 0 ? __int_as_float(0x00400000) : __int_as_float(e << 23));
    };
    float z = 0.f;
#pragma unroll
    for (int x = 0; x < N; ++x) {
      const int d = lane * N + x;
      z += q[x] * kcs[x] * code_value(a.fmt, __ldg(a.k_cache + r * D + d)) * scale(a.k_scale, d);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    z *= a.sm_scale;
    z = a.cap > 0.f ? a.cap * tanh_f32(z * (1.f / a.cap)) * kLog2e : z * kLog2e;
    z -= slope * static_cast<float>(pos - pj);
    const float mn = fmaxf(m, z), f = ex2(m - mn), p = ex2(z - mn);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int x = 0; x < N; ++x) {
      const int d = lane * N + x;
      o[x] = o[x] * f + p * (code_value(a.fmt, __ldg(a.v_cache + r * D + d)) * scale(a.v_scale, d));
    }
  };
  for (int j = 0; j < min(pre, wf); ++j) see(j, j);
  for (int j = wf; j < ctx; ++j) see(j, j);
  for (int i = row - lo, d = depth; i >= 0; i = parent(i), --d)
    if (a.window == 0 || depth - d < a.window) see(ctx + i, ctx + d);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const long at = (static_cast<long>(row) * a.hq + h) * D + lane * N;
#pragma unroll
  for (int x = 0; x < N; ++x) {
    const float v = o[x] * inv * vcs[x];
    if (a.out_f32) reinterpret_cast<float*>(a.out)[at + x] = v;
    else reinterpret_cast<__nv_bfloat16*>(a.out)[at + x] = __float2bfloat16_rn(v);
  }
}

}  // namespace

size_t tree_workspace_bytes(int total_q, int batch, int hq, int hkv, int d, int device) {
  return 256;
}

cudaError_t launch_tree(const PrefillArgs& a, const int32_t* parents, cudaStream_t stream) {
  const long warps = static_cast<long>(a.total_q) * a.hq;
  const unsigned grid = static_cast<unsigned>((warps + 3) / 4);
  if (a.d == 128) tree_plain_kernel<128><<<grid, 128, 0, stream>>>(a, parents);
  else tree_plain_kernel<64><<<grid, 128, 0, stream>>>(a, parents);
  return cudaGetLastError();
}

}  // namespace fp8pa
