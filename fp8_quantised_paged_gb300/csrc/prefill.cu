// prefill.cu -- the planner, the merge and the launch of the prefill attention,
// whose method prefill.cuh states.
#include "prefill.cuh"

namespace fp8pa {

namespace {

__host__ __device__ inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline int block_bound(int total_q, int batch, int G) {
  return static_cast<int>((static_cast<long long>(total_q) * G + kRows - 1) / kRows) + batch;
}

// Whether tiles are converted once for all row blocks (ready_kernel) instead of by
// each: where a request has kReadyBlocks of them or more on average, and the tiles
// of the block tables' reach fit kReadyBytes and the workspace.  One request over 16384
// tokens, once against by each: 107 and 113 us at 2 row blocks, 116 and 133 at 3, 125
// and 151 at 4, 151 and 198 at 6; eight over 4096 tokens: 135 and 146 at 2, 172 and 205
// at 3, 262 and 359 at 6 (at 2, where once is ahead by 6%, it also takes the bytes).
// The mean and the reach stand in for the lengths, which the host does not know: a long
// chunk among many single tokens, or in tables far wider than its request, is converted
// by each.  Not where the tables reach fewer than kReadyTiles tiles: a prompt of 200
// tokens takes 26.8 us both ways, and a launch more; one of 300, 28.7 and 30.9.
constexpr int kReadyBlocks = 3;
constexpr int kReadyTiles = 3;
constexpr long long kReadyBytes = 1ll << 30;
inline int tiles_per_request(int bs, int max_blocks) {
  return static_cast<int>((static_cast<long long>(bs) * max_blocks + kT - 1) / kT);
}
inline bool use_ready(int total_q, int batch, int G, int hkv, int d, int bs, int max_blocks) {
  const int tpr = tiles_per_request(bs, max_blocks);
  const double tiles = static_cast<double>(tpr) * batch * hkv;
  return tpr >= kReadyTiles &&
         static_cast<long long>(total_q) * G >=
             static_cast<long long>(kReadyBlocks) * kRows * batch &&
         tiles * (4.0 * kT * d) <= static_cast<double>(kReadyBytes);
}

inline size_t plan_layout(char* ws, int total_q, int batch, int G, int hkv, int d, int bs,
                          int max_blocks, int ranges, bool ready, PlanView* v) {
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
  t.rb = reinterpret_cast<int4*>(take(sizeof(int4) * 3 * nb));
  t.rb_pre = reinterpret_cast<int*>(take(sizeof(int) * (nb + 1)));
  t.start = reinterpret_cast<int*>(take(sizeof(int) * (ranges + 1)));
  t.item = reinterpret_cast<int*>(take(sizeof(int) * (ranges + 1)));
  t.ml = reinterpret_cast<float2*>(take(sizeof(float2) * 2 * ranges * kRows));
  t.o = reinterpret_cast<float*>(take(sizeof(float) * 2 * ranges * kRows * d));
  t.blocks = nb;
  t.tpr = tiles_per_request(bs, max_blocks);
  t.tiles = t.info = nullptr;
  if (ready) {
    const size_t tiles = static_cast<size_t>(t.tpr) * batch * hkv;
    t.tiles = reinterpret_cast<uint8_t*>(take(tiles * 4 * kT * d));
    t.info = reinterpret_cast<uint8_t*>(take(tiles * sizeof(StageInfo)));
  }
  if (v) *v = t;
  return at;
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
      const RowBlock r = make_row_block(c, b, a.window, a.G, i - v.rbase[b]);
      n = r.count;
      v.rb[3 * i] = make_int4(r.b, r.qlo, r.n, r.L);
      v.rb[3 * i + 1] = make_int4(r.pre, r.row0, r.rows, r.np);
      v.rb[3 * i + 2] = make_int4(r.skip, r.count, r.pA, r.pB);
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
  const RowBlock blk = load_row_block(pv.rb + 3 * rb);
  constexpr int TPR = D / 4;        // threads per row
  constexpr int RPC = 256 / TPR;    // rows at a time
  const int sub = threadIdx.x / TPR, d0 = (threadIdx.x % TPR) * 4;
  for (int r = blockIdx.y * kMergeRows + sub; r < min(blk.rows, (static_cast<int>(blockIdx.y) + 1) * kMergeRows);
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
    const int rr = blk.row0 + r;
    const long grow = (static_cast<long>(blk.qlo) + rr / a.G) * a.hq + kvh * a.G + rr % a.G;
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

}  // namespace

size_t prefill_workspace_bytes(int total_q, int batch, int hq, int hkv, int d, int bs,
                               int max_blocks, int device, bool least) {
  const int G = hq / hkv;
  return plan_layout(nullptr, total_q, batch, G, hkv, d, bs, max_blocks, sm_count(device),
                     !least && use_ready(total_q, batch, G, hkv, d, bs, max_blocks), nullptr);
}

cudaError_t launch_prefill(const PrefillArgs& args, cudaStream_t stream) {
  PrefillArgs a = args;
  const bool fast = a.cap <= kCapFast;
  a.cap_in = a.cap > 0.f && fast ? 2.f * kLog2e / a.cap : 1.f;
  a.tanh_in = fast ? 0.5f / kLog2e : 1.f / a.cap;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int ranges = sm_count(dev);
  // ready tiles where they pay and the workspace holds them
  const bool ready =
      use_ready(a.total_q, a.batch, a.G, a.hkv, a.d, a.bs, a.max_blocks) &&
      plan_layout(nullptr, a.total_q, a.batch, a.G, a.hkv, a.d, a.bs, a.max_blocks, ranges, true,
                  nullptr) <= a.workspace_bytes;
  PlanView pv;
  plan_layout(static_cast<char*>(a.workspace), a.total_q, a.batch, a.G, a.hkv, a.d, a.bs,
              a.max_blocks, ranges, ready, &pv);
  const int var = a.cap > 0.f ? 2 : (a.slopes ? 1 : 0);
  const bool mx = a.mode == FP8PA_SCALE_MX_BLOCK;
  const PrefillKernels fn = a.d == 128 ? pick_prefill_d128(a.fmt, var, mx, ready)
                                       : pick_prefill_d64(a.fmt, var, mx, ready);
  if ((e = ensure_smem_attr(reinterpret_cast<const void*>(fn.attend), fn.smem)) != cudaSuccess)
    return e;

  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  if (ready) {
    cfg.gridDim = dim3(static_cast<unsigned>(pv.tpr) * a.batch * a.hkv);
    cfg.blockDim = dim3(256);
    if ((e = cudaLaunchKernelEx(&cfg, fn.make, a, pv)) != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreads);
  if ((e = cudaLaunchKernelEx(&cfg, prefill_plan_kernel, a, pv, ranges)) != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(ranges));
  cfg.blockDim = dim3(static_cast<unsigned>(fn.threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(fn.smem);
  if ((e = cudaLaunchKernelEx(&cfg, fn.attend, a, pv)) != cudaSuccess) return e;
  if (ranges < 2) return cudaSuccess;
  cfg.gridDim = dim3(static_cast<unsigned>(ranges - 1), kRows / kMergeRows);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return a.d == 128 ? cudaLaunchKernelEx(&cfg, prefill_merge_kernel<128>, a, pv, ranges)
                    : cudaLaunchKernelEx(&cfg, prefill_merge_kernel<64>, a, pv, ranges);
}

}  // namespace fp8pa
