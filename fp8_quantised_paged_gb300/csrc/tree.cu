// tree.cu -- the planner and the launch of the tree attention, whose method tree.cuh
// states.
#include "ranges.cuh"
#include "tree.cuh"

namespace fp8pa {

namespace {

// What a tile costs, of a block of at most 128 rows and of a larger one (6 to 10 fifths are within
// 2 % of one another, for MX and INT8 trees of up to 64 nodes).
constexpr int kTileCost = 5, kWideCost = 7;
// What an item costs beside its tiles, 5 or 8 tiles: its time (q laid out, sums added up) is much
// the same in every instance, while a tile takes longer where codes are converted or scores
// capped.  Three ragged batches of 64 requests to 32K, 8 KV heads of 4, in us (the sum of the
// three; 64: dims):
//   cost            8    12    16    20    24    28    32    36    42    47
//   FP8          1073   980   890   797   751   700   670   647   637   646
//   FP8, bias    1080   993   911   813   771   715   698   694   699   711
//   FP8, 64       904   809   731   651   619   578   567   567   576   587
//   FP8, cap     1132  1034   962   872   849   862   875   892   910   929
//   FP8, 64, cap  988   898   834   809   824   842   860   875   896   915
//   INT8         1300  1132  1050  1042  1058  1077  1096  1117  1143  1166
//   INT8, 64     1006   868   777   738   744   763   774   789   807   824
//   MX           1334  1234  1260  1290  1309  1338  1363  1394  1427  1455
//   MX, cap      1498  1361  1331  1356  1374  1402  1428  1459  1491  1514
// Few equal requests have tiles that fall well or badly for a cost, whatever the instance, and
// both values are among the good ones: MX, 64 nodes of 1 x 32K 124, 115, 126 and 115 us at 16,
// 24, 30 and 42, 16 nodes of 8 x 2K 64, 66, 66 and 80; INT8 125, 115, 127, 115 and 57, 59, 58, 69.
inline int item_cost(bool raw, float cap) { return raw && cap == 0.f ? 42 : 24; }

// A request's tree and its visible extent; n is 0 for a request that is skipped, `flag`
// why.
__device__ __forceinline__ Chunk load_tree(const PrefillArgs& a, int b, uint32_t* flag) {
  bool bad_off, bad_len;
  Chunk c = load_chunk(a, b, &bad_off, &bad_len);
  *flag = bad_off ? FP8PA_DEVERR_Q_OFFSETS
                  : (c.n > kMaxTree ? FP8PA_DEVERR_TREE : (bad_len ? FP8PA_DEVERR_SEQ_LEN : 0u));
  if (*flag) c.n = 0;
  c.pre = min(c.pre, c.L - c.n);
  return c;
}

// Block t, of `rows` rows, of a request.  Any node may see the whole context, and the window of a node
// on the first level begins earliest.
__device__ __forceinline__ RowBlock make_tree_block(const Chunk& c, int b, int window, int G,
                                                    int rows, int t) {
  RowBlock r;
  r.b = b;
  r.qlo = c.qlo;
  r.n = c.n;
  r.L = c.L;
  r.pre = c.pre;
  r.row0 = t * rows;
  r.rows = min(rows, c.n * G - r.row0);
  r.pA = c.L - c.n;  // tokens ahead of the tree
  r.pB = c.L - 1;
  r.np = (c.pre + kT - 1) / kT;
  r.skip = max(window_first(window, r.pA) / kT - r.np, 0);
  r.count = (c.L + kT - 1) / kT - r.skip;
  return r;
}

// CTA 0 plans blocks of `rows` rows (cost: of an item); CTA 1 + b writes the lines of request
// b's nodes, a thread each.
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(const PrefillArgs a,
                                                                 const PlanView v,
                                                                 const int32_t* parents,
                                                                 uint32_t* lines, int32_t* depths,
                                                                 int rows, int cost, int ranges) {
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ int s_parent[kMaxTree];
  __shared__ uint32_t s_line[kMaxTree][kLineWords];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  uint32_t flag;
  if (blockIdx.x > 0) {
    const Chunk c = load_tree(a, blockIdx.x - 1, &flag);
    if (tid < c.n) {
      int p = __ldg(parents + c.qlo + tid);
      if (p < -1 || p >= tid) {
        raise_error(a.err, FP8PA_DEVERR_TREE);
        p = -1;
      }
      s_parent[tid] = p;
#pragma unroll
      for (int i = 0; i < kLineWords; ++i) s_line[tid][i] = 0;
    }
    __syncthreads();
    if (tid < c.n) {
      int depth = -1;
      for (int i = tid; i >= 0; i = s_parent[i])  // parents come first
        if (++depth < a.window || a.window == 0) s_line[tid][i >> 5] |= 1u << (i & 31);
      depths[c.qlo + tid] = depth;
    }
    __syncthreads();
    for (int i = tid; i < c.n * kLineWords; i += kPlanThreads)
      lines[static_cast<long>(c.qlo) * kLineWords + i] = s_line[i / kLineWords][i % kLineWords];
    return;
  }
  int carry = 0;
  for (int base = 0; base < a.batch; base += kPlanThreads) {
    const int b = base + tid;
    int n = 0;
    if (b < a.batch) {
      const Chunk c = load_tree(a, b, &flag);
      if (flag) raise_error(a.err, flag);
      // overlapping or repeated offsets cannot add blocks beyond the bound
      n = static_cast<int>((static_cast<long long>(c.n) * a.G + rows - 1) / rows);
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
  int wide = 0;
  for (int base = 0; base < blocks; base += kPlanThreads) {
    const int i = base + tid;
    int n = 0, nw = 0;
    if (i < blocks) {
      const int b = last_le(v.rbase, a.batch, i);
      const Chunk c = load_tree(a, b, &flag);
      const RowBlock r = make_tree_block(c, b, a.window, a.G, rows, i - v.rbase[b]);
      n = r.count;
      nw = r.rows > kTreeRows ? n : 0;
      v.rb[3 * i] = make_int4(r.b, r.qlo, r.n, r.L);
      v.rb[3 * i + 1] = make_int4(r.pre, r.row0, r.rows, r.np);
      v.rb[3 * i + 2] = make_int4(r.skip, r.count, r.pA, r.pB);
    }
    int ex;
    const int total = block_scan(n, &ex, s_warp);
    if (i < blocks) v.rb_pre[i] = carry + ex;
    carry += total;
    const int more = block_scan(nw, &ex, s_warp);
    if (i < blocks) v.rb_wide[i] = wide + ex;
    wide += more;
  }
  if (tid == 0) {
    v.rb_pre[blocks] = carry;
    v.rb_wide[blocks] = wide;
  }
  __syncthreads();
  cut_ranges(v, blocks, carry, a.hkv, ranges, cost, [&](int i) {
    return static_cast<long long>(kTileCost) * v.rb_pre[i] +
           static_cast<long long>(kWideCost - kTileCost) * v.rb_wide[i] +
           static_cast<long long>(cost) * i;
  });
}

size_t tree_layout(char* ws, int total_q, int batch, int G, int d, int ranges, PlanView* v,
                   uint32_t** line, int32_t** depth) {
  const int nb = block_bound(total_q, batch, G, kTreeRows);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = ws + at;
    at += align256(bytes);
    return p;
  };
  PlanView t{};
  t.head = reinterpret_cast<int*>(take(16));
  t.rbase = reinterpret_cast<int*>(take(sizeof(int) * (batch + 1)));
  t.rb = reinterpret_cast<int4*>(take(sizeof(int4) * 3 * nb));
  t.rb_pre = reinterpret_cast<int*>(take(sizeof(int) * (nb + 1)));
  t.rb_wide = reinterpret_cast<int*>(take(sizeof(int) * (nb + 1)));
  t.start = reinterpret_cast<int*>(take(sizeof(int) * (ranges + 1)));
  t.item = reinterpret_cast<int*>(take(sizeof(int) * (ranges + 1)));
  t.ml = reinterpret_cast<float2*>(take(sizeof(float2) * 2 * ranges * kRows));
  t.o = reinterpret_cast<float*>(take(sizeof(float) * 2 * ranges * kRows * d));
  t.blocks = nb;
  char* l = take(sizeof(uint32_t) * kLineWords * total_q);
  char* e = take(sizeof(int32_t) * total_q);
  if (v) {
    *v = t;
    *line = reinterpret_cast<uint32_t*>(l);
    *depth = reinterpret_cast<int32_t*>(e);
  }
  return at;
}

}  // namespace

size_t tree_workspace_bytes(int total_q, int batch, int hq, int hkv, int d, int device) {
  return tree_layout(nullptr, total_q, batch, hq / hkv, d, sm_count(device), nullptr, nullptr,
                     nullptr);
}

cudaError_t launch_tree(const PrefillArgs& args, const int32_t* parents, cudaStream_t stream) {
  PrefillArgs a = args;
  const bool fast = a.cap <= kCapFast;
  a.cap_in = a.cap > 0.f && fast ? 2.f * kLog2e / a.cap : 1.f;
  a.tanh_in = fast ? 0.5f / kLog2e : 1.f / a.cap;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int ranges = sm_count(dev);
  PlanView pv;
  uint32_t* line;
  int32_t* depth;
  tree_layout(static_cast<char*>(a.workspace), a.total_q, a.batch, a.G, a.d, ranges, &pv, &line,
              &depth);
  const int var = a.cap > 0.f ? 2 : (a.slopes ? 1 : 0);
  const bool raw = a.fmt != FP8PA_INT8 && a.mode != FP8PA_SCALE_MX_BLOCK;
  const bool st = a.mode == FP8PA_SCALE_CHANNEL_STATIC;
  const TreeKernel fn = a.d == 128 ? pick_tree_d128(raw, st, var) : pick_tree_d64(raw, st, var);
  if ((e = ensure_smem_attr(reinterpret_cast<const void*>(fn.fn), fn.smem)) != cudaSuccess)
    return e;
  CUtensorMap mk{}, mv{};
  if (raw) {
    const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.hkv * a.bs;
    const CUtensorMapSwizzle swz =
        a.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    if (!encode_tensor_map_2d_u8(&mk, a.k_cache, a.d, rows, a.d, a.bs, swz) ||
        !encode_tensor_map_2d_u8(&mv, a.v_cache, a.d, rows, a.d, a.bs, swz))
      return cudaErrorInvalidValue;
  }

  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(1u + static_cast<unsigned>(a.batch));
  cfg.blockDim = dim3(kPlanThreads);
  if ((e = cudaLaunchKernelEx(&cfg, tree_plan_kernel, a, pv, parents, line, depth,
                              raw ? kTreeRows : kRows, item_cost(raw, a.cap), ranges)) !=
      cudaSuccess)
    return e;
  cfg.gridDim = dim3(static_cast<unsigned>(ranges));
  cfg.blockDim = dim3(static_cast<unsigned>(fn.threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(fn.smem);
  const TreeView tv{line, depth, make_fast_div(static_cast<uint32_t>(a.G))};
  if ((e = cudaLaunchKernelEx(&cfg, fn.fn, a, pv, tv, mk, mv)) != cudaSuccess) return e;
  return launch_merge_ranges(a, pv, ranges, stream);
}

}  // namespace fp8pa
