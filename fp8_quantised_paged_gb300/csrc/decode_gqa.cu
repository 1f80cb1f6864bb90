// decode_gqa.cu -- split-K paged decode attention for grouped-query heads.
//
// Method ("Llama 3 70B FP8 deployment", dpshk.com/news/5605006, sec. 1.2:
// GQA; "DeepSeek V4 950", 2kiu.com/news/4508674, sec. 2.3: softmax and
// accumulation in FP32; "DeepSeek-V4.1 512K", hotelren.com/news/5711065,
// sec. 2.2: blockwise attention with an online softmax, sec. 3.3: paged
// blocks through a per-request block table):
//   out[b][h] = sum_t softmax_t(sm_scale * q[b][h] . k^_t) v^_t,
//   k^ = decode(code) * scale, query head h reading KV head h / G.
//
// GB300 design.
//  * Work is the flat list of units (request b, page j).  The planner
//    (plan.cuh) cuts it into equal contiguous ranges, one per resident CTA.
//    A CTA's warps are the KV heads of one head set and walk the range's
//    pages together, so they read each block's adjacent per-head slices.  A
//    range that crosses a request boundary yields one partial per request;
//    the merge (merge.cu) folds the partials of each output row with the
//    log-sum-exp rule.  Balance is exact for ragged batches and a
//    128K-token request spreads over the whole GPU.
//  * Each warp streams its pages, as 16-token slices, through a private
//    ring of shared-memory stages filled by the tensor-copy engine (TMA,
//    2-D boxes of 16 x head_dim bytes with the 128/64-byte swizzle) plus 1-D
//    bulk copies of the per-token scales, completion tracked by mbarriers.
//    One lane issues; no thread waits on another CTA.  Every wait is
//    bounded.
//  * The G <= 8 heads sharing a KV head form a tiny dense contraction
//    (16 tokens x 8 heads x head_dim per tile).  GB300's FP32 pipe cannot
//    keep up with HBM on it (about 8 FMA per cached byte), so QK^T and PV
//    run on warp MMA (m16n8k16, f16 in, f32 accumulate) over codes (FP8 or
//    INT8) converted exactly to f16 in registers.  Scales stay outside the
//    contraction: the per-token K scale multiplies the score, the per-token
//    V scale folds into P, per-channel K scales fold into q (as an f16 high
//    and low part; with G <= 4 both parts share one MMA's head columns),
//    per-channel V scales multiply the output; MX block exponents scale the
//    f16 fragments by exact powers of two.  Power-of-two normalisers keep q
//    and P inside f16's range.
//  * Softmax runs in FP32 in the log2 domain with warp-shuffle maxima.
#include "gqa_split.cuh"

namespace fp8pa {

namespace {

// ---------------------------------------------------------------- planner
// One warp; lets the split kernel launch at once (it waits for the plan).
__global__ void __launch_bounds__(32) plan_kernel(const int32_t* seq_lens, int B, int qlen,
                                                  int qw, int groups, int bs, int max_blocks,
                                                  int workers, int* ws, uint32_t* err,
                                                  int upages) {
  griddep_wait();  // inputs may come from the kernel before us in the stream
  griddep_launch_dependents();
  plan_warp(seq_lens, B, qlen, qw, groups, bs, max_blocks, workers, ws, err, upages);
}

}  // namespace

int g_decode_workers_override = 0;
cudaEvent_t g_split_ev_start = nullptr, g_split_ev_stop = nullptr;

// Number of page ranges the planner cuts (GQA: one per resident CTA over the
// head sets; MLA: one per SM over the head groups, times the head groups).
int decode_workers(const DecodeShape& s, int fmt, int mode, int device) {
  const int sms = sm_count(device);
  if (s.mla) {
    // one CTA per SM (202 or 221 KB of shared memory); a whole number of
    // head-group sets (H = Hq / 32, or Hq / 64 on tensor cores)
    const int H = s.hq / mla_group_heads(s);
    int ranges = (g_decode_workers_override > 0 ? g_decode_workers_override : sms) / H;
    return (ranges < 1 ? 1 : ranges) * H;
  }
  if (g_decode_workers_override > 0) return g_decode_workers_override;
  if (s.gqa_tc) return gqa_tc_workers(s, device);
  const auto k = pick<GqaParams>(s.d, s.bs, fmt, kernel_mode(mode, s.hq / s.hkv, s.gs));
  const int qw = gqa_qw(s);
  const int wpc = gqa_wpc(s.hkv, qw, k), hsets = s.hkv / (wpc / qw);
  const int per_sm = ctas_per_sm(reinterpret_cast<const void*>(k.fn), wpc * 32, k.smem(wpc));
  const int ranges = sms * per_sm / hsets;
  return ranges < 1 ? 1 : ranges;
}

// Pieces are numbered per request (the planner runs over pages only) and
// each piece holds one row per head group (KV head for GQA, 32-head group for
// MLA) and query head of the group.
size_t decode_workspace_bytes(const DecodeShape& s) {
  const int groups = s.mla ? s.hq / mla_group_heads(s) : s.hkv;
  const int G = s.hq / groups;
  const int qw = s.mla ? 1 : gqa_qw(s);
  const size_t bp = s.batch / qw;  // planned requests
  const size_t ranges = s.mla ? static_cast<size_t>(s.workers / groups) : s.workers;
  const size_t plan = align256(sizeof(int) * (kPlanHeader + 2 * (bp + 1)));
  const size_t rows = (ranges + bp) * groups * qw * G;
  const size_t ml = align256(rows * 2 * sizeof(float));
  const size_t o = align256(rows * static_cast<size_t>(s.dv) * sizeof(float));
  return plan + ml + o;
}

cudaError_t launch_decode_gqa(const DecodeShape& s, const DecodeArgs& a, cudaStream_t stream) {
  if (s.gqa_tc) return launch_decode_gqa_tc(s, a, stream);
  const int G = s.hq / s.hkv;
  const auto k = pick<GqaParams>(s.d, s.bs, a.fmt, kernel_mode(a.mode, G, a.gs));
  const int qw = gqa_qw(s);
  const int bp = s.batch / qw;  // planned requests
  const int wpc = gqa_wpc(s.hkv, qw, k), hsets = s.hkv / (wpc / qw);
  const int smem = k.smem(wpc);
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(k.fn), smem);
  if (e != cudaSuccess) return e;

  CUtensorMap tmk, tmv;
  const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * s.hkv * s.bs;
  const CUtensorMapSwizzle swz =
      s.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!encode_tensor_map_2d_u8(&tmk, a.k_cache, s.d, rows, s.d, 16, swz) ||
      !encode_tensor_map_2d_u8(&tmv, a.v_cache, s.d, rows, s.d, 16, swz))
    return cudaErrorInvalidValue;

  char* ws = static_cast<char*>(a.workspace);
  int* plan = reinterpret_cast<int*>(ws);
  const size_t plan_bytes = align256(sizeof(int) * (kPlanHeader + 2 * (bp + 1)));
  const size_t prow = (static_cast<size_t>(s.workers) + bp) * s.hkv * qw * G;
  float* part_ml = reinterpret_cast<float*>(ws + plan_bytes);
  float* part_o = reinterpret_cast<float*>(ws + plan_bytes + align256(prow * 2 * sizeof(float)));

  if (!a.plan_ready) {
    e = launch_plan(a.seq_lens, bp, s.qlen, qw, 1, s.bs, s.max_blocks, s.workers, plan, a.err,
                    stream);
    if (e != cudaSuccess) return e;
  }
  // Every kernel of the decode is launched with programmatic stream
  // serialisation: it may start while its predecessor drains, and waits
  // (griddepcontrol.wait) before reading anything that predecessor wrote.
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  GqaParams p;
  p.q = a.q;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.block_tables = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.plan = plan;
  p.part_ml = part_ml;
  p.part_o = part_o;
  p.err = a.err;
  p.B = bp;
  p.hq = s.hq;
  p.hkv = s.hkv;
  p.G = G;
  p.max_blocks = s.max_blocks;
  p.num_blocks = a.num_blocks;
  p.qlen = s.qlen;
  p.qw = qw;
  p.gs = a.gs;
  p.hp = segment_scale_heads(s.hkv);
  p.qk_scale_log2 = a.sm_scale * 1.4426950408889634f;
  cfg.gridDim = dim3(static_cast<unsigned>(s.workers) * hsets);
  cfg.blockDim = dim3(wpc * 32);
  cfg.dynamicSmemBytes = smem;
  if (g_split_ev_start) cudaEventRecord(g_split_ev_start, stream);
  e = cudaLaunchKernelEx(&cfg, k.fn, tmk, tmv, p);
  if (e != cudaSuccess) return e;
  if (g_split_ev_stop) cudaEventRecord(g_split_ev_stop, stream);

  return launch_merge(plan, part_ml, part_o, a.out, bp, qw, s.hq, s.hkv, G, s.dv, a.out_dtype,
                      stream);
}

cudaError_t launch_plan(const int32_t* seq_lens, int batch, int qlen, int qw, int groups, int bs,
                        int max_blocks, int workers, int* plan, uint32_t* err,
                        cudaStream_t stream, int upages) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(32);
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_kernel, seq_lens, batch, qlen, qw, groups, bs, max_blocks,
                            workers, plan, err, upages);
}

}  // namespace fp8pa
