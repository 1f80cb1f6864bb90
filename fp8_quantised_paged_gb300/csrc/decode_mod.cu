// decode_mod.cu -- grouped-query decode with score modifiers: a sliding
// window, an always-visible prefix, tanh-capped scores and a distance bias.
//
//   z_j = sm_scale q . k^_j;  z_j = cap tanh(z_j / cap);  z_j -= slope |i - j|
//   out = sum_j softmax(z)_j v^_j over j < prefix or i - window < j <= i
//
// The split kernel of decode_gqa.cu (gqa_split.cuh) with the modifiers applied
// to a tile's scores in registers.  It is bound by the codes and scales that
// it streams from HBM, so what counts is which pages are read: the planner
// below counts only the pages of the prefix and of the window, and the split
// kernel's cursor steps over the gap between them.
//
// 4 requests of 131072 tokens with a distance bias: 202 us, 5.5 TB/s (82% of a
// plain copy's rate).  12 of 16384 under a window of 4096: 35 us for 104 MB, where the
// plain decode of 12 of 4100 takes 33: 15 are the bytes at the streaming rate, the rest
// what every split launch pays (its prologue, the first pages' latency, the tail) and
// the planner and the merge around it; 48 of them, 415 MB, take 90.  64 ragged requests,
// 546 MB of static-scale codes under capped scores: 127 us, 4.3 TB/s, with two CTAs on
// an SM (this variant keeps to 128 registers; with the plain kernel's one CTA, 167 us);
// the cap is 2.5 us of it.  Without modifiers set, 12 of 16384 take 85 us a call, the
// plain decode's 80.6: the modifiers' own instructions cost 6%.
#include "gqa_split.cuh"

namespace fp8pa {

namespace {

__global__ void __launch_bounds__(32) plan_mod_kernel(const int32_t* seq_lens, ScoreMods mods,
                                                      int B, int bs, int max_blocks, int workers,
                                                      int* ws, uint32_t* err) {
  griddep_wait();
  griddep_launch_dependents();
  plan_warp_pages(B, 1, workers, ws, [&](int b) {
    bool bad;
    const int L = visible_len(seq_lens, b, 1, max_blocks * bs, &bad);
    if (bad) raise_error(err, FP8PA_DEVERR_SEQ_LEN);
    const int np = (prefix_len(mods, b, L) + bs - 1) / bs;
    return (L + bs - 1) / bs - max(window_first(mods, L - 1) / bs - np, 0);
  });
}

}  // namespace

cudaError_t launch_decode_mod(const DecodeShape& s, const DecodeArgs& a, const ScoreMods& mods,
                              size_t workspace_bytes, cudaStream_t stream) {
  const int G = s.hq / s.hkv;
  const auto k = pick<GqaModParams>(s.d, s.bs, a.fmt, kernel_mode(a.mode, G, a.gs));
  const void* fn = reinterpret_cast<const void*>(k.fn);
  const int wpc = gqa_wpc(s.hkv, 1, k), hsets = s.hkv / wpc;
  const int smem = k.smem(wpc);
  cudaError_t e = ensure_smem_attr(fn, smem);
  if (e != cudaSuccess) return e;
  // One page range per resident CTA of this kernel, or the plain decode's number
  // where that is less and the workspace holds no more (the size function's answer
  // is for the scale mode with the most ranges, and holds them).
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  int workers = s.workers;
  if (g_decode_workers_override <= 0) {
    DecodeShape own = s;
    own.workers = max(1, sm_count(dev) * ctas_per_sm(fn, wpc * 32, smem) / hsets);
    if (own.workers < workers || decode_workspace_bytes(own) <= workspace_bytes)
      workers = own.workers;
  }

  CUtensorMap tmk, tmv;
  const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * s.hkv * s.bs;
  const CUtensorMapSwizzle swz =
      s.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!encode_tensor_map_2d_u8(&tmk, a.k_cache, s.d, rows, s.d, 16, swz) ||
      !encode_tensor_map_2d_u8(&tmv, a.v_cache, s.d, rows, s.d, 16, swz))
    return cudaErrorInvalidValue;

  char* ws = static_cast<char*>(a.workspace);
  int* plan = reinterpret_cast<int*>(ws);
  const size_t plan_bytes = align256(sizeof(int) * (kPlanHeader + 2 * (s.batch + 1)));
  const size_t prow = (static_cast<size_t>(workers) + s.batch) * s.hkv * G;
  float* part_ml = reinterpret_cast<float*>(ws + plan_bytes);
  float* part_o = reinterpret_cast<float*>(ws + plan_bytes + align256(prow * 2 * sizeof(float)));

  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(32);
  e = cudaLaunchKernelEx(&cfg, plan_mod_kernel, a.seq_lens, mods, s.batch, s.bs, s.max_blocks,
                         workers, plan, a.err);
  if (e != cudaSuccess) return e;

  GqaModParams p;
  p.q = a.q;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.block_tables = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.plan = plan;
  p.part_ml = part_ml;
  p.part_o = part_o;
  p.err = a.err;
  p.B = s.batch;
  p.hq = s.hq;
  p.hkv = s.hkv;
  p.G = G;
  p.max_blocks = s.max_blocks;
  p.num_blocks = a.num_blocks;
  p.qlen = 1;
  p.qw = 1;
  p.gs = a.gs;
  p.hp = segment_scale_heads(s.hkv);
  p.qk_scale_log2 = a.sm_scale * kLog2e;
  p.mods = mods;
  p.sm_scale = a.sm_scale;
  cfg.gridDim = dim3(static_cast<unsigned>(workers) * hsets);
  cfg.blockDim = dim3(wpc * 32);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, k.fn, tmk, tmv, p);
  if (e != cudaSuccess) return e;
  return launch_merge(plan, part_ml, part_o, a.out, s.batch, 1, s.hq, s.hkv, G, s.dv, a.out_dtype,
                      stream);
}

}  // namespace fp8pa
