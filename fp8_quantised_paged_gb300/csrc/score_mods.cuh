// score_mods.cuh -- the score modifiers of the decode and prefill calls: a
// tanh cap, a distance bias, a sliding window and an always-visible prefix.
#pragma once

#include "common.cuh"

namespace fp8pa {

constexpr float kLog2e = 1.4426950408889634f;

struct ScoreMods {
  const int32_t* prefix_lens;  // [requests] or NULL
  const float* slopes;         // [n_q_heads] or NULL
  float cap;                   // 0: scores are not capped
  int window;                  // 0: none
};

// Visible keys of a query at position `pos` of a request of `L` cached
// tokens: [first, last] and [0, prefix).
__device__ __forceinline__ int prefix_len(const ScoreMods& m, int b, int L) {
  return m.prefix_lens ? min(max(__ldg(m.prefix_lens + b), 0), L) : 0;
}
// (Compared before it is subtracted: a window may be any int, and the positions of a
// chunk longer than its request begin below zero.)
__device__ __forceinline__ int window_first(int window, int pos) {
  return window > 0 && pos >= window ? pos - window + 1 : 0;
}
__device__ __forceinline__ int window_first(const ScoreMods& m, int pos) {
  return window_first(m.window, pos);
}

// Caps up to this take tanh as 1 - 2 / (2^x + 1), x = 2 log2(e) z / cap, whatever
// x is: the quotient is good to 2^-21, so the score is off by 2^-20 cap at most,
// 2^-14 here, for two special-function operations and three others.  Larger caps
// need tanh_f32, good relative to the score: 2048 queries over a window of 4096 take
// 751 us under a cap of 100, 466 under one of 50; 64 ragged decodes 135 and 128.
constexpr float kCapFast = 64.f;
// The cap that the kernels take.  Scores within 2^-60 of zero weigh the same, to 2^-59,
// so a smaller cap is this one, whose 2 / cap leaves the scores' factors in fp32.
// Larger caps scale z by 1 / cap, which fp32 holds (FLT_MAX's as a subnormal, off by
// 2^-150 and so by 2^-22 of z), and multiply the tanh by cap before log2(e), as cap
// log2(e) need not be finite.
inline float kernel_cap(float cap) { return cap > 0.f ? (cap < 0x1p-60f ? 0x1p-60f : cap) : 0.f; }
// 1 / x, good to 2^-23; 0 for an infinity.
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// cap tanh(z / cap) in the log2 domain, cap_log2 = cap log2(e).
__device__ __forceinline__ float cap_fast(float x, float cap_log2) {
  return fmaf(rcp_fast(ex2(x) + 1.f), -2.f * cap_log2, cap_log2);
}

// tanh x to a relative error of about 2^-21, so that cap * tanh(z / cap) is
// as near to z as fp32 for any cap.  Above 0.55, 1 - 2 / (e^2|x| + 1) loses at
// most one bit to the subtraction; below, the Taylor series to x^13, whose
// first dropped term is 1.46e-3 x^14 = 3.4e-7 of x at 0.55.
__device__ __forceinline__ float tanh_f32(float x) {
  const float x2 = x * x;
  float p = 21844.0f / 6081075.0f;
  p = fmaf(p, x2, -1382.0f / 155925.0f);
  p = fmaf(p, x2, 62.0f / 2835.0f);
  p = fmaf(p, x2, -17.0f / 315.0f);
  p = fmaf(p, x2, 2.0f / 15.0f);
  p = fmaf(p, x2, -1.0f / 3.0f);
  const float small = fmaf(p * x2, x, x);
  const float a = fabsf(x);
  const float e = ex2(a * (2.0f * kLog2e));
  const float big = copysignf(1.0f - __fdividef(2.0f, e + 1.0f), x);
  return a < 0.55f ? small : big;
}

}  // namespace fp8pa
