// prefill_d64.cu -- the prefill kernel's instances for head_dim 64.
#include "prefill.cuh"

namespace fp8pa {

PrefillFn pick_prefill_d64(int fmt, int var, bool mx, int* smem) {
  return pick_fmt<64>(fmt, var, mx, smem);
}

}  // namespace fp8pa
