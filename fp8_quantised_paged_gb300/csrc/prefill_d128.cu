// prefill_d128.cu -- the prefill kernel's instances for head_dim 128.
#include "prefill.cuh"

namespace fp8pa {

PrefillFn pick_prefill_d128(int fmt, int var, bool mx, int* smem) {
  return pick_fmt<128>(fmt, var, mx, smem);
}

}  // namespace fp8pa
