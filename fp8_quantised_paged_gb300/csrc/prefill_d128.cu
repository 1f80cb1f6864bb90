// prefill_d128.cu -- the prefill kernel's instances for head_dim 128.
#include "prefill.cuh"

namespace fp8pa {

PrefillKernels pick_prefill_d128(int fmt, int var, bool mx, bool ready) {
  return pick_fmt<128>(fmt, var, mx, ready);
}

}  // namespace fp8pa
