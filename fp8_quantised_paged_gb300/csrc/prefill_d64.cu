// prefill_d64.cu -- the prefill kernel's instances for head_dim 64.
#include "prefill.cuh"

namespace fp8pa {

PrefillKernels pick_prefill_d64(int fmt, int var, bool mx, bool ready) {
  return pick_fmt<64>(fmt, var, mx, ready);
}

}  // namespace fp8pa
