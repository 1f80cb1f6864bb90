// tree_d128.cu -- the tree attention's instances for head_dim 128.
#include "tree.cuh"

namespace fp8pa {

TreeKernel pick_tree_d128(bool raw, int var) {
  return raw ? pick_tree<128, true>(var) : pick_tree<128, false>(var);
}

}  // namespace fp8pa
