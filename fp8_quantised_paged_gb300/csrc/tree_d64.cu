// tree_d64.cu -- the tree attention's instances for head_dim 64.
#include "tree.cuh"

namespace fp8pa {

TreeKernel pick_tree_d64(bool raw, int var) {
  return raw ? pick_tree<64, true>(var) : pick_tree<64, false>(var);
}

}  // namespace fp8pa
