// tree_d64.cu -- the tree attention's instances for head_dim 64.
#include "tree.cuh"

namespace fp8pa {

TreeKernel pick_tree_d64(bool raw, bool st, int var) { return pick_tree<64>(raw, st, var); }

}  // namespace fp8pa
