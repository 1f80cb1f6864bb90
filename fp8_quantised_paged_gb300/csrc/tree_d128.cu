// tree_d128.cu -- the tree attention's instances for head_dim 128.
#include "tree.cuh"

namespace fp8pa {

TreeKernel pick_tree_d128(bool raw, bool st, int var) { return pick_tree<128>(raw, st, var); }

}  // namespace fp8pa
