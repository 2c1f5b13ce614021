// attn_tree_i8.cu -- attention of trees over a paged cache of int8 (see attn_tree.cuh).
#include "attn_tree.cuh"

namespace qw {
cudaError_t launch_attn_tree_i8(const TreeArgs &a, int d, int grid, cudaStream_t st) {
  return launch_tree_kv<kPagedI8>(a, d, grid, st);
}
}  // namespace qw
