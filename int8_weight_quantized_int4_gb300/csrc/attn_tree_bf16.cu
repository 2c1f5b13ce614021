// attn_tree_bf16.cu -- attention of trees over a paged cache of bf16 (see attn_tree.cuh).
#include "attn_tree.cuh"

namespace qw {
cudaError_t launch_attn_tree_bf16(const TreeArgs &a, int d, int grid, cudaStream_t st) {
  return launch_tree_kv<kPagedBf16>(a, d, grid, st);
}
}  // namespace qw
