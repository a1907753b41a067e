// Attention of new tokens over a paged cache: the instances of tree_wide.cuh for a
// cache's own sequences.
#include "tree_wide.cuh"

namespace wise {

template cudaError_t launch_tree_rows<false>(const TreeLaunch&, const CUtensorMap*, cudaStream_t);

int64_t tree_workspace_bytes(int32_t batch, int32_t kv_heads, int32_t heads, int32_t n, int32_t head_dim) {
  const int64_t rows = (int64_t)(heads / kv_heads) * n;
  return workspace_layout(tree_units(batch, kv_heads, rows), rows, head_dim, false).bytes;
}

cudaError_t launch_tree(const TreeLaunch& t, const CUtensorMap* maps, cudaStream_t stream) {
  return launch_tree_rows<false>(t, maps, stream);
}

}  // namespace wise
