// The instances of tree_narrow.cuh for a cache's own sequences.
#include "tree_narrow.cuh"

namespace wise {

template cudaError_t launch_tree_narrow<false>(const TreeParams&, const CUtensorMap*, cudaStream_t);

}  // namespace wise
