// The instances of tree_narrow.cuh for groups of sequences over what they share.
#include "tree_narrow.cuh"

namespace wise {

template cudaError_t launch_tree_narrow<true>(const TreeParams&, const CUtensorMap*, cudaStream_t);

}  // namespace wise
