// Tree decode on the tensor cores, dk = 64, dv = 64.
#include "la_tree_mma.cuh"

namespace la {
cudaError_t tree_mma_64_64(const TreeArgs& a) { return treemma::dispatch<64, 64>(a); }
}  // namespace la
