// Tree decode on the tensor cores, dk = 128, dv = 64.
#include "la_tree_mma.cuh"

namespace la {
cudaError_t tree_mma_128_64(const TreeArgs& a) { return treemma::dispatch<128, 64>(a); }
}  // namespace la
