// Tree decode on the tensor cores, dk = 64, dv = 128.
#include "la_tree_mma.cuh"

namespace la {
cudaError_t tree_mma_64_128(const TreeArgs& a) { return treemma::dispatch<64, 128>(a); }
}  // namespace la
