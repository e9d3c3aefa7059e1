// Tree decode on the tensor cores, dk = 128, dv = 128.
#include "la_tree_mma.cuh"

namespace la {
cudaError_t tree_mma_128_128(const TreeArgs& a) { return treemma::dispatch<128, 128>(a); }
}  // namespace la
