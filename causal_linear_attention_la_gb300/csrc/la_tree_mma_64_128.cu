// Tree decode on the tensor cores, dk = 64, dv = 128.
#include "la_tree_small.cuh"
#include "la_tree_wide.cuh"

namespace la {
cudaError_t tree_mma_64_128(const TreeArgs& a) {
  if (a.T <= treesmall::TP)
    return a.z == nullptr ? treesmall::launch<64, 128, true>(a) : treesmall::launch<64, 128, false>(a);
  return a.z == nullptr ? treewide::launch<64, 128, true>(a) : treewide::launch<64, 128, false>(a);
}
}  // namespace la
