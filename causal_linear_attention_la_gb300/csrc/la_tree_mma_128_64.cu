// Tree decode on the tensor cores, dk = 128, dv = 64.
#include "la_tree_small.cuh"
#include "la_tree_wide.cuh"

namespace la {
cudaError_t tree_mma_128_64(const TreeArgs& a) {
  if (a.T <= treesmall::TP)
    return a.z == nullptr ? treesmall::launch<128, 64, true>(a) : treesmall::launch<128, 64, false>(a);
  return a.z == nullptr ? treewide::launch<128, 64, true>(a) : treewide::launch<128, 64, false>(a);
}
}  // namespace la
