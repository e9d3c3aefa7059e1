// Tree decode on the tensor cores, dk = 64, dv = 128.
#include "la_tree_small.cuh"
#include "la_tree_wide.cuh"

namespace la {
cudaError_t tree_mma_64_128(const TreeArgs& a) {
  const bool delta = a.z == nullptr;
  if (a.T <= treesmall::TP) return delta ? treesmall::launch<64, 128, true>(a) : treesmall::launch<64, 128, false>(a);
  if (a.T <= 32) return delta ? treewide::launch<64, 128, 32, true>(a) : treewide::launch<64, 128, 32, false>(a);
  return delta ? treewide::launch<64, 128, 64, true>(a) : treewide::launch<64, 128, 64, false>(a);
}
}  // namespace la
