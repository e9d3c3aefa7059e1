// Tree decode on the tensor cores, dk = 128, dv = 64.
#include "la_tree_small.cuh"
#include "la_tree_wide.cuh"

namespace la {
cudaError_t tree_mma_128_64(const TreeArgs& a) {
  const bool delta = a.z == nullptr;
  if (a.T <= treesmall::TP) return delta ? treesmall::launch<128, 64, true>(a) : treesmall::launch<128, 64, false>(a);
  if (a.T <= 32) return delta ? treewide::launch<128, 64, 32, true>(a) : treewide::launch<128, 64, 32, false>(a);
  return delta ? treewide::launch<128, 64, 64, true>(a) : treewide::launch<128, 64, 64, false>(a);
}
}  // namespace la
