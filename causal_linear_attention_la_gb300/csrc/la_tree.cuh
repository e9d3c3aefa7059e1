// Shared by the tree-decode kernels: the path of every node of a drafted tree.
#pragma once

#include "la_spec.cuh"

namespace la {

// The parent of node i, -1 for a child of the committed state. Anything that
// is not an earlier node counts as -1, so that a walk up the parents ends and
// no index leaves the tree whatever the caller's array holds.
__device__ __forceinline__ int tree_parent(const int* parent, int i) {
  const int p = parent[i];
  return p >= 0 && p < i ? p : -1;
}

// The nodes on node i's path, i among them, as a bit mask. `par` holds the
// sanitised parents.
__device__ __forceinline__ unsigned long long tree_path_mask(const int* par, int i) {
  unsigned long long m = 0ull;
  for (int p = i; p >= 0; p = par[p]) m |= 1ull << p;
  return m;
}

// a^n for 0 <= n <= kTreeMax by squaring: at most 12 roundings, and exact for
// a = 0 and a = 1, where exp2(n log2 a) would give 0 * inf.
__device__ __forceinline__ float tree_power(float a, int n) {
  float r = 1.f;
  for (; n > 0; n >>= 1, a *= a)
    if (n & 1) r *= a;
  return r;
}

__device__ __forceinline__ int clamp_count(const int* count, int b, int T) {
  return count == nullptr ? T : min(max(count[b], 0), T);
}

}  // namespace la
