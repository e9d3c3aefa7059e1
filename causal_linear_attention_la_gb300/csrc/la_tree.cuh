// Shared by the tree-decode kernels: the path of every node of a drafted tree.
#pragma once

#include <atomic>

#include "la_spec.cuh"

namespace la {

// The parent of node i, -1 for a child of the committed state. Anything that
// is not an earlier node counts as -1, so that a walk up the parents ends and
// no index leaves the tree whatever the caller's array holds.
__device__ __forceinline__ int tree_parent(const int* parent, int i) {
  const int p = parent[i];
  return p >= 0 && p < i ? p : -1;
}

// The nodes on each node's path, the node among them, as bit masks, and the
// path's length: one warp, lane l for nodes l and l + 32, by pointer doubling
// (after r rounds a mask holds the nearest 2^r nodes and `up` points past
// them), six rounds for the longest path. Entries n .. n_pad-1 are zero.
// `up` is scratch of kTreeMax ints.
__device__ __forceinline__ void tree_masks(const int* parent, int n, int n_pad, unsigned long long* mask, int* depth,
                                           int* up) {
  const int lane = threadIdx.x & 31;
  unsigned long long m[2];
  int u[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    m[h] = i < n ? 1ull << i : 0ull;
    u[h] = i < n ? tree_parent(parent, i) : -1;
  }
  while (__any_sync(0xffffffffu, u[0] >= 0 || u[1] >= 0)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 32 * h;
      if (i < n) {
        mask[i] = m[h];
        up[i] = u[h];
      }
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (u[h] >= 0) {
        m[h] |= mask[u[h]];
        u[h] = up[u[h]];
      }
    __syncwarp();
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    if (i < n_pad) {
      mask[i] = m[h];
      depth[i] = __popcll(m[h]);
    }
  }
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

// Lets a kernel use `bytes` of dynamic shared memory and counts the CTAs of it
// that the current device holds at once, asked for once per device.
struct KernelOnce {
  static constexpr int kDevices = 64;
  std::atomic<int> held[kDevices] = {};
  template <typename Kernel>
  cudaError_t prepare(Kernel kern, int threads, int bytes, int* resident) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev >= 0 && dev < kDevices;
    *resident = keep ? held[dev].load(std::memory_order_relaxed) : 0;
    if (*resident > 0) return cudaSuccess;
    int sms = 0, per = 0;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, threads, bytes);
    if (e != cudaSuccess) return e;
    *resident = sms * (per > 0 ? per : 1);
    if (keep) held[dev].store(*resident, std::memory_order_relaxed);
    return cudaSuccess;
  }
};

}  // namespace la
