// Internal declarations of the speculative-decoding operators: tree decode,
// draft verification, state advance and the packed state pool.
#pragma once

#include "la_internal.cuh"

namespace la {

constexpr int kTreeMax = 64;   // nodes per tree (LA_TREE_MAX): one 64-bit ancestor mask each

struct TreeArgs {
  const float* S; const float* z;            // z null: delta rule
  const void* q; const void* k; const void* v;
  const int* parent; const int* count;       // count null: T nodes everywhere
  void* out;
  int BH, H, T, dk, dv;
  const float* alpha;                        // null: no decay
  float eps; la_dtype dtype;
  cudaStream_t stream;
};

struct AdvanceArgs {
  const float* S; const float* z; float* S_out; float* z_out;   // z null: delta rule
  const void* k; const void* v;
  const int* path; const int* accepted;      // null: rows 0, 1, ...; null: T tokens
  int BH, H, T, dk, dv;
  const float* alpha; la_dtype dtype;
  cudaStream_t stream;
};

struct VerifyArgs {
  const void* target; const void* draft;     // draft null: tree form
  const int* tokens; const int* parent; const int* count;
  const float* uniform;
  int* path; int* accepted; int* next;       // path: tree form only
  int B, T, V; la_dtype dtype;
  cudaStream_t stream;
};

struct PackArgs {
  float* S; float* z;                        // z null: none stored
  unsigned char* codes; unsigned char* scales; float* z_pool;
  const int* slot;
  int B, H, dk, dv, slots;
  cudaStream_t stream;
};

// Tree decode: on the CUDA cores (any head sizes and types), and on the tensor
// cores where tree_on_tensor_cores says so.
cudaError_t simt_tree(const TreeArgs& a);
cudaError_t tree_mma_64_64(const TreeArgs& a);
cudaError_t tree_mma_64_128(const TreeArgs& a);
cudaError_t tree_mma_128_64(const TreeArgs& a);
cudaError_t tree_mma_128_128(const TreeArgs& a);
inline bool tree_on_tensor_cores(int dk, int dv, la_dtype dtype) {
  return dtype == LA_BF16 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128);
}
cudaError_t state_advance(const AdvanceArgs& a);
cudaError_t verify(const VerifyArgs& a);
cudaError_t state_pack(const PackArgs& a);
cudaError_t state_unpack(const PackArgs& a);

// One-shot test switch (la_test_timeout_next_tree): true once after the
// switch has been set.
bool take_tree_timeout_test();

// The current la_set_path setting.
int current_path();

}  // namespace la
