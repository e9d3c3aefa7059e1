// Internal declarations of the gated delta rule (forward, backward, steps) and
// of the norm with rotation that feeds it.
#pragma once

#include "la_internal.cuh"

namespace la {

// One-shot test switch (la_test_timeout_next_gated): true once after the host
// asked for it. The chains' (0) or the gradients' (1) next tensor-core launch takes it.
bool take_gated_timeout_test(int kernel);

// Shapes and inputs of a call over whole sequences: packed ones with offsets,
// nseq = B of N tokens without.
struct GatedArgs {
  const void* q; const void* k; const void* v;
  const float* g; const float* beta;
  const float* S0; float* S_final;             // either may be null
  const int* offsets;                          // null: sequences of N tokens
  void* out;
  // backward
  const void* dout; const float* dS; float* dS0;
  void* dq; void* dk_; void* dv_; void* dg; void* dbeta;
  int B, Hk, H, N, dk, dv, nseq;
  float scale; la_dtype dtype;
  void* workspace; size_t workspace_bytes;
  cudaStream_t stream;
};

struct GatedStepArgs {
  const float* S; float* S_out;
  const void* q; const void* k; const void* v;
  const float* g; const float* beta; const int* count;
  void* out;
  int B, Hk, H, T, dk, dv;
  float scale; la_dtype dtype;
  cudaStream_t stream;
};

// A sequence's rows: sequence s of [heads][rows] arrays starts at row `lo` of
// batch `b` and has n tokens. Chunk slots: a sequence's chunks of C tokens take
// consecutive slots from `slot` on, no two sequences the same (lo / C + s where
// sequences are packed: there are ceil(n / C) <= (hi / C - lo / C) + 1 of them).
struct SeqRange {
  int b; int lo; int n; int slot;
};
__device__ __forceinline__ SeqRange seq_range(const int* offsets, int s, int N, int C) {
  SeqRange r;
  if (offsets == nullptr) {
    r.b = s; r.lo = 0; r.n = N; r.slot = s * ((N + C - 1) / C);
  } else {
    r.b = 0;
    r.lo = min(max(offsets[s], 0), N);
    r.n = min(max(offsets[s + 1], r.lo), N) - r.lo;
    r.slot = r.lo / C + s;
  }
  return r;
}
// Which sequence the CTAs number r take, by one whole warp: packed ones the longest
// first, so that no long one begins when the others end (backward of 32 heads, nine sequences of
// 8192 rows: chains 359 us against 439 in their order). Every warp counts the ranks anew, for
// up to 64 of them; more are many short ones.
__device__ __forceinline__ int sequence_of(const int* offsets, int r, int nseq, int N) {
  if (offsets == nullptr || nseq > 64) return r;
  const int lane = threadIdx.x & 31;
  int n[2], rank[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) n[i] = lane + 32 * i < nseq ? seq_range(offsets, lane + 32 * i, N, 1).n : -1;
#pragma unroll
  for (int half = 0; half < 2; ++half)
    for (int j = 32 * half; j < min(nseq, 32 * half + 32); ++j) {
      const int other = __shfl_sync(0xffffffffu, n[half], j & 31);
#pragma unroll
      for (int i = 0; i < 2; ++i) rank[i] += other > n[i] || (other == n[i] && j < lane + 32 * i);
    }
  const unsigned a = __ballot_sync(0xffffffffu, n[0] >= 0 && rank[0] == r);
  const unsigned b = __ballot_sync(0xffffffffu, n[1] >= 0 && rank[1] == r);
  return a != 0 ? __ffs(a) - 1 : 31 + __ffs(b);
}
// The reverse chain (false) or the one that keeps the states of CTA `b` of `grid`, and
// its number among these: reverse ones, which take longer, first, for packed sequences
// those of a sequence (`unit` CTAs) after each other.
__device__ __forceinline__ bool second_chain(unsigned b, unsigned grid, bool packed, unsigned unit, unsigned& number) {
  if (!packed) {
    number = b % (grid / 2);
    return b >= grid / 2;
  }
  const unsigned w = b % (2 * unit);
  number = b / (2 * unit) * unit + w % unit;
  return w >= unit;
}
// Slots that seq_range can give for these sizes.
inline long long chunk_slots(int B, int N, int nseq, bool packed, int C) {
  return packed ? (long long)N / C + nseq : (long long)B * ((N + C - 1) / C);
}
// The chunk of slot `slot`: its sequence, first row and number of tokens (0:
// the slot holds none). The last sequence whose slots start at or before it.
struct ChunkRange {
  int s; int b; int row; int n; int first;     // row: in the batch; first: rows before it in its sequence
};
__device__ __forceinline__ ChunkRange chunk_range(const int* offsets, int nseq, int slot, int N, int C) {
  ChunkRange c;
  int s;
  if (offsets == nullptr) {
    s = slot / ((N + C - 1) / C);
  } else {
    int lo = 0, hi = nseq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (min(max(offsets[mid], 0), N) / C + mid <= slot) lo = mid; else hi = mid - 1;
    }
    s = lo;
  }
  const SeqRange r = seq_range(offsets, s, N, C);
  c.s = s; c.b = r.b;
  c.first = (slot - r.slot) * C;
  c.row = r.lo + c.first;
  c.n = c.first < 0 ? 0 : min(C, r.n - c.first);
  if (c.n < 0) c.n = 0;
  return c;
}

// A log decay as the chunks' sums take it: exp(-128) is zero in fp32, and a sum
// of 64 of them is far from fp64's end. NaN stays.
__device__ __forceinline__ double clamp_log(float g) { return g < -128.f ? -128.0 : (double)g; }

// Token by token on the CUDA cores: any head size and type.
cudaError_t simt_gated_forward(const GatedArgs& a);
cudaError_t simt_gated_backward(const GatedArgs& a);
cudaError_t simt_gated_steps(const GatedStepArgs& a);
size_t simt_gated_backward_workspace(int B, int H, int N, int dk, int dv, int nseq, bool packed);

// Zeros in the rows of `count` arrays [heads][N][row bytes] that no packed sequence has.
constexpr int kClearMost = 8;
cudaError_t clear_outside(void* const* rows, const int* row_bytes, const int* heads, int count, const int* offsets, int N,
                          int nseq, cudaStream_t stream);

// On the tensor cores: bf16, dk and dv in {64, 128}.
inline bool gated_on_tensor_cores(int dk, int dv, la_dtype dtype) {
  return dtype == LA_BF16 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128);
}
cudaError_t mma_gated_forward(const GatedArgs& a);
cudaError_t mma_gated_backward(const GatedArgs& a);
size_t mma_gated_forward_workspace(int B, int H, int N, int dk, int dv, int nseq, bool packed);
size_t mma_gated_backward_workspace(int B, int H, int N, int dk, int dv, int nseq, bool packed);

struct NormArgs {
  const void* x[2]; void* y[2];                // queries, keys
  const float* w[2];
  const int* positions; const float* freqs;
  int B, N, H[2], d, rot;
  long long stride[2][3];
  int l2, interleaved; float eps; la_dtype dtype;
  // backward
  const void* dy[2]; void* dx[2]; float* dw[2];
  long long dstride[2][3];
  float* workspace;
  cudaStream_t stream;
};
cudaError_t norm_rotate(const NormArgs& a);
cudaError_t norm_rotate_backward(const NormArgs& a);
size_t norm_rotate_backward_workspace(int B, int N, int Hq, int Hk, int d, la_dtype dtype);

}  // namespace la
