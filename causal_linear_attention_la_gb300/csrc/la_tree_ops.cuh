// Building blocks of the tree decode on the tensor cores (bf16 rows, dk and dv
// in {64, 128}; the formulas are those of la_tree_simt.cu).
//
// The largest operand of the products, the state, is fp32 in memory. A lane
// takes the values that are its own share of the transposed 16 x 16 A operand
// of mma.m16n8k16 and splits them in registers; the nodes are the N of the
// products, which goes in steps of 8:
//   D[c][i] = sum_r S[r][c] x_i[r]         M = values c, N = nodes i, K = keys r
// (tcgen05.mma would want the two parts written to tensor memory first: the
// whole state again as bf16 high and low, 64 KiB a head, for products that
// take 8 cycles an instruction here and hide under the loads.)
//
// Precision: fp32 operands go in as bf16 high and low parts, x = hi + lo + e
// with |e| <= 2^-18 |x| (two roundings to nearest of 2^-9 each), and the
// products hi hi + lo hi + hi lo leave out lo lo, 2^-18 of the term at most:
// below 2^-16 of the sum of the terms' magnitudes in all, far under the 2^-9 of
// the bf16 result. Rows that are bf16 as they are (the delta rule's q and k,
// and v) have no low part. Sums are fp32.
//
// Weights of nodes off a path are zeros in the products, which would turn an
// infinite or NaN value into NaN for everybody: such values are left out of
// the operand and added by hand to the nodes below them.
#pragma once

#include <cudaTypedefs.h>

#include "la_sm100.cuh"
#include "la_tree.cuh"

namespace la {
namespace treeops {

constexpr uint64_t kWaitNs = 2000000000ull;    // bound of every wait for a copy

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ float low_half(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_half(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// a and b as bf16 pairs: high parts and what they leave
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2(a, b);
  lo = pack2(a - low_half(hi), b - high_half(hi));
}

// phi from one exponential: 2^-21 of the value, well inside the 2^-18 of its
// two bf16 parts (|x| log2(e) is rounded to 2^-24 of itself, and beyond |x| = 8
// phi is below 2^-11 of the 1 that a zero gives)
__device__ __forceinline__ float phi_fast(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * 1.4426950408889634f));
  return x >= 0.f ? x + 1.f : e;
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ bool nonfinite_half(uint32_t h) { return (h & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ bool nonfinite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

// Eight consecutive values of one row as they lie in memory -> shared memory
// with each block of 16 columns' even columns before its odd ones (row g of
// the A operand is column 2g, row g + 8 column 2g + 1).
__device__ __forceinline__ void store_columns(uint8_t* row, int chunk, const uint4& x) {
  uint2 even, odd;
  even.x = __byte_perm(x.x, x.y, 0x5410);
  even.y = __byte_perm(x.z, x.w, 0x5410);
  odd.x = __byte_perm(x.x, x.y, 0x7632);
  odd.y = __byte_perm(x.z, x.w, 0x7632);
  uint8_t* p = row + (chunk >> 1) * 32 + (chunk & 1) * 8;
  *reinterpret_cast<uint2*>(p) = even;
  *reinterpret_cast<uint2*>(p + 16) = odd;
}


__device__ __forceinline__ void prefetch_l2(const void* p, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// A 16-byte piece of a q and of a k row as bf16 hi and lo of their feature
// maps (qh, ql, kh, kl); returns the piece's part of phi(q) . z.
__device__ __forceinline__ float feature_rows(const uint4& xq, const uint4& xk, const float (&zz)[8], uint4 (&o)[4]) {
  const uint32_t* pq = reinterpret_cast<const uint32_t*>(&xq);
  const uint32_t* pk = reinterpret_cast<const uint32_t*>(&xk);
  uint32_t* qh = reinterpret_cast<uint32_t*>(&o[0]);
  uint32_t* ql = reinterpret_cast<uint32_t*>(&o[1]);
  uint32_t* kh = reinterpret_cast<uint32_t*>(&o[2]);
  uint32_t* kl = reinterpret_cast<uint32_t*>(&o[3]);
  float zq = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f0 = phi_fast(low_half(pq[w])), f1 = phi_fast(high_half(pq[w]));
    zq = fmaf(f0, zz[2 * w], zq);
    zq = fmaf(f1, zz[2 * w + 1], zq);
    split2(f0, f1, qh[w], ql[w]);
    split2(phi_fast(low_half(pk[w])), phi_fast(high_half(pk[w])), kh[w], kl[w]);
  }
  return zq;
}

// Values of a piece that are not finite become zero; returns whether there
// were any.
__device__ __forceinline__ int clear_nonfinite(uint4& x) {
  uint32_t* p = reinterpret_cast<uint32_t*>(&x);
  int any = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (nonfinite_half(p[w])) { p[w] &= 0xffff0000u; any = 1; }
    if (nonfinite_half(p[w] >> 16)) { p[w] &= 0x0000ffffu; any = 1; }
  }
  return any;
}

// The states [BH][DK][DV] fp32 in boxes of 32 columns (128 bytes, swizzled) x
// `rows` rows.
template <int DK, int DV>
cudaError_t state_map(CUtensorMap* m, const float* S, int BH, int rows) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    cudaDriverEntryPointQueryResult found;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)DV, (cuuint64_t)DK, (cuuint64_t)BH};
  const cuuint64_t strides[2] = {(cuuint64_t)DV * 4, (cuuint64_t)DK * DV * 4};
  const cuuint32_t box[3] = {32, (cuuint32_t)rows, 1};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float*>(S), dims, strides, box, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace treeops
}  // namespace la
