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
// with |lo| <= 2^-8 |x| and |e| <= 2^-17 |x| (bf16 rounds by up to 2^-8, and what
// it leaves is below half a step of hi). The products hi hi + lo hi + hi lo leave
// out lo lo, up to 2^-16 of the term: with both operands' e a product is off by
// 2^-15 of itself at most. A pair weight is such a product (2^-15), split again
// before it meets v (2^-17), and the denominator sums the weights (2^-15): an
// output is off by 2^-13.8 of the sum of its terms' magnitudes at worst, 2^-17.5
// on random rows, besides its own rounding of 2^-8. A fourth product for lo lo
// would take a third more mma and leave 2^-14.6. Rows that are bf16 as they are
// (the delta rule's q and k, and v) have no low part. Sums are fp32.
//
// Weights of nodes off a path are zeros in the products, which would turn an
// infinite or NaN value into NaN for everybody: such values are left out of
// the operand and added by hand to the nodes below them, and a delta-rule tree
// with such an increment is done again on the CUDA cores, path by path.
//
// The delta rule's increments U = (I + A)^-1 R, R = V - K S, A the masked key
// products, are solved block by block of 16 nodes with the same products:
//   U_b = (I + A_bb)^-1 (R_b - sum_{b' < b} A_bb' U_b'),
// the inverses of the 16 x 16 unit triangles once per head. A warp has all
// nodes of its 16 columns, and the accumulator of a product (rows: columns of
// the state, nodes across) is laid out as the next one's A operand, so that U
// stays in registers. (A thread per column, substituting node by node, took
// 31000 of a CTA's 51000 cycles for 64 nodes.)
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

// a and b as bf16 pairs: high parts and what they leave. A high part stops at
// bf16's largest number, 2^128 - 2^120: fp32 goes on up to 2^128 - 2^104, and an
// infinite high part would leave -inf (or, for an infinite value, NaN). So the
// low part has what is beyond, infinities too, and a product with them is
// infinite and not NaN.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
  lo = pack2(a - low_half(hi), b - high_half(hi));
}

// phi from one exponential: 2^-21 of the value, well inside the 2^-17 of its
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
// were any (0 * x is NaN for those and 0 for all others: one packed product a
// pair).
__device__ __forceinline__ int clear_nonfinite(uint4& x) {
  uint32_t* p = reinterpret_cast<uint32_t*>(&x);
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
  __nv_bfloat162 probe = zero;
#pragma unroll
  for (int w = 0; w < 4; ++w) probe = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(p + w), zero, probe);
  const uint32_t bits = *reinterpret_cast<const uint32_t*>(&probe);
  if ((bits & 0x7fff7fffu) == 0u) return 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (nonfinite_half(p[w])) p[w] &= 0xffff0000u;
    if (nonfinite_half(p[w] >> 16)) p[w] &= 0x0000ffffu;
  }
  return 1;
}

// Column m of the inverse of a 16 x 16 unit lower triangle I + A (A fp32, rows
// of 16, zero on and above the diagonal), as bf16 hi and lo into column m of
// the tile at `hi` (and `lo`), rows `pitch` bytes apart.
__device__ __forceinline__ void invert_unit_triangle(const float* A, int m, uint8_t* hi, uint8_t* lo, int pitch) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float y = i == m ? 1.f : 0.f;
#pragma unroll
    for (int l0 = 0; l0 < i; l0 += 4) {
      const float4 a = *reinterpret_cast<const float4*>(A + 16 * i + l0);
      const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int l = l0; l < (l0 + 4 < i ? l0 + 4 : i); ++l) y = fmaf(-av[l - l0], x[l], y);
    }
    x[i] = y;
    const __nv_bfloat16 h = __float2bfloat16_rn(y);
    *reinterpret_cast<__nv_bfloat16*>(hi + i * pitch + 2 * m) = h;
    *reinterpret_cast<__nv_bfloat16*>(lo + i * pitch + 2 * m) = __float2bfloat16_rn(y - __bfloat162float(h));
  }
}

// The accumulators of a block of 16 nodes as the A operand of the next product.
__device__ __forceinline__ void as_operand(const float (&d0)[4], const float (&d1)[4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split2(d0[0], d0[1], hi[0], lo[0]);
  split2(d0[2], d0[3], hi[1], lo[1]);
  split2(d1[0], d1[1], hi[2], lo[2]);
  split2(d1[2], d1[3], hi[3], lo[3]);
}

// d0, d1 (nodes 0-7 and 8-15 of a block) += X Y^T: X a block's operand, Y a 16 x
// 16 tile in shared memory at this lane's matrix address `hi` (`lo`).
__device__ __forceinline__ void mma_block(float (&d0)[4], float (&d1)[4], const uint32_t (&xh)[4], const uint32_t (&xl)[4],
                                          uint32_t hi, uint32_t lo) {
  uint32_t yh[4], yl[4];
  ldmatrix4(yh, hi);
  ldmatrix4(yl, lo);
  mma(d0, xh, yh[0], yh[2]);
  mma(d1, xh, yh[1], yh[3]);
  mma(d0, xl, yh[0], yh[2]);
  mma(d1, xl, yh[1], yh[3]);
  mma(d0, xh, yl[0], yl[2]);
  mma(d1, xh, yl[1], yl[3]);
}

__device__ __forceinline__ bool any_nonfinite(const float (&d)[4]) {
  return nonfinite(d[0]) || nonfinite(d[1]) || nonfinite(d[2]) || nonfinite(d[3]);
}

// A delta-rule tree by the whole CTA on the CUDA cores, path by path: for trees
// whose increments are not all finite. `work` holds n (2 (n + 1) + DV) floats.
template <int DK, int DV>
__device__ __noinline__ void delta_tree_by_paths(const float* S, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                                 const __nv_bfloat16* v, __nv_bfloat16* out,
                                                 const unsigned long long* mask, int n, float* work) {
  float* kk = work;                            // [n][n + 1]
  float* qk = kk + n * (n + 1);
  float* u = qk + n * (n + 1);                 // [n][DV]
  __syncthreads();
  for (int x = threadIdx.x; x < n * n; x += blockDim.x) {
    const int i = x / n, j = x % n;
    float a = 0.f, b = 0.f;
    if ((mask[i] >> j) & 1)
      for (int r = 0; r < DK; ++r) {
        const float y = __bfloat162float(k[j * DK + r]);
        a = fmaf(__bfloat162float(k[i * DK + r]), y, a);
        b = fmaf(__bfloat162float(q[i * DK + r]), y, b);
      }
    kk[i * (n + 1) + j] = a;
    qk[i * (n + 1) + j] = b;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < DV; c += blockDim.x) {
    for (int j = 0; j < n; ++j) {
      float x = __bfloat162float(v[j * DV + c]), y = 0.f;
      for (int r = 0; r < DK; ++r) y = fmaf(S[r * DV + c], __bfloat162float(k[j * DK + r]), y);
      x -= y;
      for (unsigned long long m = mask[j] & ((1ull << j) - 1); m != 0ull; m &= m - 1) {
        const int l = __ffsll((long long)m) - 1;
        x = fmaf(-kk[j * (n + 1) + l], u[l * DV + c], x);
      }
      u[j * DV + c] = x;
    }
    for (int i = 0; i < n; ++i) {
      float y = 0.f;
      for (int r = 0; r < DK; ++r) y = fmaf(S[r * DV + c], __bfloat162float(q[i * DK + r]), y);
      for (unsigned long long m = mask[i]; m != 0ull; m &= m - 1) {
        const int l = __ffsll((long long)m) - 1;
        y = fmaf(qk[i * (n + 1) + l], u[l * DV + c], y);
      }
      out[(long long)i * DV + c] = __float2bfloat16_rn(y);
    }
  }
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
