// Tree decode on the tensor cores (bf16 rows, dk and dv in {64, 128}; the
// formulas are those of la_tree_simt.cu).
//
// What bounds it: the state is read once (64 KiB at d = 128, against 1 KiB a
// node of rows), so few nodes are bound by HBM, and 64 nodes by the products
// if they run on the CUDA cores (16 nodes on 2048 d = 128 states there: 159
// us). The products are small and their largest operand, the state, is fp32 in
// memory: a lane loads the state's values that are its own share of the
// transposed 16 x 16 A operand of mma.m16n8k16 straight from global memory
// into registers and splits them there, so that the state never passes through
// shared or tensor memory, and the nodes are the N of the product, which goes
// in steps of 8:
//   D[c][i] = sum_r S[r][c] x_i[r]         M = values c, N = nodes i, K = keys r
// Any order of r serves as long as both operands agree; the one taken gives a
// lane four consecutive keys of its two consecutive values (a warp's load
// touches whole 64-byte pieces of four state rows) and makes a B fragment one
// 8-byte load.
//
// Precision: fp32 operands go in as bf16 high and low parts, x = hi + lo + e
// with |e| <= 2^-18 |x| (two roundings to nearest of 2^-9 each), and the
// products hi hi + lo hi + hi lo leave out lo lo, 2^-18 of the term at most:
// below 2^-16 of the sum of the terms' magnitudes in all, far under the 2^-9 of
// the bf16 result. Rows that are bf16 as they are (the delta rule's q and k,
// and v) have no low part. Sums are fp32.
//
// One CTA per (batch, head), one warp per 16 value columns:
//   rows      q and k (the feature map applied) as hi and lo, v, into shared
//             memory; the tree's ancestor masks
//   pairs     W[i][j] = x_i . k_j under the mask (with the decay's weight), 16 x
//             8 tiles dealt to the warps, stored as hi and lo
//   read      D = S^T x_i for all nodes, the state's registers used once
//   path      D += V^T W^T, in steps of 16 nodes j <= i
//   delta     the read runs for the keys first; R = v - S^T k is solved for u
//             column by column in blocks of 8 nodes, and u (hi and lo) takes
//             the place of v
// Weights of nodes off the path are zeros in these products, which would turn
// an infinite or NaN value into NaN for everybody: such values are left out
// of the operand and added by hand to the nodes below them (`bad`).
#pragma once

#include "la_tree.cuh"

namespace la {
namespace treemma {

template <int DK, int DV, int NTM, bool kDelta>
struct Shape {
  static constexpr int NT = 2 * DV;            // threads: a warp per 16 columns
  static constexpr int NW = DV / 16;
  static constexpr int KS = DK / 16;           // K steps of the read
  static constexpr int TM = 8 * NTM;           // most nodes
  static constexpr int QP = 2 * DK + 32;       // bytes per row of q, k: 8-byte fragment loads without bank conflicts
  static constexpr int VP = 2 * DV + 16;       // bytes per row of v (or u) for transposed matrix loads
  static constexpr int WP = NTM == 2 ? 48 : 144;   // bytes per row of W
  static constexpr int RP = DV + 8;            // floats per row of R
  static constexpr int AP = TM + 4;            // floats per row of the key products
};

// Byte offsets in shared memory for up to `TP` nodes (a multiple of 16).
template <int DK, int DV, int NTM, bool kDelta>
struct Layout {
  int qh, ql, kh, kl, v, vl, wh, wl, r, a, mask, depth, up, pw, zq, den, bad, total;
  __host__ __device__ constexpr explicit Layout(int TP)
      : qh(0), ql(0), kh(0), kl(0), v(0), vl(0), wh(0), wl(0), r(0), a(0), mask(0), depth(0), up(0), pw(0), zq(0), den(0), bad(0),
        total(0) {
    using Sh = Shape<DK, DV, NTM, kDelta>;
    int at = 0;
    qh = at;
    at += TP * Sh::QP;
    kh = at;
    at += TP * Sh::QP;
    if (kDelta) {
      // u replaces q and k, which are done with when it is written
      v = 0;
      vl = TP * Sh::VP;
      if (at < 2 * TP * Sh::VP) at = 2 * TP * Sh::VP;
      r = at;
      at += TP * Sh::RP * 4;
      a = at;
      at += TP * Sh::AP * 4;
    } else {
      ql = at;
      at += TP * Sh::QP;
      kl = at;
      at += TP * Sh::QP;
      v = at;
      at += TP * Sh::VP;
    }
    wh = at;
    at += TP * Sh::WP;
    wl = at;
    at += TP * Sh::WP;
    mask = at;
    at += TP * 8;
    bad = at;
    at += 16;
    depth = at;
    at += TP * 4;
    up = at;
    at += TP * 4;
    pw = at;
    at += (kTreeMax + 4) * 4;
    zq = at;
    at += TP * 4;
    den = at;
    at += NTM * TP * 4;
    total = at;
  }
};

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

template <int DK, int DV, int NTM, bool kDelta>
__global__ void __launch_bounds__(2 * DV, 512 / (2 * DV))
tree_mma_kernel(const float* __restrict__ S, const float* __restrict__ z, const __nv_bfloat16* __restrict__ q,
                const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                const int* __restrict__ parent, const int* __restrict__ count, __nv_bfloat16* __restrict__ out, int H,
                int ntok, const float* __restrict__ alpha, float eps, int ahead) {
  using Sh = Shape<DK, DV, NTM, kDelta>;
  constexpr int NT = Sh::NT, NW = Sh::NW, KS = Sh::KS, QP = Sh::QP, VP = Sh::VP, WP = Sh::WP, RP = Sh::RP, AP = Sh::AP;
  extern __shared__ __align__(16) uint8_t sm[];
  const long long bh = blockIdx.x;
  const int b = (int)(bh / H), h = (int)(bh % H), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = clamp_count(count, b, ntok);
  if (n == 0) return;
  const Layout<DK, DV, NTM, kDelta> L((ntok + 15) & ~15);
  const int TP = (n + 15) & ~15, tiles = (n + 7) >> 3;
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(sm + L.mask);
  unsigned int* bad = reinterpret_cast<unsigned int*>(sm + L.bad);
  int* depth = reinterpret_cast<int*>(sm + L.depth);
  float* pw = reinterpret_cast<float*>(sm + L.pw);
  float* zqs = reinterpret_cast<float*>(sm + L.zq);      // phi(q_i) . z
  float* den = reinterpret_cast<float*>(sm + L.den);     // [tile of j][i]: sums of W over a tile
  float* R = reinterpret_cast<float*>(sm + L.r);
  float* A = reinterpret_cast<float*>(sm + L.a);

  const __nv_bfloat16* qb = q + bh * (long long)ntok * DK;
  const __nv_bfloat16* kb = k + bh * (long long)ntok * DK;
  const __nv_bfloat16* vb = v + bh * (long long)ntok * DV;
  __nv_bfloat16* ob = out + bh * (long long)ntok * DV;
  const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);

  // ---- the first rows and the whole state, all loads in flight
  constexpr int CH = DK / 8, RPP = NT / CH;        // 16-byte pieces per row of q and k, rows per pass
  constexpr int CHV = DV / 8, RPV = NT / CHV;
  const int ch = tid % CH, chv = tid % CHV;
  int i = tid / CH, iv = tid / CHV;
  uint4 xq = zero4, xk = zero4, xv = zero4;
  if (i < n) {
    xq = *reinterpret_cast<const uint4*>(qb + i * DK + 8 * ch);
    xk = *reinterpret_cast<const uint4*>(kb + i * DK + 8 * ch);
  }
  if (!kDelta && iv < n) xv = *reinterpret_cast<const uint4*>(vb + iv * DV + 8 * chv);
  float zz[8];
  if (!kDelta) {
    const float4 z0 = *reinterpret_cast<const float4*>(z + bh * DK + 8 * ch);
    const float4 z1 = *reinterpret_cast<const float4*>(z + bh * DK + 8 * ch + 4);
    zz[0] = z0.x; zz[1] = z0.y; zz[2] = z0.z; zz[3] = z0.w;
    zz[4] = z1.x; zz[5] = z1.y; zz[6] = z1.z; zz[7] = z1.w;
  }
  const int g = lane >> 2, t = lane & 3;
  const int c0 = 16 * warp + 2 * g;                // this lane's columns: c0, c0 + 1
  float2 s[KS][4];
  {
    const float* Sb = S + bh * (long long)(DK * DV) + (4 * t) * DV + c0;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[ks][e] = *reinterpret_cast<const float2*>(Sb + (16 * ks + e) * DV);
  }
  // the state and rows of the CTA that follows in this one's place, into L2
  if (tid == NT - 1 && bh + ahead < gridDim.x) {
    prefetch_l2(S + (bh + ahead) * (long long)(DK * DV), DK * DV * 4);
    prefetch_l2(q + (bh + ahead) * (long long)ntok * DK, ntok * DK * 2);
    prefetch_l2(k + (bh + ahead) * (long long)ntok * DK, ntok * DK * 2);
    prefetch_l2(v + (bh + ahead) * (long long)ntok * DV, ntok * DV * 2);
  }
  if (!kDelta && alpha != nullptr) {
    const float a = alpha[h];
    for (int d = tid; d <= kTreeMax; d += NT) pw[d] = tree_power(a, d);
  }

  // ---- rows
  for (;;) {
    if (kDelta) {
      if (i < TP) {
        *reinterpret_cast<uint4*>(sm + L.qh + i * QP + 16 * ch) = xq;
        *reinterpret_cast<uint4*>(sm + L.kh + i * QP + 16 * ch) = xk;
      }
    } else {
      uint4 qh, ql, kh, kl;
      const uint32_t* pq = reinterpret_cast<const uint32_t*>(&xq);
      const uint32_t* pk = reinterpret_cast<const uint32_t*>(&xk);
      uint32_t* pqh = reinterpret_cast<uint32_t*>(&qh);
      uint32_t* pql = reinterpret_cast<uint32_t*>(&ql);
      uint32_t* pkh = reinterpret_cast<uint32_t*>(&kh);
      uint32_t* pkl = reinterpret_cast<uint32_t*>(&kl);
      float zq = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f0 = phi_fast(low_half(pq[w])), f1 = phi_fast(high_half(pq[w]));
        zq = fmaf(f0, zz[2 * w], zq);
        zq = fmaf(f1, zz[2 * w + 1], zq);
        split2(f0, f1, pqh[w], pql[w]);
        split2(phi_fast(low_half(pk[w])), phi_fast(high_half(pk[w])), pkh[w], pkl[w]);
      }
      if (i < TP) {
        *reinterpret_cast<uint4*>(sm + L.qh + i * QP + 16 * ch) = qh;
        *reinterpret_cast<uint4*>(sm + L.ql + i * QP + 16 * ch) = ql;
        *reinterpret_cast<uint4*>(sm + L.kh + i * QP + 16 * ch) = kh;
        *reinterpret_cast<uint4*>(sm + L.kl + i * QP + 16 * ch) = kl;
      }
      // phi(q_i) . z over the CH lanes of the row
#pragma unroll
      for (int o = 1; o < CH; o <<= 1) zq += __shfl_xor_sync(0xffffffffu, zq, o);
      if (ch == 0 && i < TP) zqs[i] = zq;
    }
    i += RPP;
    if (i >= TP) break;
    xq = xk = zero4;
    if (i < n) {
      xq = *reinterpret_cast<const uint4*>(qb + i * DK + 8 * ch);
      xk = *reinterpret_cast<const uint4*>(kb + i * DK + 8 * ch);
    }
  }
  int odd_values = 0;
  if (!kDelta) {
    for (;;) {
      if (iv < TP) {
        uint32_t* p = reinterpret_cast<uint32_t*>(&xv);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if (nonfinite_half(p[w])) { p[w] &= 0xffff0000u; odd_values = 1; }
          if (nonfinite_half(p[w] >> 16)) { p[w] &= 0x0000ffffu; odd_values = 1; }
        }
        store_columns(sm + L.v + iv * VP, chv, xv);
      }
      iv += RPV;
      if (iv >= TP) break;
      xv = iv < n ? *reinterpret_cast<const uint4*>(vb + iv * DV + 8 * chv) : zero4;
    }
  }
  if (warp == NW - 1)
    tree_masks(parent + (long long)b * ntok, n, TP, mask, depth, reinterpret_cast<int*>(sm + L.up));
  unsigned long long spoilt = 0ull;                // nodes with values that v's operand leaves out
  if (kDelta) {
    if (tid == 0) bad[0] = bad[1] = 0u;
    __syncthreads();
  } else if (__syncthreads_or(odd_values)) {
    if (tid == 0) bad[0] = bad[1] = 0u;
    __syncthreads();
    for (int x = tid; x < n * DV; x += NT)
      if (nonfinite(__bfloat162float(vb[x]))) atomicOr(bad + ((x / DV) >> 5), 1u << ((x / DV) & 31));
    __syncthreads();
    spoilt = (unsigned long long)bad[0] | ((unsigned long long)bad[1] << 32);
  }

  // ---- pairs: tiles of 16 nodes i x 8 nodes j, j <= i's tile
  {
    int id = 0;
    for (int mi = 0; mi < TP / 16; ++mi)
      for (int nj = 0; nj < min(2 * mi + 2, tiles); ++nj, ++id) {
        if (id % NW != warp) continue;
        const uint8_t* xa = sm + (16 * mi + g) * QP + 8 * t;
        const uint8_t* ya = sm + L.kh + (8 * nj + g) * QP + 8 * t;
        float d[4] = {}, d2[4] = {};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint2 bk = *reinterpret_cast<const uint2*>(ya + 32 * ks);
          const uint2 a0 = *reinterpret_cast<const uint2*>(xa + L.qh + 32 * ks);
          const uint2 a1 = *reinterpret_cast<const uint2*>(xa + L.qh + 8 * QP + 32 * ks);
          const uint32_t qa[4] = {a0.x, a1.x, a0.y, a1.y};
          mma(d, qa, bk.x, bk.y);
          if constexpr (kDelta) {
            const uint2 k0 = *reinterpret_cast<const uint2*>(xa + L.kh + 32 * ks);
            const uint2 k1 = *reinterpret_cast<const uint2*>(xa + L.kh + 8 * QP + 32 * ks);
            const uint32_t ka[4] = {k0.x, k1.x, k0.y, k1.y};
            mma(d2, ka, bk.x, bk.y);
          } else {
            const uint2 bl = *reinterpret_cast<const uint2*>(ya + (L.kl - L.kh) + 32 * ks);
            const uint2 l0 = *reinterpret_cast<const uint2*>(xa + L.ql + 32 * ks);
            const uint2 l1 = *reinterpret_cast<const uint2*>(xa + L.ql + 8 * QP + 32 * ks);
            const uint32_t la[4] = {l0.x, l1.x, l0.y, l1.y};
            mma(d2, qa, bl.x, bl.y);
            mma(d2, la, bk.x, bk.y);
          }
        }
        // lane: rows 16 mi + g (+ 8), columns 8 nj + 2t (+ 1)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 16 * mi + g + 8 * e, col = 8 * nj + 2 * t;
          const unsigned long long m = mask[row];
          float w0 = d[2 * e], w1 = d[2 * e + 1];
          if constexpr (kDelta) {
            const float a0 = d2[2 * e], a1 = d2[2 * e + 1];
            A[col * AP + row] = row != col && ((m >> col) & 1) ? a0 : 0.f;
            A[(col + 1) * AP + row] = row != col + 1 && ((m >> (col + 1)) & 1) ? a1 : 0.f;
          } else {
            w0 += d2[2 * e];
            w1 += d2[2 * e + 1];
            if (alpha != nullptr) {
              w0 *= pw[max(depth[row] - depth[col], 0)];
              w1 *= pw[max(depth[row] - depth[col + 1], 0)];
            }
          }
          w0 = (m >> col) & 1 ? w0 : 0.f;
          w1 = (m >> (col + 1)) & 1 ? w1 : 0.f;
          uint32_t hi, lo;
          split2(w0, w1, hi, lo);
          *reinterpret_cast<uint32_t*>(sm + L.wh + row * WP + 2 * col) = hi;
          *reinterpret_cast<uint32_t*>(sm + L.wl + row * WP + 2 * col) = lo;
          if constexpr (!kDelta) {
            float x = w0 + w1;                     // over the row's four lanes
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            if (t == 0) den[nj * TP + row] = x;
          }
        }
      }
    // the j of a last half step that no tile covers
    if (tiles & 1) {
      for (int x = tid; x < TP * 4; x += NT) {
        const int row = x >> 2, col = 8 * tiles + 2 * (x & 3);
        *reinterpret_cast<uint32_t*>(sm + L.wh + row * WP + 2 * col) = 0u;
        *reinterpret_cast<uint32_t*>(sm + L.wl + row * WP + 2 * col) = 0u;
      }
    }
  }

  // ---- read: D[c][i] = sum_r S[r][c] x_i[r]
  float acc[NTM][4];
  auto read_state = [&](int hi_off, int lo_off) {
#pragma unroll
    for (int nt = 0; nt < NTM; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
    const uint8_t* xb = sm + g * QP + 8 * t;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t ah[4], al[4];
      split2(s[ks][0].x, s[ks][1].x, ah[0], al[0]);
      split2(s[ks][0].y, s[ks][1].y, ah[1], al[1]);
      split2(s[ks][2].x, s[ks][3].x, ah[2], al[2]);
      split2(s[ks][2].y, s[ks][3].y, ah[3], al[3]);
#pragma unroll
      for (int nt = 0; nt < NTM; ++nt)
        if (nt < tiles) {
          const uint2 bh2 = *reinterpret_cast<const uint2*>(xb + hi_off + nt * 8 * QP + 32 * ks);
          mma(acc[nt], ah, bh2.x, bh2.y);
          mma(acc[nt], al, bh2.x, bh2.y);
          if constexpr (!kDelta) {
            const uint2 bl2 = *reinterpret_cast<const uint2*>(xb + lo_off + nt * 8 * QP + 32 * ks);
            mma(acc[nt], ah, bl2.x, bl2.y);
          }
        }
    }
  };

  if constexpr (kDelta) {
    read_state(L.kh, 0);
    // R = v - S^T k
#pragma unroll
    for (int nt = 0; nt < NTM; ++nt)
      if (nt < tiles) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 8 * nt + 2 * t + e;
          const uint32_t x = j < n ? *reinterpret_cast<const uint32_t*>(vb + j * DV + c0) : 0u;
          *reinterpret_cast<float2*>(R + j * RP + c0) = make_float2(low_half(x) - acc[nt][e], high_half(x) - acc[nt][2 + e]);
        }
      }
  }
  read_state(L.qh, L.ql);
  __syncthreads();

  if constexpr (kDelta) {
    // ---- u_j = R_j - sum_{l on j's path} (k_j.k_l) u_l: a thread per column,
    // blocks of 8 nodes: all earlier nodes' part first (8 sums at a time),
    // then the block's own triangle. `off`: earlier nodes whose u is not
    // finite in this column; while there is none, the zeros of A leave the
    // other paths out.
    for (int c = tid; c < DV; c += NT) {
      unsigned long long off = 0ull;
      for (int j0 = 0; j0 < TP; j0 += 8) {
        float u[8];
        if (j0 < n) {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = R[(j0 + e) * RP + c];
          for (int l = 0; l < j0; ++l) {
            const float ul = R[l * RP + c];
            const float4 a0 = *reinterpret_cast<const float4*>(A + l * AP + j0);
            const float4 a1 = *reinterpret_cast<const float4*>(A + l * AP + j0 + 4);
            const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
            if (!((off >> l) & 1)) {
#pragma unroll
              for (int e = 0; e < 8; ++e) u[e] = fmaf(-av[e], ul, u[e]);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if ((mask[j0 + e] >> l) & 1) u[e] = fmaf(-av[e], ul, u[e]);
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int l = 0; l < e; ++l) {
              const float x = fmaf(-A[(j0 + l) * AP + j0 + e], u[l], u[e]);
              u[e] = (mask[j0 + e] >> (j0 + l)) & 1 ? x : u[e];
            }
            if (j0 + e >= n) u[e] = 0.f;
            if (nonfinite(u[e])) off |= 1ull << (j0 + e);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = 0.f;
        }
        const int at = (c >> 4) * 32 + (c & 1) * 16 + ((c & 15) >> 1) * 2;   // even columns of a block first
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = j0 + e;
          R[j * RP + c] = u[e];
          const float x = nonfinite(u[e]) ? 0.f : u[e];
          const __nv_bfloat16 hi = __float2bfloat16_rn(x);
          *reinterpret_cast<__nv_bfloat16*>(sm + L.v + j * VP + at) = hi;
          *reinterpret_cast<__nv_bfloat16*>(sm + L.vl + j * VP + at) = __float2bfloat16_rn(x - __bfloat162float(hi));
        }
      }
      if (off & 0xffffffffull) atomicOr(bad, (unsigned int)off);
      if (off >> 32) atomicOr(bad + 1, (unsigned int)(off >> 32));
    }
    __syncthreads();
  } else {
    // the read's part of a node decays along its whole path
    if (alpha != nullptr) {
#pragma unroll
      for (int nt = 0; nt < NTM; ++nt)
        if (nt < tiles) {
          const float p0 = pw[depth[8 * nt + 2 * t]], p1 = pw[depth[8 * nt + 2 * t + 1]];
          acc[nt][0] *= p0;
          acc[nt][1] *= p1;
          acc[nt][2] *= p0;
          acc[nt][3] *= p1;
        }
    }
  }

  // ---- path: D[c][i] += sum_j V[j][c] W[i][j], j in steps of 16
  {
    const int mat = lane >> 3, rr = lane & 7;
    const uint32_t va = static_cast<uint32_t>(__cvta_generic_to_shared(sm + L.v)) + (rr + (mat >> 1) * 8) * VP +
                        32 * warp + (mat & 1) * 16;
    const uint8_t* wb = sm + L.wh + g * WP + 4 * t;
#pragma unroll
    for (int js = 0; js < NTM / 2; ++js)
      if (2 * js < tiles) {
        uint32_t a[4], al[4];
        ldmatrix4t(a, va + js * 16 * VP);
        if constexpr (kDelta) ldmatrix4t(al, va + (L.vl - L.v) + js * 16 * VP);
#pragma unroll
        for (int nt = 2 * js; nt < NTM; ++nt)
          if (nt < tiles) {
            const uint8_t* w = wb + nt * 8 * WP + 32 * js;
            const uint32_t h0 = *reinterpret_cast<const uint32_t*>(w), h1 = *reinterpret_cast<const uint32_t*>(w + 16);
            const uint8_t* wl = w + (L.wl - L.wh);
            const uint32_t l0 = *reinterpret_cast<const uint32_t*>(wl), l1 = *reinterpret_cast<const uint32_t*>(wl + 16);
            mma(acc[nt], a, h0, h1);
            mma(acc[nt], a, l0, l1);
            if constexpr (kDelta) mma(acc[nt], al, h0, h1);
          }
      }
  }
  // ---- out: lane holds nodes 8 nt + 2t (+ 1), columns c0, c0 + 1
  if constexpr (kDelta) spoilt = (unsigned long long)bad[0] | ((unsigned long long)bad[1] << 32);
#pragma unroll
  for (int nt = 0; nt < NTM; ++nt)
    if (nt < tiles) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int node = 8 * nt + 2 * t + e;
        if (node >= n) continue;
        float o0 = acc[nt][e], o1 = acc[nt][2 + e];
        if (spoilt != 0ull) {
          for (unsigned long long m = mask[node] & spoilt; m != 0ull; m &= m - 1) {
            const int j = __ffsll((long long)m) - 1;
            float x0, x1;
            if constexpr (kDelta) {
              x0 = R[j * RP + c0];
              x1 = R[j * RP + c0 + 1];
            } else {
              const uint32_t x = *reinterpret_cast<const uint32_t*>(vb + j * DV + c0);
              x0 = low_half(x);
              x1 = high_half(x);
            }
            const float w = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(sm + L.wh + node * WP + 2 * j)) +
                            __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(sm + L.wl + node * WP + 2 * j));
            if (nonfinite(x0)) o0 = fmaf(w, x0, o0);
            if (nonfinite(x1)) o1 = fmaf(w, x1, o1);
          }
        }
        if constexpr (!kDelta) {
          // den_i = a^d_i phi(q_i).z + sum_j W[i][j] + eps
          float x = zqs[node];
          if (alpha != nullptr) x *= pw[depth[node]];
#pragma unroll
          for (int nj = 0; nj <= nt; ++nj) x += den[nj * TP + node];
          const float r = 1.f / (x + eps);
          o0 *= r;
          o1 *= r;
        }
        *reinterpret_cast<uint32_t*>(ob + (long long)node * DV + c0) = pack2(o0, o1);
      }
    }
}

template <int DK, int DV, int NTM, bool kDelta>
cudaError_t launch(const TreeArgs& a) {
  const Layout<DK, DV, NTM, kDelta> L((a.T + 15) & ~15);
  constexpr Layout<DK, DV, NTM, kDelta> most(8 * NTM);
  static_assert(most.total <= 232448, "shared memory budget");
  auto kern = tree_mma_kernel<DK, DV, NTM, kDelta>;
  static SharedMemoryOnce once;
  cudaError_t e = once.allow(kern, most.total);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0, resident = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kern, 2 * DV, L.total);
  if (e != cudaSuccess) return e;
  kern<<<a.BH, 2 * DV, L.total, a.stream>>>(a.S, a.z, (const __nv_bfloat16*)a.q, (const __nv_bfloat16*)a.k,
                                            (const __nv_bfloat16*)a.v, a.parent, a.count, (__nv_bfloat16*)a.out, a.H, a.T,
                                            a.alpha, a.eps, sms * resident);
  e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

template <int DK, int DV>
cudaError_t dispatch(const TreeArgs& a) {
  if (a.z == nullptr) return a.T <= 16 ? launch<DK, DV, 2, true>(a) : launch<DK, DV, 8, true>(a);
  return a.T <= 16 ? launch<DK, DV, 2, false>(a) : launch<DK, DV, 8, false>(a);
}

}  // namespace treemma
}  // namespace la
