// Tree decode on the tensor cores for 17 to 64 nodes (the formulas of
// la_tree_simt.cu, the operands and precision of la_tree_ops.cuh).
//
// With 64 nodes at d = 128 a head moves 128 KiB (5600 cycles of an SM's share
// of HBM) and takes 2256 mma instructions, 4500 cycles of the SM's tensor pipe:
// the two are level, and what costs is everything beside them. One CTA per
// (batch, head), two per SM: one warp per 16 value columns and one more that
// brings the state in and works out the ancestor masks.
//   rows    phi(q), phi(k) as bf16 hi and lo, v, phi(q).z; the next pass's
//           loads in flight while one is worked on
//   pairs   16 x 16 tiles of node pairs on and below the diagonal, dealt to
//           the warps; mask and decay applied, W stored as hi and lo, row sums
//           per tile
//   read    D = S^T x: the state comes by TMA in slabs of 16 or 32 rows (boxes
//           of 32 columns with the 128-byte swizzle, so that a fragment's rows
//           lie in different banks) through two buffers; a slab is used for
//           all nodes at once
//   path    D += V^T W^T in steps of 16 nodes, out
// Up to 32 nodes three CTAs share an SM and slabs have 16 rows. Up to 48 nodes
// the slabs have buffers of their own and start with the CTA; above, two CTAs
// per SM leave no room and the buffers are where phi(k) was, from the pairs on.
// 1536 decay-gated d = 128 states of up to 64 nodes: 60 us, the tensor pipe at
// 0.29, the issue slots at 0.41 - chains of dependent steps. What did not help:
// the state straight from global memory into the lanes' registers (fragments
// of 64 bytes, twice the wavefronts: 79 us), two warps per 16 columns (half as
// many instructions again: 70 us), a ring of four slabs, the whole state at
// once with two CTAs for 32 nodes (51 us for 1536 full trees, three CTAs 47),
// CTAs of an SM started apart.
//
// The delta rule reads for keys and queries in one pass over the slabs and
// solves for u in registers (la_tree_ops.cuh) after the extra warp has inverted
// the diagonal blocks.
#pragma once

#include "la_tree_ops.cuh"

namespace la {
namespace treewide {

using namespace treeops;

// TM: most nodes, 32 or 64
template <int DK, int DV, int TM, bool kDelta>
struct Wide {
  static constexpr int SLAB = TM == 32 ? 16 : 32;        // state rows per slab
  static constexpr int NT = 2 * DV, NW = DV / 16;
  static constexpr int SLABS = DK / SLAB;
  static constexpr int BUF = SLAB * DV * 4;              // bytes of a slab
  static constexpr int QP = 2 * DK + 16, VP = 2 * DV + 16;
  static constexpr int WP = 2 * TM + 16;
  int ring, qh, ql, kh, kl, v, wh, wl, ah, al, tri, mask, depth, up, pw, zq, den, rden, bad, bar, total;
  bool overlay;                                          // the ring lies where phi(k) was
  __host__ __device__ constexpr explicit Wide(int TP)
      : ring(0), qh(0), ql(0), kh(0), kl(0), v(0), wh(0), wl(0), ah(0), al(0), tri(0), mask(0), depth(0), up(0), pw(0),
        zq(0), den(0), rden(0), bad(0), bar(0), total(0), overlay(false) {
    int at = 0;
    overlay = !kDelta && TM == 64 && TP > 48 && 2 * TP * QP >= 2 * BUF;
    if (!overlay) at += 2 * BUF;
    kh = at;
    at += TP * QP;
    if (!kDelta) {
      kl = at;
      at += TP * QP;
    }
    qh = at;
    at += TP * QP;
    if (kDelta) {
      // the key products: -A below the diagonal blocks, their inverses on it
      // (bf16 hi and lo), the diagonal blocks themselves (fp32)
      ah = at;
      at += TP * WP;
      al = at;
      at += TP * WP;
      tri = at;
      at += TP * 16 * 4;
    } else {
      ql = at;
      at += TP * QP;
      v = at;
      at += TP * VP;
    }
    wh = at;
    at += TP * WP;
    wl = at;
    at += TP * WP;
    mask = at;
    at += TP * 8;
    depth = at;
    at += TP * 4;
    up = at;
    at += TP * 4;
    pw = at;
    at += (kTreeMax + 4) * 4;
    zq = at;
    at += TP * 4;
    den = at;
    at += 4 * TP * 4;
    rden = at;
    at += TP * 4;
    bad = at;
    at += 16;
    bar = at;
    at += 32;
    total = at;
  }
};

template <int DK, int DV, int TM, bool kDelta>
__global__ void __launch_bounds__(2 * DV + 32, (DV == 128 ? 2 : 3) + (TM == 32 ? 1 : 0))
tree_wide_kernel(const __grid_constant__ CUtensorMap map_s, const float* __restrict__ S, const float* __restrict__ z,
                 const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                 const __nv_bfloat16* __restrict__ v, const int* __restrict__ parent, const int* __restrict__ count,
                 __nv_bfloat16* __restrict__ out, int H, int ntok, const float* __restrict__ alpha, float eps,
                 int* status, int stall) {
  using Sh = Wide<DK, DV, TM, kDelta>;
  constexpr int NT = Sh::NT, NW = Sh::NW, SLAB = Sh::SLAB, SLABS = Sh::SLABS, BUF = Sh::BUF, QP = Sh::QP, VP = Sh::VP, WP = Sh::WP,
                KS = DK / 16, NTM = TM / 8;
  extern __shared__ __align__(1024) uint8_t sm[];
  const long long bh = blockIdx.x;
  const int b = (int)(bh / H), h = (int)(bh % H), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = clamp_count(count, b, ntok);
  if (n == 0) return;
  if ((sm100::smem_u32(sm) & 1023u) != 0u) {       // the swizzle goes by address bits
    if (tid == 0) atomicExch(status, (int)LA_ERR_TIMEOUT);
    return;
  }
  const Sh L((ntok + 15) & ~15);
  const int TP = (n + 15) & ~15, tiles = (n + 7) >> 3, blocks = TP / 16;
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(sm + L.mask);
  unsigned int* bad = reinterpret_cast<unsigned int*>(sm + L.bad);
  int* depth = reinterpret_cast<int*>(sm + L.depth);
  float* pw = reinterpret_cast<float*>(sm + L.pw);
  float* zqs = reinterpret_cast<float*>(sm + L.zq);
  float* den = reinterpret_cast<float*>(sm + L.den);     // [block of j][i]: sums of W over a tile
  float* rden = reinterpret_cast<float*>(sm + L.rden);
  float* tri = reinterpret_cast<float*>(sm + L.tri);     // [block][16][16]: A on the diagonal
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L.bar);
  uint64_t* empty = full + 2;
  volatile int* abort = reinterpret_cast<volatile int*>(bad + 2);        // a wait gave up
  const uint32_t base = sm100::smem_u32(sm);
  const __nv_bfloat16* qb = q + bh * (long long)ntok * DK;
  const __nv_bfloat16* kb = k + bh * (long long)ntok * DK;
  const __nv_bfloat16* vb = v + bh * (long long)ntok * DV;
  __nv_bfloat16* ob = out + bh * (long long)ntok * DV;
  const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
  int odd_values = 0;

  auto load_slab = [&](int s) {                    // lane 0 of the extra warp
    uint64_t* bar = full + (s & 1);
    // (stall, for tests: 16 bytes more than come, so that the waits run out)
    sm100::mbar_arrive_expect_tx(bar, BUF + (stall && s == 0 ? 16 : 0));
    for (int x = 0; x < DV / 32; ++x)
      sm100::tma_load_3d(sm + L.ring + (s & 1) * BUF + x * (SLAB * 128), &map_s, bar, 32 * x, SLAB * s, (int)bh);
  };

  if (warp == NW) {
    if (lane == 0) {
      sm100::mbar_init(full, 1);
      sm100::mbar_init(full + 1, 1);
      sm100::mbar_init(empty, NW);
      sm100::mbar_init(empty + 1, NW);
      sm100::fence_mbar_init();
      if (L.overlay) {
        prefetch_l2(S + bh * (long long)(DK * DV), DK * DV * 4);
      } else {
        load_slab(0);
        load_slab(1);
      }
      bad[0] = bad[1] = 0u;
      *abort = 0;
    }
    __syncwarp();
    tree_masks(parent + (long long)b * ntok, n, TP, mask, depth, reinterpret_cast<int*>(sm + L.up));
    if (!kDelta && alpha != nullptr)
      for (int d = lane; d <= kTreeMax; d += 32) pw[d] = tree_power(alpha[h], d);
  } else {
    // ---- rows: batches of up to four passes, all loads of a batch in flight
    constexpr int CH = DK / 8, RPP = NT / CH, CHV = DV / 8, RPV = NT / CHV;
    constexpr int PB = TM / RPP < 4 ? (TM + RPP - 1) / RPP : 4, PV = TM / RPV;
    const int ch = tid % CH, chv = tid % CHV;
    uint4 xv[PV];
    if (!kDelta) {
#pragma unroll
      for (int p = 0; p < PV; ++p) {
        const int iv = tid / CHV + p * RPV;
        xv[p] = iv < n ? *reinterpret_cast<const uint4*>(vb + iv * DV + 8 * chv) : zero4;
      }
    }
    float zz[8];
    if (!kDelta) {
      const float4 z0 = *reinterpret_cast<const float4*>(z + bh * DK + 8 * ch);
      const float4 z1 = *reinterpret_cast<const float4*>(z + bh * DK + 8 * ch + 4);
      zz[0] = z0.x; zz[1] = z0.y; zz[2] = z0.z; zz[3] = z0.w;
      zz[4] = z1.x; zz[5] = z1.y; zz[6] = z1.z; zz[7] = z1.w;
    }
#pragma unroll 1
    for (int i0 = 0; i0 < TP; i0 += PB * RPP) {
      uint4 xq[PB], xk[PB];
#pragma unroll
      for (int p = 0; p < PB; ++p) {
        const int i = i0 + p * RPP + tid / CH;
        xq[p] = xk[p] = zero4;
        if (i < n) {
          xq[p] = *reinterpret_cast<const uint4*>(qb + i * DK + 8 * ch);
          xk[p] = *reinterpret_cast<const uint4*>(kb + i * DK + 8 * ch);
        }
      }
#pragma unroll
      for (int p = 0; p < PB; ++p) {
        if (i0 + p * RPP >= TP) break;               // the same for all lanes
        const int i = i0 + p * RPP + tid / CH;
        if constexpr (kDelta) {
          if (i < TP) {
            *reinterpret_cast<uint4*>(sm + L.qh + i * QP + 16 * ch) = xq[p];
            *reinterpret_cast<uint4*>(sm + L.kh + i * QP + 16 * ch) = xk[p];
          }
        } else {
          uint4 o[4];
          float zq = feature_rows(xq[p], xk[p], zz, o);
          if (i < TP) {
            *reinterpret_cast<uint4*>(sm + L.qh + i * QP + 16 * ch) = o[0];
            *reinterpret_cast<uint4*>(sm + L.ql + i * QP + 16 * ch) = o[1];
            *reinterpret_cast<uint4*>(sm + L.kh + i * QP + 16 * ch) = o[2];
            *reinterpret_cast<uint4*>(sm + L.kl + i * QP + 16 * ch) = o[3];
          }
#pragma unroll
          for (int off = 1; off < CH; off <<= 1) zq += __shfl_xor_sync(0xffffffffu, zq, off);
          if (i < TP) zqs[i] = zq;                     // the same number from every lane of the row: no divergence
        }
      }
    }
    if constexpr (!kDelta) {
#pragma unroll
      for (int p = 0; p < PV; ++p) {
        const int iv = tid / CHV + p * RPV;
        if (iv < TP) {
          odd_values |= clear_nonfinite(xv[p]);
          store_columns(sm + L.v + iv * VP, chv, xv[p]);
        }
      }
    }
  }
  unsigned long long spoilt = 0ull;
  if (__syncthreads_or(odd_values)) {
    for (int x = tid; x < n * DV; x += NT + 32)
      if (nonfinite(__bfloat162float(vb[x]))) atomicOr(bad + ((x / DV) >> 5), 1u << ((x / DV) & 31));
    __syncthreads();
    spoilt = (unsigned long long)bad[0] | ((unsigned long long)bad[1] << 32);
  }

  const int g = lane >> 2, t = lane & 3;
  // lane's row address of a 16 x 16 block as four 8 x 8 matrices: (rows 0-7,
  // k 0-7), (rows 8-15, k 0-7), (rows 0-7, k 8-15), (rows 8-15, k 8-15)
  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lcol = (lane >> 4) * 16;
  const uint32_t frag = base + lrow * QP + lcol;
  if (warp < NW) {
    // ---- pairs: tiles of 16 nodes i x 16 nodes j, j's block <= i's
    for (int id = warp; id < blocks * (blocks + 1) / 2; id += NW) {
      int mi = 0;
      while ((mi + 1) * (mi + 2) / 2 <= id) ++mi;
      const int mj = id - mi * (mi + 1) / 2;
      const uint32_t qa0 = frag + L.qh + 16 * mi * QP, ka0 = frag + L.kh + 16 * mj * QP;
      float d[2][4] = {}, d2[2][4] = {};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t qa[4], kb4[4], x4[4], y4[4];
        ldmatrix4(qa, qa0 + 32 * ks);
        ldmatrix4(kb4, ka0 + 32 * ks);
        mma(d[0], qa, kb4[0], kb4[2]);
        mma(d[1], qa, kb4[1], kb4[3]);
        if constexpr (kDelta) {
          ldmatrix4(x4, frag + L.kh + 16 * mi * QP + 32 * ks);
          mma(d2[0], x4, kb4[0], kb4[2]);
          mma(d2[1], x4, kb4[1], kb4[3]);
        } else {
          ldmatrix4(x4, ka0 + (L.kl - L.kh) + 32 * ks);
          ldmatrix4(y4, qa0 + (L.ql - L.qh) + 32 * ks);
          mma(d2[0], qa, x4[0], x4[2]);
          mma(d2[1], qa, x4[1], x4[3]);
          mma(d2[0], y4, kb4[0], kb4[2]);
          mma(d2[1], y4, kb4[1], kb4[3]);
        }
      }
      // lane: rows 16 mi + g (+ 8), columns 16 mj + 8 nj + 2t (+ 1)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = g + 8 * e, row = 16 * mi + r, dr = depth[row];
        const uint32_t m = (uint32_t)(mask[row] >> (16 * mj)) >> (2 * t);     // bits 0, 1, 8, 9: this lane's columns
        float sum = 0.f;
#pragma unroll
        for (int nj = 0; nj < 2; ++nj) {
          const int c = 8 * nj + 2 * t, col = 16 * mj + c;
          const bool on0 = (m >> (8 * nj)) & 1, on1 = (m >> (8 * nj + 1)) & 1;
          float w0 = d[nj][2 * e], w1 = d[nj][2 * e + 1];
          uint32_t hi, lo;
          if constexpr (kDelta) {
            const float a0 = on0 && (mi != mj || r != c) ? d2[nj][2 * e] : 0.f;
            const float a1 = on1 && (mi != mj || r != c + 1) ? d2[nj][2 * e + 1] : 0.f;
            if (mi == mj) {
              *reinterpret_cast<float2*>(tri + row * 16 + c) = make_float2(a0, a1);
            } else {
              split2(-a0, -a1, hi, lo);
              *reinterpret_cast<uint32_t*>(sm + L.ah + row * WP + 2 * col) = hi;
              *reinterpret_cast<uint32_t*>(sm + L.al + row * WP + 2 * col) = lo;
            }
          } else {
            w0 += d2[nj][2 * e];
            w1 += d2[nj][2 * e + 1];
            if (alpha != nullptr) {
              w0 *= pw[max(dr - depth[col], 0)];
              w1 *= pw[max(dr - depth[col + 1], 0)];
            }
          }
          w0 = on0 ? w0 : 0.f;
          w1 = on1 ? w1 : 0.f;
          sum += w0 + w1;
          split2(w0, w1, hi, lo);
          *reinterpret_cast<uint32_t*>(sm + L.wh + row * WP + 2 * col) = hi;
          *reinterpret_cast<uint32_t*>(sm + L.wl + row * WP + 2 * col) = lo;
        }
        if constexpr (!kDelta) {
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          den[mj * TP + row] = sum;                // the same number from the row's four lanes
        }
      }
    }
  }
  // (overlay: the buffers were ordinary memory until here, the copies' next)
  if (L.overlay) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();

  // ---- read: D[c][i] = sum_r S[r][c] x_i[r], slab by slab
  float acc[NTM][4], acck[kDelta ? NTM : 1][4];
#pragma unroll
  for (int nt = 0; nt < NTM; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[nt][e] = 0.f;
      if (kDelta) acck[nt][e] = 0.f;
    }
  const int c0 = 16 * warp + 2 * g;                // this lane's columns: c0, c0 + 1
  int lost = 0;                                    // a wait gave up: nothing is stored
  if (warp == NW) {
    if (L.overlay && lane == 0) {
      load_slab(0);
      load_slab(1);
    }
    __syncwarp();
    if constexpr (kDelta)
      for (int x = lane; x < TP; x += 32) {        // 16 lanes per diagonal block
        const int at16 = (x & ~15) * WP + 2 * (x & ~15);
        invert_unit_triangle(tri + (x & ~15) * 16, x & 15, sm + L.ah + at16, sm + L.al + at16, WP);
      }
    __syncwarp();
    if (lane == 0) {
      int s = 2;
      for (; s < SLABS; ++s) {
        if (!sm100::mbar_wait(empty + (s & 1), ((s >> 1) - 1) & 1, abort, kWaitNs)) {
          lost = 1;
          break;
        }
        load_slab(s);
      }
      // nothing in flight when the CTA ends, whatever became of the others: the
      // last two slabs that were asked for (the ones before them have been read)
      for (int x = s - 2; x < s; ++x)
        if (!sm100::mbar_drain(full + (x & 1), (x >> 1) & 1, kWaitNs)) lost = 1;
    }
    __syncwarp();
    if (!kDelta)
      for (int i = lane; i < n; i += 32) {
        float x = zqs[i];
        if (alpha != nullptr) x *= pw[depth[i]];
        for (int mj = 0; mj <= i / 16; ++mj) x += den[mj * TP + i];
        rden[i] = 1.f / (x + eps);
      }
  } else {
    // rows 2t and 2t + 1 of a step (2t + 8 and 2t + 9 likewise): the 16-byte
    // piece of column c0 lies at its index XOR the row's low three bits
    const int piece = (warp & 1) * 4 + (g >> 1);
    const uint8_t* box = sm + L.ring + (warp >> 1) * (SLAB * 128) + (g & 1) * 8;
    const uint8_t* even = box + 2 * t * 128 + ((piece ^ (2 * t)) << 4);
    const uint8_t* odd = box + (2 * t + 1) * 128 + ((piece ^ (2 * t + 1)) << 4);
#pragma unroll
    for (int s = 0; s < SLABS; ++s) {
      if (!sm100::mbar_wait(full + (s & 1), (s >> 1) & 1, abort, kWaitNs)) lost = 1;
#pragma unroll
      for (int kk = 0; kk < SLAB / 16; ++kk) {
        const int at = (s & 1) * BUF + 2048 * kk;
        const float2 s0 = *reinterpret_cast<const float2*>(even + at);
        const float2 s1 = *reinterpret_cast<const float2*>(odd + at);
        const float2 s2 = *reinterpret_cast<const float2*>(even + at + 1024);
        const float2 s3 = *reinterpret_cast<const float2*>(odd + at + 1024);
        uint32_t ah[4], al[4];
        split2(s0.x, s1.x, ah[0], al[0]);
        split2(s0.y, s1.y, ah[1], al[1]);
        split2(s2.x, s3.x, ah[2], al[2]);
        split2(s2.y, s3.y, ah[3], al[3]);
        const uint32_t xa = frag + 32 * (s * (SLAB / 16) + kk);
#pragma unroll
        for (int ib = 0; ib < NTM / 2; ++ib)
          if (ib < blocks) {
            uint32_t x4[4];
            ldmatrix4(x4, xa + L.qh + 16 * ib * QP);
            mma(acc[2 * ib], ah, x4[0], x4[2]);
            mma(acc[2 * ib + 1], ah, x4[1], x4[3]);
            mma(acc[2 * ib], al, x4[0], x4[2]);
            mma(acc[2 * ib + 1], al, x4[1], x4[3]);
            if constexpr (kDelta) {
              ldmatrix4(x4, xa + L.kh + 16 * ib * QP);
              mma(acck[2 * ib], ah, x4[0], x4[2]);
              mma(acck[2 * ib + 1], ah, x4[1], x4[3]);
              mma(acck[2 * ib], al, x4[0], x4[2]);
              mma(acck[2 * ib + 1], al, x4[1], x4[3]);
            } else {
              ldmatrix4(x4, xa + L.ql + 16 * ib * QP);
              mma(acc[2 * ib], ah, x4[0], x4[2]);
              mma(acc[2 * ib + 1], ah, x4[1], x4[3]);
            }
          }
      }
      __syncwarp();
      if (lane == 0 && !lost && s + 2 < SLABS) sm100::mbar_arrive(empty + (s & 1));
    }
  }
  if constexpr (kDelta) {
    // R = v - S^T k, all of this lane's values of v in flight at once
    if (warp < NW) {
#pragma unroll
      for (int nt = 0; nt < NTM; ++nt)
        if (nt < 2 * blocks) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = 8 * nt + 2 * t + e;
            const uint32_t x = j < n ? *reinterpret_cast<const uint32_t*>(vb + j * DV + c0) : 0u;
            acck[nt][e] = low_half(x) - acck[nt][e];
            acck[nt][2 + e] = high_half(x) - acck[nt][2 + e];
          }
        }
    }
  }
  if (__syncthreads_or(lost)) {
    if (tid == 0) atomicExch(status, (int)LA_ERR_TIMEOUT);
    return;
  }

  uint32_t uh[kDelta ? NTM / 2 : 1][4], ul[kDelta ? NTM / 2 : 1][4];     // u as the A operand, block by block
  if constexpr (kDelta) {
    int odd_u = 0;
    if (warp < NW) {
      const uint32_t at = base + L.ah + lrow * WP + lcol;
#pragma unroll
      for (int ib = 0; ib < NTM / 2; ++ib)
        if (ib < blocks) {
          // R less the earlier blocks' part, through the triangle
          float (&r0)[4] = acck[2 * ib], (&r1)[4] = acck[2 * ib + 1];
          float u[2][4] = {};
#pragma unroll
          for (int jb = 0; jb < ib; ++jb)
            mma_block(r0, r1, uh[jb], ul[jb], at + 16 * ib * WP + 32 * jb, at + (L.al - L.ah) + 16 * ib * WP + 32 * jb);
          uint32_t rh[4], rl[4];
          as_operand(r0, r1, rh, rl);
          mma_block(u[0], u[1], rh, rl, at + 16 * ib * WP + 32 * ib, at + (L.al - L.ah) + 16 * ib * WP + 32 * ib);
          odd_u |= any_nonfinite(u[0]) || any_nonfinite(u[1]);
          as_operand(u[0], u[1], uh[ib], ul[ib]);
        }
    }
    if (__syncthreads_or(odd_u)) {
      delta_tree_by_paths<DK, DV>(S + bh * (long long)(DK * DV), qb, kb, vb, ob, mask, n, reinterpret_cast<float*>(sm));
      return;
    }
  }
  if (warp >= NW) return;

  if (!kDelta && alpha != nullptr) {
    // the read's part of a node decays along its whole path
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

  // ---- path: D[c][i] += sum_j V[j][c] W[i][j], j in steps of 16
  {
    const uint32_t va = base + L.v + ((lane & 7) + (lane >> 4) * 8) * VP + 32 * warp + ((lane >> 3) & 1) * 16;
    const uint32_t wa = base + L.wh + lrow * WP + lcol;
#pragma unroll
    for (int js = 0; js < NTM / 2; ++js)
      if (js < blocks) {
        uint32_t a[4];
        if constexpr (!kDelta) ldmatrix4t(a, va + js * 16 * VP);
#pragma unroll
        for (int ib = js; ib < NTM / 2; ++ib)
          if (ib < blocks) {
            const uint32_t w = wa + ib * 16 * WP + 32 * js;
            if constexpr (kDelta) {
              mma_block(acc[2 * ib], acc[2 * ib + 1], uh[js], ul[js], w, w + (L.wl - L.wh));
            } else {
              uint32_t wh[4], wl[4];
              ldmatrix4(wh, w);
              ldmatrix4(wl, w + (L.wl - L.wh));
              mma(acc[2 * ib], a, wh[0], wh[2]);
              mma(acc[2 * ib + 1], a, wh[1], wh[3]);
              mma(acc[2 * ib], a, wl[0], wl[2]);
              mma(acc[2 * ib + 1], a, wl[1], wl[3]);
            }
          }
      }
  }

  // ---- out: lane holds nodes 8 nt + 2t (+ 1), columns c0, c0 + 1
  if (!kDelta && spoilt != 0ull) {
    // the values left out of v, for the nodes below them
#pragma unroll
    for (int nt = 0; nt < NTM; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int node = 8 * nt + 2 * t + e;
        if (node >= n) continue;
        for (unsigned long long m = mask[node] & spoilt; m != 0ull; m &= m - 1) {
          const int j = __ffsll((long long)m) - 1;
          const uint32_t x = *reinterpret_cast<const uint32_t*>(vb + j * DV + c0);
          const float w = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(sm + L.wh + node * WP + 2 * j)) +
                          __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(sm + L.wl + node * WP + 2 * j));
          if (nonfinite(low_half(x))) acc[nt][e] = fmaf(w, low_half(x), acc[nt][e]);
          if (nonfinite(high_half(x))) acc[nt][2 + e] = fmaf(w, high_half(x), acc[nt][2 + e]);
        }
      }
  }
  {
    __nv_bfloat16* o = ob + (2 * t) * DV + c0;
    const float* rd = rden + 2 * t;
#pragma unroll
    for (int nt = 0; nt < NTM; ++nt)
      if (nt < tiles) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float r = kDelta ? 1.f : rd[8 * nt + e];
          const uint32_t x = pack2(acc[nt][e] * r, acc[nt][2 + e] * r);
          if (8 * nt + 2 * t + e < n) *reinterpret_cast<uint32_t*>(o + (8 * nt + e) * DV) = x;
        }
      }
  }
}

template <int DK, int DV, int TM, bool kDelta>
cudaError_t launch(const TreeArgs& a) {
  using Sh = Wide<DK, DV, TM, kDelta>;
  constexpr Sh most(TM), middle(TM == 32 ? 32 : 48);
  constexpr int bytes = most.total > middle.total ? most.total : middle.total;
  // two CTAs per SM, three for 32 nodes (228 KiB, 1 KiB of it taken by each CTA)
  static_assert(bytes + 1024 <= (TM == 32 ? 77824 : 116736), "shared memory of an SM's CTAs");
  static_assert(!kDelta || (TM * (2 * (TM + 1) + DV) * 4 <= most.mask && 32 * (2 * 33 + DV) * 4 <= Sh(32).mask &&
                            (TM == 32 || 48 * (2 * 49 + DV) * 4 <= middle.mask)),
                "room for delta_tree_by_paths");
  static_assert(Sh::SLABS >= 2, "both buffers are filled first");
  static_assert(most.ring % 1024 == 0 && Sh::BUF % 1024 == 0, "the swizzle goes by address bits");
  const Sh L((a.T + 15) & ~15);
  auto kern = tree_wide_kernel<DK, DV, TM, kDelta>;
  static KernelOnce once;
  int resident = 0;
  cudaError_t e = once.prepare(kern, Sh::NT + 32, bytes, &resident);
  if (e != cudaSuccess) return e;
  int* status = device_status_ptr();
  if (status == nullptr) return cudaErrorNotReady;
  CUtensorMap map_s;
  e = state_map<DK, DV>(&map_s, a.S, a.BH, Sh::SLAB);
  if (e != cudaSuccess) return e;
  kern<<<a.BH, Sh::NT + 32, L.total, a.stream>>>(map_s, a.S, a.z, (const __nv_bfloat16*)a.q, (const __nv_bfloat16*)a.k,
                                                 (const __nv_bfloat16*)a.v, a.parent, a.count, (__nv_bfloat16*)a.out,
                                                 a.H, a.T, a.alpha, a.eps, status, take_tree_timeout_test() ? 1 : 0);
  e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace treewide
}  // namespace la
