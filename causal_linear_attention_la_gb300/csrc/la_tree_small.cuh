// Tree decode on the tensor cores for up to 16 nodes (the formulas of
// la_tree_simt.cu, the operands and precision of la_tree_ops.cuh).
//
// With few nodes the call is bound by the state's way to the products: one 64
// KiB read a head, of which the lanes' own fragment loads reach L1 in 64-byte
// pieces, two wavefronts each (47 us for 16 nodes on 2048 d = 128 states, L1
// at half of its rate, 11000 cycles a CTA). Here the whole state comes by TMA,
// in boxes of 32 columns with the 128-byte swizzle, so that a fragment's rows
// lie in different banks (row by row as bulk copies of 512 bytes: 60 cycles of
// issue each, 52 us); the boxes are under way while q, k and v are prepared. 16
// nodes on 2048 states take 30 us, 0.82 of what HBM allows.
//
// One CTA per (batch, head), two per SM at d = 128: one warp per 16 value
// columns and one more that starts the copies and works out the ancestor
// masks; an SM's two CTAs start apart. Three
// barriers:
//   rows    phi(q), phi(k) as bf16 hi and lo, v, phi(q).z
//   pairs   every warp a 16 x 16 product over its own keys (K split over the
//           warps: a chain of few products), the partial sums joined by a
//           thread per pair, which applies mask and decay and stores W as hi
//           and lo; 1 / den
//   read    D = S^T x, then D += V^T W^T, out
// The delta rule reads for the keys as well and multiplies by the inverse
// triangle before the path.
#pragma once

#include "la_tree_ops.cuh"

namespace la {
namespace treesmall {

using namespace treeops;

constexpr int TP = 16;                         // nodes
constexpr int PP = 18;                         // floats per row of a partial pair product
constexpr int WPB = 48;                        // bytes per row of W

template <int DK, int DV, bool kDelta>
struct Small {
  static constexpr int NT = 2 * DV, NW = DV / 16, KS = DK / 16;
  static constexpr int KW = NW < KS ? NW : KS;           // parts of K in the pair products
  static constexpr int BOX = DK * 128;                   // bytes of one box of the state: dk rows x 32 columns
  static constexpr int QP = 2 * DK + 16;                 // bytes per row of q, k (matrix loads without bank conflicts)
  static constexpr int VP = 2 * DV + 16;                 // bytes per row of v, u
  static constexpr int S = 0;
  static constexpr int QH = S + DK * DV * 4;
  static constexpr int QL = QH + TP * QP;
  static constexpr int KH = QL + (kDelta ? 0 : TP * QP);
  static constexpr int KL = KH + TP * QP;
  static constexpr int V = KL + (kDelta ? 0 : TP * QP);
  static constexpr int PART = V + (kDelta ? 0 : TP * VP);
  static constexpr int PART2 = PART + KW * TP * PP * 4;  // delta: k_j . k_l
  static constexpr int A = PART2 + (kDelta ? KW * TP * PP * 4 : 0);
  static constexpr int WH = A + (kDelta ? TP * TP * 4 : 0);
  static constexpr int WL = WH + TP * WPB;
  static constexpr int LH = WL + TP * WPB;               // delta: the inverse triangle
  static constexpr int LL = LH + (kDelta ? TP * WPB : 0);
  static constexpr int MASK = LL + (kDelta ? TP * WPB : TP * 0);
  static constexpr int DEPTH = MASK + TP * 8;
  static constexpr int UP = DEPTH + TP * 4;
  static constexpr int PW = UP + TP * 4;
  static constexpr int ZQ = PW + 80;
  static constexpr int RDEN = ZQ + TP * 4;
  static constexpr int BAD = RDEN + TP * 4;
  static constexpr int BAR = BAD + 16;
  static constexpr int BYTES = BAR + 16;
  static_assert(QH % 16 == 0 && PART % 16 == 0 && A % 16 == 0 && WH % 16 == 0 && LH % 16 == 0 && MASK % 16 == 0 && BAR % 8 == 0, "alignment");
  static_assert(TP * (2 * (TP + 1) + DV) * 4 <= MASK, "room for delta_tree_by_paths");
  // two CTAs per SM (228 KiB, 1 KiB of it taken by each CTA)
  static_assert(BYTES + 1024 <= 116736, "shared memory of two CTAs");
};

template <int DK, int DV, bool kDelta>
__global__ void __launch_bounds__(2 * DV + 32, DV == 128 ? 2 : 4)
tree_small_kernel(const __grid_constant__ CUtensorMap map_s, const float* __restrict__ S, const float* __restrict__ z, const __nv_bfloat16* __restrict__ q,
                  const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                  const int* __restrict__ parent, const int* __restrict__ count, __nv_bfloat16* __restrict__ out, int H,
                  int ntok, const float* __restrict__ alpha, float eps, int* status, int stall, unsigned late0,
                  unsigned late1) {
  using L = Small<DK, DV, kDelta>;
  constexpr int NT = L::NT, NW = L::NW, KS = L::KS, KW = L::KW, BOX = L::BOX, QP = L::QP, VP = L::VP;
  extern __shared__ __align__(1024) uint8_t sm[];
  const long long bh = blockIdx.x;
  const int b = (int)(bh / H), h = (int)(bh % H), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // an SM's first CTAs start at once and then keep step, all at their loads and
  // all at their products: half of them start 1.5 us later
  if (blockIdx.x >= late0 && blockIdx.x < late1) __nanosleep(1500);
  const int n = clamp_count(count, b, ntok);
  if (n == 0) return;
  if ((sm100::smem_u32(sm) & 1023u) != 0u) {       // the swizzle goes by address bits
    if (tid == 0) atomicExch(status, (int)LA_ERR_TIMEOUT);
    return;
  }
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(sm + L::MASK);
  unsigned int* bad = reinterpret_cast<unsigned int*>(sm + L::BAD);
  int* depth = reinterpret_cast<int*>(sm + L::DEPTH);
  float* pw = reinterpret_cast<float*>(sm + L::PW);
  float* zqs = reinterpret_cast<float*>(sm + L::ZQ);
  float* rden = reinterpret_cast<float*>(sm + L::RDEN);
  float* part = reinterpret_cast<float*>(sm + L::PART);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
  const uint32_t base = sm100::smem_u32(sm);
  const __nv_bfloat16* qb = q + bh * (long long)ntok * DK;
  const __nv_bfloat16* kb = k + bh * (long long)ntok * DK;
  const __nv_bfloat16* vb = v + bh * (long long)ntok * DV;
  __nv_bfloat16* ob = out + bh * (long long)ntok * DV;
  const int tiles = (n + 7) >> 3;
  int odd_values = 0;

  if (warp == NW) {
    // ---- the state's boxes, the tree
    if (lane == 0) {
      sm100::mbar_init(bar, 1);
      sm100::fence_mbar_init();
      // (stall, for tests: 16 bytes more than come, so that the waits run out)
      sm100::mbar_arrive_expect_tx(bar, DK * DV * 4 + (stall ? 16 : 0));
      for (int x = 0; x < DV / 32; ++x) sm100::tma_load_3d(sm + L::S + x * BOX, &map_s, bar, 32 * x, 0, (int)bh);
      bad[0] = 0u;
    }
    __syncwarp();
    tree_masks(parent + (long long)b * ntok, n, TP, mask, depth, reinterpret_cast<int*>(sm + L::UP));
    if (!kDelta && alpha != nullptr && lane <= TP) pw[lane] = tree_power(alpha[h], lane);
  } else {
    // ---- rows: a thread has a 16-byte piece of q and of k, and one of v
    constexpr int CH = DK / 8, RPP = NT / CH, CHV = DV / 8;
    static_assert(NT / CHV == TP, "one pass over v");
    const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
    const int ch = tid % CH, chv = tid % CHV, iv = tid / CHV;
    constexpr int PASSES = (TP + RPP - 1) / RPP;
    uint4 xq[PASSES], xk[PASSES], xv = zero4;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int i = tid / CH + p * RPP;
      xq[p] = xk[p] = zero4;
      if (i < n) {
        xq[p] = *reinterpret_cast<const uint4*>(qb + i * DK + 8 * ch);
        xk[p] = *reinterpret_cast<const uint4*>(kb + i * DK + 8 * ch);
      }
    }
    if (!kDelta && iv < n) xv = *reinterpret_cast<const uint4*>(vb + iv * DV + 8 * chv);
    if constexpr (kDelta) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int i = tid / CH + p * RPP;
        if (i < TP) {
          *reinterpret_cast<uint4*>(sm + L::QH + i * QP + 16 * ch) = xq[p];
          *reinterpret_cast<uint4*>(sm + L::KH + i * QP + 16 * ch) = xk[p];
        }
      }
    } else {
      float zz[8];
      const float4 z0 = *reinterpret_cast<const float4*>(z + bh * DK + 8 * ch);
      const float4 z1 = *reinterpret_cast<const float4*>(z + bh * DK + 8 * ch + 4);
      zz[0] = z0.x; zz[1] = z0.y; zz[2] = z0.z; zz[3] = z0.w;
      zz[4] = z1.x; zz[5] = z1.y; zz[6] = z1.z; zz[7] = z1.w;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int i = tid / CH + p * RPP;
        uint4 o[4];
        float zq = feature_rows(xq[p], xk[p], zz, o);
        if (i < TP) {
          *reinterpret_cast<uint4*>(sm + L::QH + i * QP + 16 * ch) = o[0];
          *reinterpret_cast<uint4*>(sm + L::QL + i * QP + 16 * ch) = o[1];
          *reinterpret_cast<uint4*>(sm + L::KH + i * QP + 16 * ch) = o[2];
          *reinterpret_cast<uint4*>(sm + L::KL + i * QP + 16 * ch) = o[3];
        }
#pragma unroll
        for (int off = 1; off < CH; off <<= 1) zq += __shfl_xor_sync(0xffffffffu, zq, off);
        if (i < TP) zqs[i] = zq;                     // the same number from every lane of the row: no divergence
      }
      odd_values = clear_nonfinite(xv);
      store_columns(sm + L::V + iv * VP, chv, xv);
    }
  }
  unsigned long long spoilt = 0ull;
  if (__syncthreads_or(odd_values)) {
    for (int x = tid; x < n * DV; x += NT + 32)
      if (nonfinite(__bfloat162float(vb[x]))) atomicOr(bad, 1u << (x / DV));
    __syncthreads();
    spoilt = bad[0];
  }

  const int g = lane >> 2, t = lane & 3;
  // lane's row address of a 16 x 16 block as four 8 x 8 matrices: (rows 0-7,
  // k 0-7), (rows 8-15, k 0-7), (rows 0-7, k 8-15), (rows 8-15, k 8-15)
  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lcol = (lane >> 4) * 16;
  const uint32_t qfrag = base + L::QH + lrow * QP + lcol;
  if (warp < NW) {
    // ---- pairs over this warp's keys: the A fragment of rows i and, from the
    // same loads of the k rows, the B fragments of both halves of j
    const int k0 = warp % KW;
    const bool mine0 = NW <= KS || warp / KW == 0, mine1 = (NW <= KS || warp / KW == 1) && tiles > 1;
    float d[2][4] = {}, d2[2][4] = {};
    for (int ks = k0; ks < KS; ks += KW) {
      uint32_t qa[4], kb4[4];
      ldmatrix4(qa, qfrag + 32 * ks);
      ldmatrix4(kb4, qfrag + (L::KH - L::QH) + 32 * ks);
      if constexpr (kDelta) {
        if (mine0) mma(d[0], qa, kb4[0], kb4[2]);
        if (mine1) mma(d[1], qa, kb4[1], kb4[3]);
        if (mine0) mma(d2[0], kb4, kb4[0], kb4[2]);
        if (mine1) mma(d2[1], kb4, kb4[1], kb4[3]);
      } else {
        uint32_t ql4[4], kl4[4];
        ldmatrix4(ql4, qfrag + (L::QL - L::QH) + 32 * ks);
        ldmatrix4(kl4, qfrag + (L::KL - L::QH) + 32 * ks);
        if (mine0) {
          mma(d[0], qa, kb4[0], kb4[2]);
          mma(d2[0], qa, kl4[0], kl4[2]);
          mma(d2[0], ql4, kb4[0], kb4[2]);
        }
        if (mine1) {
          mma(d[1], qa, kb4[1], kb4[3]);
          mma(d2[1], qa, kl4[1], kl4[3]);
          mma(d2[1], ql4, kb4[1], kb4[3]);
        }
      }
    }
    float* pd = part + k0 * TP * PP;
    float* pd2 = reinterpret_cast<float*>(sm + L::PART2) + k0 * TP * PP;
#pragma unroll
    for (int nj = 0; nj < 2; ++nj)
      if (nj == 0 ? mine0 : mine1) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = (g + 8 * e) * PP + 8 * nj + 2 * t;
          if constexpr (kDelta) {
            *reinterpret_cast<float2*>(pd + at) = make_float2(d[nj][2 * e], d[nj][2 * e + 1]);
            *reinterpret_cast<float2*>(pd2 + at) = make_float2(d2[nj][2 * e], d2[nj][2 * e + 1]);
          } else {
            *reinterpret_cast<float2*>(pd + at) = make_float2(d[nj][2 * e] + d2[nj][2 * e], d[nj][2 * e + 1] + d2[nj][2 * e + 1]);
          }
        }
      }
  }
  __syncthreads();
  if (warp < NW) {
    // ---- join: a thread per pair, 16 lanes a row
    for (int x = tid; x < TP * TP; x += NT) {
      const int i = x >> 4, j = x & 15;
      const unsigned long long m = mask[i];
      const bool on = (m >> j) & 1;
      float w = 0.f;
      if (on) {
#pragma unroll
        for (int p = 0; p < KW; ++p) w += part[p * TP * PP + i * PP + j];
        if (!kDelta && alpha != nullptr) w *= pw[depth[i] - depth[j]];
      }
      uint32_t hi, lo;
      split2(w, 0.f, hi, lo);
      *reinterpret_cast<uint16_t*>(sm + L::WH + i * WPB + 2 * j) = (uint16_t)hi;
      *reinterpret_cast<uint16_t*>(sm + L::WL + i * WPB + 2 * j) = (uint16_t)lo;
      if constexpr (kDelta) {
        float a = 0.f;
        if (on && i != j) {
          const float* p2 = reinterpret_cast<const float*>(sm + L::PART2);
#pragma unroll
          for (int p = 0; p < KW; ++p) a += p2[p * TP * PP + i * PP + j];
        }
        reinterpret_cast<float*>(sm + L::A)[i * TP + j] = a;
      } else {
        float s = w;
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (j == 0) {
          float zq = zqs[i];
          if (alpha != nullptr) zq *= pw[depth[i]];
          rden[i] = 1.f / (zq + s + eps);
        }
      }
    }
  }
  if constexpr (kDelta) {
    __syncthreads();
    if (warp == NW && lane < TP)
      invert_unit_triangle(reinterpret_cast<const float*>(sm + L::A), lane, sm + L::LH, sm + L::LL, WPB);
  }

  // ---- read: D[c][i] = sum_r S[r][c] x_i[r]
  const bool here = sm100::mbar_drain(bar, 0, kWaitNs);
  const int c0 = 16 * warp + 2 * g;
  float acc[2][4] = {}, acck[2][4] = {};           // (acck: delta rule)
  uint32_t vr[2][2];                               // delta: this lane's values of v
  if (warp < NW) {
    if constexpr (kDelta) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 8 * nt + 2 * t + e;
          vr[nt][e] = j < n ? *reinterpret_cast<const uint32_t*>(vb + j * DV + c0) : 0u;
        }
    }
    // rows 2t and 2t + 1 of a step (2t + 8 and 2t + 9 likewise): the 16-byte
    // piece of column c0 lies at its index XOR the row's low three bits
    const int piece = (warp & 1) * 4 + (g >> 1);
    const uint8_t* box = sm + L::S + (warp >> 1) * BOX + (g & 1) * 8;
    const uint8_t* even = box + 2 * t * 128 + ((piece ^ (2 * t)) << 4);
    const uint8_t* odd = box + (2 * t + 1) * 128 + ((piece ^ (2 * t + 1)) << 4);
    const uint32_t xa = base + lrow * QP + lcol;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const float2 s0 = *reinterpret_cast<const float2*>(even + 2048 * ks);
      const float2 s1 = *reinterpret_cast<const float2*>(odd + 2048 * ks);
      const float2 s2 = *reinterpret_cast<const float2*>(even + 2048 * ks + 1024);
      const float2 s3 = *reinterpret_cast<const float2*>(odd + 2048 * ks + 1024);
      uint32_t ah[4], al[4], x4[4], y4[4];
      split2(s0.x, s1.x, ah[0], al[0]);
      split2(s0.y, s1.y, ah[1], al[1]);
      split2(s2.x, s3.x, ah[2], al[2]);
      split2(s2.y, s3.y, ah[3], al[3]);
      ldmatrix4(x4, xa + L::QH + 32 * ks);
      ldmatrix4(y4, xa + (kDelta ? L::KH : L::QL) + 32 * ks);
      mma(acc[0], ah, x4[0], x4[2]);
      mma(acc[0], al, x4[0], x4[2]);
      mma(kDelta ? acck[0] : acc[0], ah, y4[0], y4[2]);
      if constexpr (kDelta) mma(acck[0], al, y4[0], y4[2]);
      if (tiles > 1) {
        mma(acc[1], ah, x4[1], x4[3]);
        mma(acc[1], al, x4[1], x4[3]);
        mma(kDelta ? acck[1] : acc[1], ah, y4[1], y4[3]);
        if constexpr (kDelta) mma(acck[1], al, y4[1], y4[3]);
      }
    }
  }
  // W, 1 / den, the inverse triangle; without its state the CTA ends here and
  // stores nothing, after another wait for what may still be in flight
  if (__syncthreads_or(!here)) {
    (void)sm100::mbar_drain(bar, 0, kWaitNs);
    if (tid == 0) atomicExch(status, (int)LA_ERR_TIMEOUT);
    return;
  }

  uint32_t a[4], al[4];                            // v or u as the A operand
  if constexpr (kDelta) {
    int odd_u = 0;
    if (warp < NW) {
      const uint32_t la = base + L::LH + lrow * WPB + lcol;
      float u[2][4] = {};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          acck[nt][e] = low_half(vr[nt][e]) - acck[nt][e];
          acck[nt][2 + e] = high_half(vr[nt][e]) - acck[nt][2 + e];
        }
      as_operand(acck[0], acck[1], a, al);
      mma_block(u[0], u[1], a, al, la, la + (L::LL - L::LH));
      odd_u = any_nonfinite(u[0]) || any_nonfinite(u[1]);
      as_operand(u[0], u[1], a, al);
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
    for (int nt = 0; nt < 2; ++nt) {
      const float p0 = pw[depth[8 * nt + 2 * t]], p1 = pw[depth[8 * nt + 2 * t + 1]];
      acc[nt][0] *= p0;
      acc[nt][1] *= p1;
      acc[nt][2] *= p0;
      acc[nt][3] *= p1;
    }
  }
  // ---- path: D[c][i] += sum_j V[j][c] W[i][j]
  {
    const uint32_t wa = base + L::WH + lrow * WPB + lcol;
    if constexpr (kDelta) {
      mma_block(acc[0], acc[1], a, al, wa, wa + (L::WL - L::WH));
    } else {
      uint32_t wh[4], wl[4];
      ldmatrix4t(a, base + L::V + ((lane & 7) + (lane >> 4) * 8) * VP + 32 * warp + ((lane >> 3) & 1) * 16);
      ldmatrix4(wh, wa);
      ldmatrix4(wl, wa + (L::WL - L::WH));
      mma(acc[0], a, wh[0], wh[2]);
      mma(acc[1], a, wh[1], wh[3]);
      mma(acc[0], a, wl[0], wl[2]);
      mma(acc[1], a, wl[1], wl[3]);
    }
  }
  // ---- out
  if (!kDelta && spoilt != 0ull) {
    // the values left out of v, for the nodes below them
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int node = 8 * nt + 2 * t + e;
        for (unsigned long long m = mask[node] & spoilt; m != 0ull; m &= m - 1) {
          const int j = __ffsll((long long)m) - 1;
          const uint32_t x = *reinterpret_cast<const uint32_t*>(vb + j * DV + c0);
          const float w = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(sm + L::WH + node * WPB + 2 * j)) +
                          __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(sm + L::WL + node * WPB + 2 * j));
          if (nonfinite(low_half(x))) acc[nt][e] = fmaf(w, low_half(x), acc[nt][e]);
          if (nonfinite(high_half(x))) acc[nt][2 + e] = fmaf(w, high_half(x), acc[nt][2 + e]);
        }
      }
  }
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int node = 8 * nt + 2 * t + e;
      const float r = kDelta ? 1.f : rden[node];
      if (node < n) *reinterpret_cast<uint32_t*>(ob + node * DV + c0) = pack2(acc[nt][e] * r, acc[nt][2 + e] * r);
    }
}

template <int DK, int DV, bool kDelta>
cudaError_t launch(const TreeArgs& a) {
  using L = Small<DK, DV, kDelta>;
  auto kern = tree_small_kernel<DK, DV, kDelta>;
  static KernelOnce once;
  int resident = 0;
  cudaError_t e = once.prepare(kern, L::NT + 32, L::BYTES, &resident);
  if (e != cudaSuccess) return e;
  int* status = device_status_ptr();
  if (status == nullptr) return cudaErrorNotReady;
  CUtensorMap map_s;
  e = state_map<DK, DV>(&map_s, a.S, a.BH, DK);
  if (e != cudaSuccess) return e;
  // Worth its wait with several CTAs to come for each place, none for a call that
  // is over after a few. Without and with it, 16 nodes on 2048, 4096 and 8192
  // states, us: d = 128 32.4 31.2, 58.3 56.9, 109.5 108.1 (4 nodes on 2048 29.1
  // 27.9); dk = 128, dv = 64 22.2 21.8, 39.7 39.1, 73.7 73.3; dk = 64, dv = 128
  // 21.3 21.0, 37.9 37.7, 71.0 70.7; d = 64, four CTAs an SM, 12.8 12.8, 22.6
  // 22.3, 40.7 40.5 (4 nodes 10.8 10.8, 19.6 19.7, 35.4 35.5). By the delta rule
  // up to 5 % less time, level at d = 64.
  const unsigned late1 = a.BH >= 4LL * resident ? (unsigned)resident : 0u, late0 = late1 / 2;
  kern<<<a.BH, L::NT + 32, L::BYTES, a.stream>>>(map_s, a.S, a.z, (const __nv_bfloat16*)a.q, (const __nv_bfloat16*)a.k,
                                                 (const __nv_bfloat16*)a.v, a.parent, a.count, (__nv_bfloat16*)a.out,
                                                 a.H, a.T, a.alpha, a.eps, status, take_tree_timeout_test() ? 1 : 0,
                                                 late0, late1);
  e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace treesmall
}  // namespace la
