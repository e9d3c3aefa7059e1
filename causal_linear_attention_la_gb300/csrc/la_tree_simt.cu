// Tree decode on the CUDA cores: every node of a drafted tree reads the state
// of its own path; the committed state is not written.
//
// With anc(i) the nodes from a child of the root down to i, d_i = |anc(i)| and
// a the head's decay (1 without), node i's state is the recurrence run along
// its path, S_i = a S_parent + phi(k_i) v_i^T, so that
//   num_i = a^d_i S^T phi(q_i) + sum_{j in anc(i)} a^(d_i - d_j) (phi(q_i).phi(k_j)) v_j
//   den_i = a^d_i z.phi(q_i)   + sum_{j in anc(i)} a^(d_i - d_j) phi(q_i).phi(k_j) + eps
// ("Linear Attention: KV를 고정 크기 상태에 누적하기", section "상태 갱신과 읽기를
// 식으로 정리하기", the masked sums of "상태공간모델·선형 어텐션", section 2, with
// the ancestor mask in place of the causal one). The delta rule's increments
// along a path solve the same triangular system as along a sequence,
//   u_j = v_j - S^T k_j - sum_{l in anc(j), l != j} (k_j.k_l) u_l,
//   out_i = S^T q_i + sum_{j in anc(i)} (q_i.k_j) u_j,
// whose matrix is lower triangular because a parent comes before its children.
//
// One CTA per (batch, head). The state is read once, straight into registers: a
// warp holds whole columns (each lane E rows of four), so that the nodes pass by
// it without a barrier, G at a time, and their sums over the rows meet in the
// warp, halving what a lane holds at each exchange. The pair products and the
// sums over the path are register tiles from shared memory. Everything is fp32;
// small trees are bound by the chain of these steps, large ones by the read's
// shared-memory loads and exchanges (d = 128: 20 cycles a warp and node against
// 16 for its arithmetic) with the few warps that the registers leave.
// 1536 fp32 states: 64 nodes at d = 128 197 us, with the delta rule 381 (350 and
// 668 with the read's sums met in shared memory, v beside q and k throughout and
// one thread per column in the delta rule's solve); at d = 64 95 and 163 (152
// and 348).
#include "la_tree.cuh"

namespace la {

namespace {

template <int DK, int DV>
struct TreeShape {
  static constexpr int CG = DV / 4;                              // float4 column groups
  // threads: 128 for the small heads, whose phases are short, 256 from there on
  // (measured before the read took its present form: 2048 states of 32 nodes at
  // d = 32 57 us with 256, 45 with 128; of 16 at d = 64 in fp32 49 and 53)
  static constexpr int NT = (CG * DK) < 128 ? (CG * DK) : DK * DV <= 1024 ? 128 : 256;
  static constexpr int RO = NT / CG;                             // node groups of the output
  static constexpr int QP = DK + 4;                              // pitch of q and k rows (bank-conflict free)
  // the read: a lane holds E rows of a column group, RL lanes of a warp all of
  // its rows; RW warps hold the state, the SPLIT copies of it share the nodes
  static constexpr int E = DK * DV <= 256 ? 2 : DK * DV <= 4096 ? 4 : DK * DV / 1024;
  static constexpr int RL = DK / E, CW = 32 / RL;
  static constexpr int RW = CG / CW, SPLIT = NT / 32 / RW;
  static constexpr int G = RL > 16 ? 8 : 4;                      // nodes at a time
  // CTAs per SM that the registers are cut for: two where a thread holds 64 of
  // them for the state; four of 256 threads (1536 fp32 states at d = 64 with four
  // and three: 16 nodes 32 and 39 us, 24 45 and 52); six of 128 (d = 32, bf16, with
  // eight and six: 16 nodes 20 and 18, 64 with the delta rule 102 and 93)
  static constexpr int CTAS = E >= 16 ? 2 : NT == 128 ? 6 : 1024 / NT;
  static_assert(RL <= 32 && CW >= 1 && RW * CW == CG && SPLIT >= 1 && SPLIT * RW * 32 == NT, "read layout");
};

// Shared-memory layout in floats for T nodes. The read's result takes the place
// of the k rows, which are done with by then, where its rows fit. The delta
// rule's key products, strictly below the diagonal, are the other triangle of
// the weights (in an array of their own: 56 nodes on 1536 d = 128 states 350 us,
// now 282). late: v comes after the read, where q (and k) were.
template <int DK, int DV, bool kDelta>
struct TreeSmem {
  int TP, WP, q, k, v, w, qs, z, den, pw, depth, mask, up, total;
  __host__ __device__ constexpr TreeSmem(int T, bool late)
      : TP(0), WP(0), q(0), k(0), v(0), w(0), qs(0), z(0), den(0), pw(0), depth(0), mask(0), up(0), total(0) {
    using Sh = TreeShape<DK, DV>;
    TP = (T + 3) & ~3;
    WP = TP + 4;
    q = 0;
    k = q + TP * Sh::QP;
    w = k + TP * Sh::QP;
    v = late ? q : w;
    w += late ? 0 : TP * DV;
    z = w + TP * WP;
    qs = DV <= Sh::QP ? k : z + DK;
    den = z + DK + (DV <= Sh::QP ? 0 : TP * DV);
    pw = den + TP;
    depth = pw + kTreeMax + 4;
    up = depth + TP;
    mask = up + TP;                 // 8-byte entries
    mask = (mask + 1) & ~1;
    total = mask + 2 * TP;
  }
  // v late where only that lets two CTAs share an SM (228 KiB, 1 KiB of it taken
  // by each CTA): 1536 states of 64 nodes at d = 128 269 us without, 197 with
  static constexpr int kHalf = 116736 - 1024;
  __host__ __device__ static constexpr bool late(int T) {
    return !kDelta && DV <= 2 * TreeShape<DK, DV>::QP && TreeSmem(T, false).total * 4 > kHalf;
  }
  static constexpr int bytes(int T) { return TreeSmem(T, late(T)).total * 4; }
  static constexpr int most() {
    int m = 0;
    for (int t = 1; t <= kTreeMax; ++t) m = bytes(t) > m ? bytes(t) : m;
    return m;
  }
};

template <typename T>
__device__ __forceinline__ void store4(T* p, float4 x);
template <>
__device__ __forceinline__ void store4<float>(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, float4 x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&a);
  u.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}

// Two fp32 values in one register pair, and the two-wide FMA: half the
// instructions of the read (16 nodes at d = 128: 81 us without, 75; in the pair
// products the registers that it takes cost more than it saves).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float sum2(uint64_t x) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
  return lo + hi;
}
__device__ __forceinline__ void fma2(uint64_t& c, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}

__device__ __forceinline__ void sub_from(float* p, float x) { *p -= x; }
__device__ __forceinline__ void sub_from(float* p, float4 x) {
  float4 y = *reinterpret_cast<const float4*>(p);
  y.x -= x.x; y.y -= x.y; y.z -= x.z; y.w -= x.w;
  *reinterpret_cast<float4*>(p) = y;
}

// x_i . y_j of M matrices x against one y, for j <= i < TP (rows of pitch QP),
// R x R pairs per thread; `f(m, i, j, dot)` stores them. With 256 threads one
// tile covers the tree and its blocks above the diagonal are left out.
template <int R, int M, int DK, int NT, int QP, typename F>
__device__ __forceinline__ void pair_tiles(const float* const (&x)[M], const float* y, int TP, F f) {
  constexpr int NJ = 16, NI = NT / NJ;
  const int tj = threadIdx.x % NJ, ti = threadIdx.x / NJ;
  for (int ib = 0; ib < TP; ib += R * NI)
    for (int jb = 0; jb < TP && jb < ib + R * NI; jb += R * NJ) {
      float acc[M][R][R] = {};
      int xr[R], yr[R];
#pragma unroll
      for (int a = 0; a < R; ++a) {
        xr[a] = min(ib + ti + NI * a, TP - 1) * QP;
        yr[a] = min(jb + tj + NJ * a, TP - 1) * QP;
      }
#pragma unroll(M == 1 ? 4 : 2)
      for (int r = 0; r < DK; r += 4) {
        float4 yv[R];
#pragma unroll
        for (int b = 0; b < R; ++b) yv[b] = *reinterpret_cast<const float4*>(y + yr[b] + r);
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int a = 0; a < R; ++a) {
            const float4 xv = *reinterpret_cast<const float4*>(x[m] + xr[a] + r);
#pragma unroll
            for (int b = 0; b < R; ++b) {
              if (NI == NJ && b > a) continue;
              acc[m][a][b] = fmaf(xv.x, yv[b].x, acc[m][a][b]);
              acc[m][a][b] = fmaf(xv.y, yv[b].y, acc[m][a][b]);
              acc[m][a][b] = fmaf(xv.z, yv[b].z, acc[m][a][b]);
              acc[m][a][b] = fmaf(xv.w, yv[b].w, acc[m][a][b]);
            }
          }
      }
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int a = 0; a < R; ++a)
#pragma unroll
          for (int b = 0; b < R; ++b) {
            const int i = ib + ti + NI * a, j = jb + tj + NJ * b;
            if (i < TP && j <= i) f(m, i, j, acc[m][a][b]);
          }
    }
}

// Tiles that fit the tree: with few nodes a large tile is mostly its clamped
// edge (13 nodes of 64 keys in 4 x 4 tiles: a third of the call).
template <int M, int DK, int NT, int QP, typename F>
__device__ __forceinline__ void pair_products(const float* const (&x)[M], const float* y, int TP, F f) {
  if (TP <= 16)
    pair_tiles<1, M, DK, NT, QP>(x, y, TP, f);
  else if (TP <= 32)
    pair_tiles<2, M, DK, NT, QP>(x, y, TP, f);
  else
    pair_tiles<4, M, DK, NT, QP>(x, y, TP, f);
}

template <int DK, int DV, typename T, bool kDelta>
__global__ void __launch_bounds__(TreeShape<DK, DV>::NT, TreeShape<DK, DV>::CTAS)
tree_simt_kernel(const float* __restrict__ S, const float* __restrict__ z, const T* __restrict__ q,
                 const T* __restrict__ k, const T* __restrict__ v, const int* __restrict__ parent,
                 const int* __restrict__ count, T* __restrict__ out, int H, int ntok,
                 const float* __restrict__ alpha, float eps) {
  using Sh = TreeShape<DK, DV>;
  constexpr int NT = Sh::NT, CG = Sh::CG, E = Sh::E, QP = Sh::QP;
  extern __shared__ __align__(16) float sm[];
  const long long bh = blockIdx.x;
  const int b = (int)(bh / H), h = (int)(bh % H), tid = threadIdx.x;
  const int n = clamp_count(count, b, ntok);
  if (n == 0) return;
  using Smem = TreeSmem<DK, DV, kDelta>;
  const bool late = Smem::late(kTreeMax) && Smem::late(ntok);      // (the first is known when compiled)
  const Smem L(n, late);
  const int TP = L.TP, WP = L.WP;
  float* fq = sm + L.q;
  float* fk = sm + L.k;
  float* vs = sm + L.v;
  float* wt = sm + L.w;
  float* qs = sm + L.qs;
  float* pw = sm + L.pw;
  int* depth = reinterpret_cast<int*>(sm + L.depth);
  int* up = reinterpret_cast<int*>(sm + L.up);
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(sm + L.mask);

  // the state: column group cg, rows VE * (rl + RL * i) .. + VE - 1
  constexpr int VE = E < 4 ? E : 4, EC = E / VE;
  const int warp = tid >> 5, lane = tid & 31;
  const int rl = lane / Sh::CW, cgr = (warp % Sh::RW) * Sh::CW + lane % Sh::CW;
  const float4* Sb = reinterpret_cast<const float4*>(S + bh * (long long)DK * DV);
  uint64_t s[E / 2][4];            // rows 2p and 2p + 1 of the lane's, four columns
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float4* at = Sb + (VE * (rl + Sh::RL * (e / VE)) + e % VE) * CG + cgr;
    const float4 x = at[0], y = at[CG];
    s[e / 2][0] = pack2(x.x, y.x);
    s[e / 2][1] = pack2(x.y, y.y);
    s[e / 2][2] = pack2(x.z, y.z);
    s[e / 2][3] = pack2(x.w, y.w);
  }

  const T* qb = q + bh * (long long)ntok * DK;
  const T* kb = k + bh * (long long)ntok * DK;
  const T* vb = v + bh * (long long)ntok * DV;
  // rows, four values at a time, several loads of a thread in flight
  auto load_rows = [&](const T* src, int width, int pitch, float* dst, bool map) {
    // (d = 128, 64 nodes: 285 us with four, 269 with eight; small heads lose)
    constexpr int U = E >= 16 ? 8 : 4;
    const int per = width / 4, all = TP * per;
    for (int x0 = tid; x0 < all; x0 += U * NT) {
      float4 f[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = x0 + u * NT;
        f[u] = x < n * per ? load4<T>(src + 4 * x) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = x0 + u * NT;
        if (x >= all) break;
        if (map && x < n * per) f[u] = make_float4(phi(f[u].x), phi(f[u].y), phi(f[u].z), phi(f[u].w));
        *reinterpret_cast<float4*>(dst + (x / per) * pitch + 4 * (x % per)) = f[u];
      }
    }
  };
  // (the masks while the state and the rows are on their way)
  if (tid >= NT - 32) tree_masks(parent + (long long)b * ntok, n, TP, mask, depth, up);
  load_rows(qb, DK, QP, fq, !kDelta);
  load_rows(kb, DK, QP, fk, !kDelta);
  if (!late) {
    load_rows(vb, DV, DV, vs, false);
  } else {
    constexpr int kLine = 128 / sizeof(T);
    for (int x = tid * kLine; x < n * DV; x += NT * kLine) asm volatile("prefetch.global.L2 [%0];" ::"l"(vb + x));
  }
  if (!kDelta) {
    for (int r = tid; r < DK; r += NT) sm[L.z + r] = z[bh * DK + r];
    const float a = alpha != nullptr ? alpha[h] : 1.f;
    for (int i = tid; i <= kTreeMax; i += NT) pw[i] = tree_power(a, i);
  }
  __syncthreads();

  // pair products under the ancestor mask
  if constexpr (kDelta) {
    const float* x[2] = {fq, fk};
    pair_products<2, DK, NT, QP>(x, fk, TP, [&](int m, int i, int j, float d) {
      if (m == 0 || i != j) wt[m == 0 ? j * WP + i : i * WP + j] = (mask[i] >> j) & 1 ? d : 0.f;
    });
  } else {
    const float* x[1] = {fq};
    pair_products<1, DK, NT, QP>(x, fk, TP, [&](int, int i, int j, float d) {
      wt[j * WP + i] = (mask[i] >> j) & 1 ? d * pw[depth[i] - depth[j]] : 0.f;
    });
  }
  __syncthreads();

  if constexpr (!kDelta) {
    // 1 / den_i, four lanes per node
    for (int i0 = 0; i0 < n; i0 += NT / 4) {
      const int i = min(i0 + tid / 4, n - 1), part = tid % 4;
      float t = 0.f, u = 0.f;
#pragma unroll 4
      for (int r = 4 * part; r < DK; r += 16) {
        const float4 x = *reinterpret_cast<const float4*>(fq + i * QP + r), y = *reinterpret_cast<const float4*>(sm + L.z + r);
        t = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, t))));
      }
#pragma unroll 4
      for (int j = part; j <= i; j += 4) u += wt[j * WP + i];
      t = fmaf(t, pw[depth[i]], u);
      t += __shfl_xor_sync(0xffffffffu, t, 1);
      t += __shfl_xor_sync(0xffffffffu, t, 2);
      if (part == 0) sm[L.den + i] = 1.f / (t + eps);
    }
  }

  // the read: rows of x against the state, G nodes at a time
  auto read_rows = [&](const float* x, auto put) {
    constexpr int G = Sh::G, RL = Sh::RL;
    for (int i0 = (warp / Sh::RW) * G; i0 < n; i0 += Sh::SPLIT * G) {
      uint64_t a2[4 * G] = {};
#pragma unroll
      for (int ec = 0; ec < EC; ++ec)
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float* row = x + min(i0 + g, n - 1) * QP + VE * (rl + RL * ec);
          uint64_t xr[VE / 2];
          if constexpr (VE == 4) {
            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(row);
            xr[0] = f.x;
            xr[1] = f.y;
          } else {
            xr[0] = *reinterpret_cast<const uint64_t*>(row);
          }
#pragma unroll
          for (int r = 0; r < VE / 2; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) fma2(a2[4 * g + c], xr[r], s[ec * (VE / 2) + r][c]);
        }
      float a[4 * G];
#pragma unroll
      for (int c = 0; c < 4 * G; ++c) a[c] = sum2(a2[c]);
      // the sums over the warp's lanes: each exchange keeps one half
#pragma unroll
      for (int o = 16, h = 2 * G; o >= Sh::CW; o >>= 1, h >>= 1) {
        const bool hi = (lane & o) != 0;
#pragma unroll
        for (int c = 0; c < 2 * G; ++c)
          if (c < h) {
            const float give = hi ? a[c] : a[c + h], keep = hi ? a[c + h] : a[c];
            a[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
      }
      constexpr int K = 4 * G / RL;            // values that a lane is left with
      if constexpr (K >= 4) {
#pragma unroll
        for (int c = 0; c < K; c += 4) {
          const int i = i0 + (rl * K + c) / 4;
          if (i < n) put(i * DV + 4 * cgr, make_float4(a[c], a[c + 1], a[c + 2], a[c + 3]));
        }
      } else {
        const int i = i0 + rl * K / 4;
        if (i < n)
#pragma unroll
          for (int c = 0; c < K; ++c) put(i * DV + 4 * cgr + (rl * K + c) % 4, a[c]);
      }
    }
  };
  if constexpr (kDelta) {
    read_rows(fk, [&](int at, auto t) { sub_from(vs + at, t); });                 // v - S^T k
    __syncthreads();                                                              // the k rows' place is the result's
  }
  read_rows(fq, [&](int at, auto t) { *reinterpret_cast<decltype(t)*>(qs + at) = t; });
  __syncthreads();

  if constexpr (kDelta) {
    // the increments in blocks of 8 rows: the paths before the block, a row's
    // four columns per thread, then the rows of the block, a column per thread
    // in registers (a column per thread all along took four to ten times as long)
    for (int j0 = 0; j0 < n; j0 += 8) {
      const int j = j0 + tid / CG;
      if (j0 > 0) {
        if (tid < 8 * CG && j < n) {
          float* to = vs + j * DV + 4 * (tid % CG);
          float4 u = *reinterpret_cast<const float4*>(to);
#pragma unroll 1
          for (unsigned long long m = mask[j] & ((1ull << j0) - 1); m != 0ull;) {
            constexpr int U = 4;             // rows' loads at a time
            float p[U];
            float4 x[U];
#pragma unroll
            for (int b = 0; b < U; ++b) {
              const bool on = m != 0ull;
              const int l = on ? __ffsll((long long)m) - 1 : 0;
              m &= m - 1;
              p[b] = on ? -wt[j * WP + l] : 0.f;
              x[b] = on ? *reinterpret_cast<const float4*>(vs + l * DV + 4 * (tid % CG)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int b = 0; b < U; ++b) {
              u.x = fmaf(p[b], x[b].x, u.x);
              u.y = fmaf(p[b], x[b].y, u.y);
              u.z = fmaf(p[b], x[b].z, u.z);
              u.w = fmaf(p[b], x[b].w, u.w);
            }
          }
          *reinterpret_cast<float4*>(to) = u;
        }
        __syncthreads();
      }
      if (tid < DV) {
        float u[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int i = min(j0 + r, n - 1);
          u[r] = vs[i * DV + tid];
          const unsigned on = (unsigned)(mask[i] >> j0);
          const float4 lo = *reinterpret_cast<const float4*>(wt + i * WP + j0), hi = *reinterpret_cast<const float4*>(wt + i * WP + j0 + 4);
          const float c[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int l = 0; l < r; ++l)
            if ((on >> l) & 1) u[r] = fmaf(-c[l], u[l], u[r]);
        }
#pragma unroll
        for (int r = 1; r < 8; ++r)
          if (j0 + r < n) vs[(j0 + r) * DV + tid] = u[r];
      }
      __syncthreads();
    }
  } else if (late) {
    load_rows(vb, DV, DV, vs, false);
    __syncthreads();
  }

  // out_i = (read + sum over the path) / den: 4 nodes x 4 columns per thread
  T* ob = out + bh * (long long)ntok * DV;
  const int cg = tid % CG;
  for (int i0 = 4 * (tid / CG); i0 < n; i0 += 4 * Sh::RO) {
    float4 acc[4];
    unsigned long long m[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int i = min(i0 + a, n - 1);
      m[a] = mask[i];
      acc[a] = *reinterpret_cast<const float4*>(qs + i * DV + 4 * cg);
      if (!kDelta) {
        const float p = pw[depth[i]];
        acc[a].x *= p; acc[a].y *= p; acc[a].z *= p; acc[a].w *= p;
      }
    }
    // the nodes on any of the four paths; one off a node's own path is left
    // out, not weighted by 0: its values may be infinite or NaN
    for (unsigned long long any = m[0] | m[1] | m[2] | m[3]; any != 0ull; any &= any - 1) {
      const int j = __ffsll((long long)any) - 1;
      const unsigned long long bit = any & (0ull - any);
      const float4 w4 = *reinterpret_cast<const float4*>(wt + j * WP + i0);
      const float4 x = *reinterpret_cast<const float4*>(vs + j * DV + 4 * cg);
      const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int a = 0; a < 4; ++a)
        if ((m[a] & bit) != 0ull) {
          acc[a].x = fmaf(w[a], x.x, acc[a].x);
          acc[a].y = fmaf(w[a], x.y, acc[a].y);
          acc[a].z = fmaf(w[a], x.z, acc[a].z);
          acc[a].w = fmaf(w[a], x.w, acc[a].w);
        }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (i0 + a >= n) break;
      if (!kDelta) {
        const float d = sm[L.den + i0 + a];
        acc[a].x *= d; acc[a].y *= d; acc[a].z *= d; acc[a].w *= d;
      }
      store4<T>(ob + (long long)(i0 + a) * DV + 4 * cg, acc[a]);
    }
  }
}

template <int DK, int DV, typename T, bool kDelta>
cudaError_t launch(const TreeArgs& a) {
  const int smem = TreeSmem<DK, DV, kDelta>::bytes(a.T);
  auto kern = tree_simt_kernel<DK, DV, T, kDelta>;
  static KernelOnce once;
  int resident = 0;
  constexpr int most = TreeSmem<DK, DV, kDelta>::most();
  static_assert(most <= 232448, "shared memory budget");
  cudaError_t e = once.prepare(kern, TreeShape<DK, DV>::NT, most, &resident);
  if (e != cudaSuccess) return e;
  kern<<<a.BH, TreeShape<DK, DV>::NT, smem, a.stream>>>(a.S, a.z, (const T*)a.q, (const T*)a.k, (const T*)a.v, a.parent,
                                                        a.count, (T*)a.out, a.H, a.T, a.alpha, a.eps);
  e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

template <int DK, int DV>
cudaError_t pick(const TreeArgs& a) {
  if (a.z == nullptr)
    return a.dtype == LA_BF16 ? launch<DK, DV, __nv_bfloat16, true>(a) : launch<DK, DV, float, true>(a);
  return a.dtype == LA_BF16 ? launch<DK, DV, __nv_bfloat16, false>(a) : launch<DK, DV, float, false>(a);
}

}  // namespace

cudaError_t simt_tree(const TreeArgs& a) {
#define LA_CASE(DK_, DV_) \
  case DK_ * 1000 + DV_:  \
    return pick<DK_, DV_>(a);
  switch (a.dk * 1000 + a.dv) {
    LA_CASE(16, 16) LA_CASE(16, 32) LA_CASE(16, 64) LA_CASE(16, 128)
    LA_CASE(32, 16) LA_CASE(32, 32) LA_CASE(32, 64) LA_CASE(32, 128)
    LA_CASE(64, 16) LA_CASE(64, 32) LA_CASE(64, 64) LA_CASE(64, 128)
    LA_CASE(128, 16) LA_CASE(128, 32) LA_CASE(128, 64) LA_CASE(128, 128)
    default: return cudaErrorInvalidValue;
  }
#undef LA_CASE
}

}  // namespace la
