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
// One CTA per (batch, head). The state is read once, straight into registers
// (thread (rg, cg): E rows, four columns, all loads in flight together); the
// nodes pass by it in groups of NB, the row groups' partial sums meet by
// shuffles within a warp and then in shared memory. The pair products and the
// sums over the path are register tiles from shared memory. Everything is
// fp32; small trees are bound by the chain of these steps.
#include "la_tree.cuh"

namespace la {

namespace {

template <int DK, int DV>
struct TreeShape {
  static constexpr int CG = DV / 4;                              // float4 column groups
  // threads: 128 for the small heads, whose phases are short (2048 states of 32
  // nodes at d = 32: 57 us with 256, 45 with 128; 64 nodes 117 and 123), 256
  // from there on (2048 fp32 states of 16 nodes at d = 64: 53 us with 128, 49)
  static constexpr int NT = (CG * DK) < 128 ? (CG * DK) : DK * DV <= 1024 ? 128 : 256;
  static constexpr int RG = NT / CG;                             // row groups
  static constexpr int E = DK / RG;                              // state rows per thread
  // CTAs per SM that the registers allow: two where a thread holds 64 of them
  // for the state, else four of 256 threads (1536 states of 24 nodes at d = 64,
  // delta rule: 113 us with two, 92 with four)
  static constexpr int CTAS = E >= 16 ? 2 : 1024 / NT;
  static constexpr int NW = NT / 32;                             // warps: row groups after a warp's own have met
  static constexpr int QP = DK + 4;                              // pitch of q and k rows (bank-conflict free)
};

// Shared-memory layout in floats for T nodes of a call with rows for `most`. The
// read's result takes the place of the k rows, which are done with by then,
// where its rows fit, and the read's groups are of 8 nodes above 16: more CTAs
// per SM (1536 fp32 states at d = 64: 24 nodes 59 -> 51 us, 64 nodes 226 -> 152,
// with the delta rule 526 -> 348; at d = 128 one CTA per SM either way).
template <int DK, int DV, bool kDelta>
struct TreeSmem {
  int TP, WP, nb, q, k, v, w, w2, qs, part, z, den, pw, depth, mask, up, total;
  __host__ __device__ constexpr TreeSmem(int T, int most)
      : TP(0), WP(0), nb(0), q(0), k(0), v(0), w(0), w2(0), qs(0), part(0), z(0), den(0), pw(0), depth(0), mask(0), up(0),
        total(0) {
    using Sh = TreeShape<DK, DV>;
    TP = (T + 3) & ~3;
    nb = most <= 16 && !kDelta ? 16 : 8;               // nodes per group of the read
    WP = TP + 4;
    q = 0;
    k = q + TP * Sh::QP;
    v = k + TP * Sh::QP;
    w = v + TP * DV;
    w2 = w + TP * WP;
    part = w2 + (kDelta ? TP * WP : 0);
    qs = DV <= Sh::QP ? k : part + nb * Sh::NW * DV;
    z = part + nb * Sh::NW * DV + (DV <= Sh::QP ? 0 : TP * DV);
    den = z + DK;
    pw = den + TP;
    depth = pw + kTreeMax + 4;
    up = depth + TP;
    mask = up + TP;                 // 8-byte entries
    mask = (mask + 1) & ~1;
    total = mask + 2 * TP;
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

// w[j][i] = x_i . y_j for j <= i < TP (rows of pitch QP), R x R per thread;
// `f(i, j, dot)` gives the value that is stored.
template <int R, int DK, int NT, int QP, typename F>
__device__ __forceinline__ void pair_tiles(const float* x, const float* y, float* w, int TP, int WP, F f) {
  constexpr int NJ = 16, NI = NT / NJ;
  const int tj = threadIdx.x % NJ, ti = threadIdx.x / NJ;
  for (int ib = 0; ib < TP; ib += R * NI)
    for (int jb = 0; jb < TP && jb < ib + R * NI; jb += R * NJ) {
      float acc[R][R] = {};
      const float* xr[R];
      const float* yr[R];
#pragma unroll
      for (int a = 0; a < R; ++a) {
        xr[a] = x + min(ib + ti + NI * a, TP - 1) * QP;
        yr[a] = y + min(jb + tj + NJ * a, TP - 1) * QP;
      }
#pragma unroll 4
      for (int r = 0; r < DK; r += 4) {
        float4 xv[R], yv[R];
#pragma unroll
        for (int a = 0; a < R; ++a) {
          xv[a] = *reinterpret_cast<const float4*>(xr[a] + r);
          yv[a] = *reinterpret_cast<const float4*>(yr[a] + r);
        }
#pragma unroll
        for (int a = 0; a < R; ++a)
#pragma unroll
          for (int b = 0; b < R; ++b) {
            acc[a][b] = fmaf(xv[a].x, yv[b].x, acc[a][b]);
            acc[a][b] = fmaf(xv[a].y, yv[b].y, acc[a][b]);
            acc[a][b] = fmaf(xv[a].z, yv[b].z, acc[a][b]);
            acc[a][b] = fmaf(xv[a].w, yv[b].w, acc[a][b]);
          }
      }
#pragma unroll
      for (int a = 0; a < R; ++a)
#pragma unroll
        for (int b = 0; b < R; ++b) {
          const int i = ib + ti + NI * a, j = jb + tj + NJ * b;
          if (i < TP && j < TP) w[j * WP + i] = f(i, j, acc[a][b]);
        }
    }
}

// Tiles that fit the tree: with few nodes a large tile is mostly its clamped
// edge (13 nodes of 64 keys in 4 x 4 tiles: a third of the call).
template <int DK, int NT, int QP, typename F>
__device__ __forceinline__ void pair_products(const float* x, const float* y, float* w, int TP, int WP, F f) {
  if (TP <= 16)
    pair_tiles<1, DK, NT, QP>(x, y, w, TP, WP, f);
  else if (TP <= 32)
    pair_tiles<2, DK, NT, QP>(x, y, w, TP, WP, f);
  else
    pair_tiles<4, DK, NT, QP>(x, y, w, TP, WP, f);
}

template <int DK, int DV, typename T, bool kDelta>
__global__ void __launch_bounds__(TreeShape<DK, DV>::NT, TreeShape<DK, DV>::CTAS)
tree_simt_kernel(const float* __restrict__ S, const float* __restrict__ z, const T* __restrict__ q,
                 const T* __restrict__ k, const T* __restrict__ v, const int* __restrict__ parent,
                 const int* __restrict__ count, T* __restrict__ out, int H, int ntok,
                 const float* __restrict__ alpha, float eps) {
  using Sh = TreeShape<DK, DV>;
  constexpr int NT = Sh::NT, CG = Sh::CG, RG = Sh::RG, E = Sh::E, NW = Sh::NW, QP = Sh::QP;
  extern __shared__ __align__(16) float sm[];
  const long long bh = blockIdx.x;
  const int b = (int)(bh / H), h = (int)(bh % H), tid = threadIdx.x;
  const int n = clamp_count(count, b, ntok);
  if (n == 0) return;
  const TreeSmem<DK, DV, kDelta> L(n, ntok);
  const int TP = L.TP, WP = L.WP, NB = L.nb;
  float* fq = sm + L.q;
  float* fk = sm + L.k;
  float* vs = sm + L.v;
  float* wt = sm + L.w;
  float* qs = sm + L.qs;
  float* part = sm + L.part;
  float* pw = sm + L.pw;
  int* depth = reinterpret_cast<int*>(sm + L.depth);
  int* up = reinterpret_cast<int*>(sm + L.up);
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(sm + L.mask);

  // the state: thread (rg, cg) holds rows rg*E .. rg*E+E-1, columns 4cg .. 4cg+3
  const int cg = tid % CG, rg = tid / CG;
  const float4* Sb = reinterpret_cast<const float4*>(S + bh * (long long)DK * DV);
  float4 s[E];
#pragma unroll
  for (int e = 0; e < E; ++e) s[e] = Sb[(rg * E + e) * CG + cg];

  const T* qb = q + bh * (long long)ntok * DK;
  const T* kb = k + bh * (long long)ntok * DK;
  const T* vb = v + bh * (long long)ntok * DV;
  // rows, four values at a time, several loads of a thread in flight
  auto load_rows = [&](const T* src, int width, int pitch, float* dst, bool map) {
    constexpr int U = 4;
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
  load_rows(vb, DV, DV, vs, false);
  if (!kDelta) {
    for (int r = tid; r < DK; r += NT) sm[L.z + r] = z[bh * DK + r];
    const float a = alpha != nullptr ? alpha[h] : 1.f;
    for (int i = tid; i <= kTreeMax; i += NT) pw[i] = tree_power(a, i);
  }
  __syncthreads();

  // pair products under the ancestor mask
  if constexpr (kDelta) {
    pair_products<DK, NT, QP>(fq, fk, wt, TP, WP, [&](int i, int j, float d) { return (mask[i] >> j) & 1 ? d : 0.f; });
    pair_products<DK, NT, QP>(fk, fk, sm + L.w2, TP, WP,
                              [&](int i, int j, float d) { return i != j && ((mask[i] >> j) & 1) ? d : 0.f; });
  } else {
    pair_products<DK, NT, QP>(fq, fk, wt, TP, WP, [&](int i, int j, float d) {
      return (mask[i] >> j) & 1 ? d * pw[depth[i] - depth[j]] : 0.f;
    });
  }

  // the read: rows of x against the state, RG partial sums per node and column
  auto read_rows = [&](const float* x, auto put) {
    for (int i0 = 0; i0 < n; i0 += NB) {
      const int m = min(NB, n - i0);
      __syncthreads();       // the previous group's partial sums have been read
#pragma unroll 2
      for (int i = 0; i < m; ++i) {
        const float* row = x + (i0 + i) * QP + rg * E;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float xr[E];
        if constexpr (E % 4 == 0) {
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(row + e);
            xr[e] = f.x; xr[e + 1] = f.y; xr[e + 2] = f.z; xr[e + 3] = f.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) xr[e] = row[e];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float c = xr[e];
          acc.x = fmaf(c, s[e].x, acc.x);
          acc.y = fmaf(c, s[e].y, acc.y);
          acc.z = fmaf(c, s[e].z, acc.z);
          acc.w = fmaf(c, s[e].w, acc.w);
        }
        // the row groups of a warp first
#pragma unroll
        for (int o = CG; o < 32; o <<= 1) {
          acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
          acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
          acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
          acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
        }
        if ((tid & 31) < CG) *reinterpret_cast<float4*>(part + (i * NW + (tid >> 5)) * DV + 4 * cg) = acc;
      }
      __syncthreads();
      for (int x2 = tid; x2 < m * DV; x2 += NT) {
        const int i = x2 / DV, c = x2 % DV;
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < NW; ++r) t += part[(i * NW + r) * DV + c];
        put((i0 + i) * DV + c, t);
      }
    }
  };
  if constexpr (kDelta) read_rows(fk, [&](int at, float t) { vs[at] -= t; });   // v - S^T k
  read_rows(fq, [&](int at, float t) { qs[at] = t; });
  __syncthreads();

  if constexpr (kDelta) {
    // u_j over column c, one thread each: row j needs the rows on its path
    const float* at = sm + L.w2;
    for (int c = tid; c < DV; c += NT)
      for (int j = 0; j < n; ++j) {
        float u = vs[j * DV + c];
        for (unsigned long long m = mask[j] & ((1ull << j) - 1); m != 0ull; m &= m - 1) {
          const int l = __ffsll((long long)m) - 1;
          u = fmaf(-at[l * WP + j], vs[l * DV + c], u);
        }
        vs[j * DV + c] = u;
      }
    __syncthreads();
  } else {
    // 1 / den_i, one warp per node
    for (int i = tid >> 5; i < n; i += NT / 32) {
      float t = 0.f;
      for (int r = tid & 31; r < DK; r += 32) t = fmaf(fq[i * QP + r], sm[L.z + r], t);
      t *= pw[depth[i]];
      for (int j = tid & 31; j <= i; j += 32) t += wt[j * WP + i];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if ((tid & 31) == 0) sm[L.den + i] = 1.f / (t + eps);
    }
    __syncthreads();
  }

  // out_i = (read + sum over the path) / den: 4 nodes x 4 columns per thread
  T* ob = out + bh * (long long)ntok * DV;
  for (int i0 = 4 * rg; i0 < n; i0 += 4 * RG) {
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

// The largest layout of any call (a call of 16 rows has the longer groups).
template <int DK, int DV, bool kDelta>
constexpr int tree_smem_most() {
  const int a = TreeSmem<DK, DV, kDelta>(16, 16).total, b = TreeSmem<DK, DV, kDelta>(kTreeMax, kTreeMax).total;
  return a > b ? a : b;
}

template <int DK, int DV, typename T, bool kDelta>
cudaError_t launch(const TreeArgs& a) {
  const int smem = TreeSmem<DK, DV, kDelta>(a.T, a.T).total * (int)sizeof(float);
  auto kern = tree_simt_kernel<DK, DV, T, kDelta>;
  static KernelOnce once;
  int resident = 0;
  constexpr int most = tree_smem_most<DK, DV, kDelta>() * (int)sizeof(float);
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
