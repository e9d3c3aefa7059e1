// State advance: the state moves along each sequence's own accepted tokens,
//   S <- a S + phi(k_j) v_j^T,  z <- a z + phi(k_j)      (a = 1 without decay)
// or, for the delta rule,
//   u = S^T k_j,  S <- S + k_j (v_j - u)^T
// over j = path[0], path[1], ... path[accepted - 1] ("Linear Attention: KV를 고정
// 크기 상태에 누적하기", section "상태 갱신과 읽기를 식으로 정리하기"; decay and
// delta rule from "Linear Attention, 곱의 순서를 바꾸면 생기는 일"), in place or into
// another buffer.
//
// Memory-bound: the state is read and written once (64 KiB each way at
// dk = dv = 128) while a handful of tokens adds rank-one updates. One CTA of
// 128 threads per (batch, head); thread (rg, cg) holds rows rg*E .. rg*E+E-1,
// columns 4cg .. 4cg+3, its loads all in flight together (32 of 16 bytes at
// d = 128), and the state is read and written as data that is not soon wanted
// again, which leaves L2 to the writes: 2048 states by up to six tokens 44 us,
// 0.91 of the floor (256 threads 52, 512 64; without the hints 46). The delta
// rule joins its reads in shared memory once a token: four row groups of 128
// threads instead of eight, 2048 states 70 -> 57 us; by up to six tokens 49 us,
// 0.82 of the floor. A sequence that accepted
// nothing is not touched in place and copied otherwise.
#include "la_spec.cuh"

namespace la {

namespace {

enum { ADV_PLAIN = 0, ADV_DECAY = 1, ADV_DELTA = 2 };

template <int DK, int DV>
struct AdvShape {
  static constexpr int CG = DV / 4;
  static constexpr int NT = (CG * DK) < 128 ? (CG * DK) : 128;
  static constexpr int RG = NT / CG;
  static constexpr int E = DK / RG;
  static constexpr int TG = 8;                       // tokens staged at a time
};

template <int E>
__device__ __forceinline__ void load_rows(const float* x, float (&r)[E]) {
  if constexpr (E % 4 == 0) {
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const float4 f = *reinterpret_cast<const float4*>(x + e);
      r[e] = f.x; r[e + 1] = f.y; r[e + 2] = f.z; r[e + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) r[e] = x[e];
  }
}

template <int DK, int DV, typename T, int kRule>
__global__ void __launch_bounds__(AdvShape<DK, DV>::NT)
advance_kernel(const float* S, const float* z, const T* __restrict__ k, const T* __restrict__ v,
               const int* __restrict__ path, const int* __restrict__ accepted, float* S_out, float* z_out, int H,
               int ntok, const float* __restrict__ alpha) {
  using Sh = AdvShape<DK, DV>;
  constexpr int NT = Sh::NT, CG = Sh::CG, RG = Sh::RG, E = Sh::E, TG = Sh::TG;
  static_assert(NT % 32 == 0 && E >= 1 && NT >= DK && NT >= DV, "layout");
  __shared__ __align__(16) float fk[TG][DK];
  __shared__ __align__(16) float vs[TG][DV];
  __shared__ __align__(16) float part[kRule == ADV_DELTA ? 2 : 1][kRule == ADV_DELTA ? RG : 1][DV];

  const long long bh = blockIdx.x;
  const int b = (int)(bh / H), h = (int)(bh % H), tid = threadIdx.x;
  // in place, a sequence without tokens is left alone before its state is read;
  // into another buffer the state is read in any case, and first
  int n = accepted == nullptr ? ntok : min(max(accepted[b], 0), ntok);
  if (S == S_out && n == 0) return;
  const float a = kRule == ADV_DECAY ? alpha[h] : 1.f;
  const int cg = tid % CG, rg = tid / CG;
  const float4* Sb = reinterpret_cast<const float4*>(S + bh * (long long)DK * DV);
  float4* So = reinterpret_cast<float4*>(S_out + bh * (long long)DK * DV);
  float4 s[E];
#pragma unroll
  for (int e = 0; e < E; ++e) s[e] = __ldcs(&Sb[(rg * E + e) * CG + cg]);
  float zr = 0.f;
  if (kRule != ADV_DELTA && tid < DK) zr = z[bh * DK + tid];
  const T* kb = k + bh * (long long)ntok * DK;
  const T* vb = v + bh * (long long)ntok * DV;
  const int* pb = path == nullptr ? nullptr : path + (long long)b * ntok;

  for (int g0 = 0; g0 < n; g0 += TG) {
    const int m = min(TG, n - g0);
    int live = m;                              // an index outside the rows ends the path
    if (pb != nullptr)
      for (int t = m - 1; t >= 0; --t) {
        const int j = pb[g0 + t];
        if (j < 0 || j >= ntok) live = t;
      }
    if (g0 > 0) __syncthreads();               // the previous group has been read
    for (int x = tid; x < live * DK; x += NT) {
      const int t = x / DK, r = x % DK;
      const int j = pb == nullptr ? g0 + t : pb[g0 + t];
      const float y = to_f32<T>(kb[(long long)j * DK + r]);
      fk[t][r] = kRule == ADV_DELTA ? y : phi(y);
    }
    for (int x = tid; x < live * DV; x += NT) {
      const int t = x / DV, c = x % DV;
      const int j = pb == nullptr ? g0 + t : pb[g0 + t];
      vs[t][c] = to_f32<T>(vb[(long long)j * DV + c]);
    }
    __syncthreads();
    for (int t = 0; t < live; ++t) {
      float ka[E];
      load_rows<E>(&fk[t][rg * E], ka);
      float4 x = *reinterpret_cast<const float4*>(&vs[t][4 * cg]);
      if constexpr (kRule == ADV_DELTA) {
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          u.x = fmaf(ka[e], s[e].x, u.x);
          u.y = fmaf(ka[e], s[e].y, u.y);
          u.z = fmaf(ka[e], s[e].z, u.z);
          u.w = fmaf(ka[e], s[e].w, u.w);
        }
        // the row groups' sums, in two buffers taken in turn: one barrier a token
        *reinterpret_cast<float4*>(&part[t & 1][rg][4 * cg]) = u;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          const float4 p = *reinterpret_cast<const float4*>(&part[t & 1][r][4 * cg]);
          x.x -= p.x; x.y -= p.y; x.z -= p.z; x.w -= p.w;
        }
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        s[e].x = fmaf(ka[e], x.x, kRule == ADV_DECAY ? a * s[e].x : s[e].x);
        s[e].y = fmaf(ka[e], x.y, kRule == ADV_DECAY ? a * s[e].y : s[e].y);
        s[e].z = fmaf(ka[e], x.z, kRule == ADV_DECAY ? a * s[e].z : s[e].z);
        s[e].w = fmaf(ka[e], x.w, kRule == ADV_DECAY ? a * s[e].w : s[e].w);
      }
      if (kRule != ADV_DELTA && tid < DK) zr = kRule == ADV_DECAY ? fmaf(a, zr, fk[t][tid]) : zr + fk[t][tid];
    }
    if (live < m) break;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) __stcs(&So[(rg * E + e) * CG + cg], s[e]);
  if (kRule != ADV_DELTA && tid < DK) z_out[bh * DK + tid] = zr;
}

template <int DK, int DV, typename T>
cudaError_t launch(const AdvanceArgs& a) {
  auto kern = a.z == nullptr ? advance_kernel<DK, DV, T, ADV_DELTA>
              : a.alpha != nullptr ? advance_kernel<DK, DV, T, ADV_DECAY> : advance_kernel<DK, DV, T, ADV_PLAIN>;
  kern<<<a.BH, AdvShape<DK, DV>::NT, 0, a.stream>>>(a.S, a.z, (const T*)a.k, (const T*)a.v, a.path, a.accepted,
                                                    a.S_out, a.z_out, a.H, a.T, a.alpha);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

cudaError_t state_advance(const AdvanceArgs& a) {
#define LA_CASE(DK_, DV_)                                          \
  case DK_ * 1000 + DV_:                                           \
    return a.dtype == LA_BF16 ? launch<DK_, DV_, __nv_bfloat16>(a) \
                              : launch<DK_, DV_, float>(a);
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
