// Norm of every head of queries and keys with their rotation by position, and
// its gradient:
//   r = (c sum x^2 + eps)^(-1/2), y = x r w, z = y turned by position * freq
//   dy = dz turned back, dw = sum dy x r, dx = r (dy w - x c r^2 sum dy w x)
// Bound: HBM (each row is read and written once). A group of d * size / 16 lanes
// takes one token's row of a head, 16 bytes a lane, and goes on through the heads
// of the token: the sines and cosines of a (token, pair) are worked out once
// and stay in registers. A rotation's partner values come from the lane that holds
// them (the raw words, normed again: half as many exchanges for bf16), or are in the
// lane itself where neighbours are turned.
//
// Angles: freq / 2 pi as a 64-bit fraction F of a turn (an integer product with the
// first 128 bits of 1 / 2 pi), the angle is the low 64 bits of position * F: exact
// for every position up to the rounding of F, 2^-64 of a turn. (In fp64, F and its
// conversions took 2600 cycles a warp: that pipe takes an instruction every 64.) Of the
// angle the top 32 bits go on. For bf16 rows their sine and cosine are the special
// function unit's, off by 2^-21, a 2^12th of a bf16 step of 1; for fp32 rows sincospif of what is
// left of whole quarters of a turn: off by 2^-25 and two steps of the value.
#include "la_gated.cuh"

namespace la {

namespace {

constexpr int NT = 256;

template <typename T>
struct Vec {
  static constexpr int V = 16 / (int)sizeof(T);
  static __device__ __forceinline__ void split(const uint4& r, float* f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        f[i] = __uint_as_float(w[i]);
      } else {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  static __device__ __forceinline__ uint4 join(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = __float_as_uint(f[i]);
      } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

struct NormKernelArgs {
  const void* x[2]; void* y[2];
  const float* w[2];
  const int* positions; const float* freqs;
  int N, H0, H1, rot;
  long long tokens;
  long long stride[2][3];
  float c, eps;
  int heads_per;                 // heads of a token that one CTA row takes
  const void* dy[2];
  long long dstride[2][3];
  float* part;                   // backward: [CTA][2][d] partial sums of the weights' gradients
};

// freq / 2 pi turns, its fraction times 2^64: m 2^e / 2 pi with the 24-bit m of a
// float, from m times 1 / 2 pi as a 128-bit fraction.
__device__ __forceinline__ unsigned long long turn_fraction(float freq) {
  constexpr unsigned long long kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;
  const uint32_t w = __float_as_uint(freq);
  const int ex = (int)((w >> 23) & 0xff);
  const unsigned long long m = ex ? (w & 0x7fffffu) | 0x800000u : w & 0x7fffffu;
  const int shift = 64 - ((ex ? ex : 1) - 150 + 64);          // of m / 2 pi's words 2^0 .. 2^-128, to the right
  const unsigned long long p0 = m * kLo, c = __umul64hi(m, kLo), p1 = m * kHi + c;
  const unsigned long long p2 = __umul64hi(m, kHi) + (p1 < c);
  unsigned long long f;
  if (shift <= -64) f = shift <= -128 ? 0 : p0 << (-64 - shift);
  else if (shift < 0) f = (p1 << -shift) | (p0 >> (64 + shift));
  else if (shift == 0) f = p1;
  else if (shift < 64) f = (p1 >> shift) | (p2 << (64 - shift));
  else f = shift < 128 ? p2 >> (shift - 64) : 0;
  return (w >> 31) ? 0ull - f : f;
}

// Cosines and signed sines at a token: z_i = y_i c_i + y_partner s_i (1 and 0
// where components are not turned). turns: F of every pair, in shared memory.
template <int V, bool kInter, bool kFine>
__device__ __forceinline__ void angles(const NormKernelArgs& p, long long token, int n, int c0,
                                       const unsigned long long* turns, float (&cs)[V], float (&sn)[V]) {
  if (c0 >= p.rot) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
    }
    return;
  }
  const long long pos = p.positions != nullptr ? (long long)p.positions[token] : n;
  const int half = p.rot / 2;
  const bool second = c0 >= half;
  const unsigned long long* f = turns + (kInter ? c0 / 2 : second ? c0 - half : c0);
#pragma unroll
  for (int i = 0; i < (kInter ? V / 2 : V); ++i) {
    // the top 32 of 64 bits: in [-1/2, 1/2) turns, off by 2^-32 of one
    const uint32_t a = (uint32_t)(((unsigned long long)pos * f[i]) >> 32);
    float s, c;
    if constexpr (kFine) {
      const uint32_t quarter = (a + 0x20000000u) >> 30;
      float s0, c0;
      sincospif((float)(int)(a - (quarter << 30)) * 4.656612873077393e-10f, &s0, &c0);     // 2^-31
      s = quarter & 1 ? c0 : s0;
      c = quarter & 1 ? -s0 : c0;
      if (quarter & 2) {
        s = -s;
        c = -c;
      }
    } else {
      __sincosf((float)(int)a * 1.4629180792671596e-9f, &s, &c);     // a pi 2^-31
    }
    if (kInter) {
      cs[2 * i] = cs[2 * i + 1] = c;
      sn[2 * i] = -s;
      sn[2 * i + 1] = s;
    } else {
      cs[i] = c;
      sn[i] = second ? s : -s;
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Words of the lane that holds the other half of a pair.
__device__ __forceinline__ uint4 swap(const uint4& r, int partner) {
  return make_uint4(__shfl_sync(0xffffffffu, r.x, partner), __shfl_sync(0xffffffffu, r.y, partner),
                    __shfl_sync(0xffffffffu, r.z, partner), __shfl_sync(0xffffffffu, r.w, partner));
}

template <int D, typename T, bool kInter, bool kRot>
__global__ void __launch_bounds__(NT, 3)
norm_rotate_kernel(const NormKernelArgs p) {
  constexpr int V = Vec<T>::V, LPR = D / V, U = 4;    // U rows in flight beside U at work
  const int lane = threadIdx.x & 31, lr = lane % LPR, c0 = lr * V;
  const int hp = p.rot / 2 / V;                       // lanes between a pair's halves
  const int partner = (lane - lr) + (kInter || c0 >= p.rot ? lr : (lr < hp ? lr + hp : lr - hp));
  __shared__ __align__(16) unsigned long long turns[kRot ? D / 2 : 1];
  if (kRot) {
    if (threadIdx.x < p.rot / 2) turns[threadIdx.x] = turn_fraction(p.freqs[threadIdx.x]);
    __syncthreads();
  }
  const int h0 = blockIdx.y * p.heads_per, h1 = min(h0 + p.heads_per, p.H0 + p.H1);
  const long long token = blockIdx.x * (long long)(NT / LPR) + threadIdx.x / LPR;
  const bool live = token < p.tokens;
  const long long tk = live ? token : 0;
  const int b = (int)(tk / p.N), n = (int)(tk % p.N);
  float cs[V], sn[V];
  if (kRot) angles<V, kInter, sizeof(T) == 4>(p, tk, n, c0, turns, cs, sn);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int Hi = i ? p.H1 : p.H0, off = i ? p.H0 : 0;
    const int a0 = max(h0 - off, 0), a1 = min(h1 - off, Hi);
    if (a0 >= a1) continue;
    // weights with the cosines and, for the partner's values, the sines
    float wc[V], ws[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int pc = kInter ? c0 + (e ^ 1) : (partner % LPR) * V + e;
      wc[e] = p.w[i] != nullptr ? p.w[i][c0 + e] : 1.f;
      if (kRot) {
        wc[e] *= cs[e];
        ws[e] = (p.w[i] != nullptr ? p.w[i][pc] : 1.f) * sn[e];
      }
    }
    const T* src = (const T*)p.x[i] + b * p.stride[i][0] + n * p.stride[i][1] + c0;
    T* dst = (T*)p.y[i] + ((long long)b * Hi * p.N + n) * D + c0;
    // (without the next rows ahead, at two CTAs an SM: 72 us for 68 at 16384 tokens of 48 heads)
    uint4 nxt[U];
#pragma unroll
    for (int u = 0; u < U; ++u) nxt[u] = __ldcs(reinterpret_cast<const uint4*>(src + min(a0 + u, a1 - 1) * p.stride[i][2]));
    for (int hb = a0; hb < a1; hb += U) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[u] = nxt[u];
        if (hb + U < a1) nxt[u] = __ldcs(reinterpret_cast<const uint4*>(src + min(hb + U + u, a1 - 1) * p.stride[i][2]));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (hb + u >= a1) break;
        float x[V], z[V];
        Vec<T>::split(raw[u], x);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) ss = fmaf(x[e], x[e], ss);
        const float r = rsqrtf(fmaf(p.c, row_sum<LPR>(ss), p.eps));
        if (kRot) {
          float xp[V];
          if (kInter) {
#pragma unroll
            for (int e = 0; e < V; ++e) xp[e] = x[e ^ 1];
          } else {
            Vec<T>::split(swap(raw[u], partner), xp);
          }
#pragma unroll
          for (int e = 0; e < V; ++e) z[e] = fmaf(x[e], wc[e], xp[e] * ws[e]) * r;
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) z[e] = x[e] * wc[e] * r;
        }
        if (live) *reinterpret_cast<uint4*>(dst + (long long)(hb + u) * p.N * D) = Vec<T>::join(z);
      }
    }
  }
}

// Gradients: one row of x and of dz, one of dx out; the weights' sums stay in
// registers over the CTA's tokens and heads.
template <int D, typename T, bool kInter, bool kRot>
__global__ void __launch_bounds__(NT, 2)
norm_rotate_backward_kernel(const NormKernelArgs p) {
  constexpr int V = Vec<T>::V, LPR = D / V, TPB = NT / LPR, U = 4;
  const int lane = threadIdx.x & 31, lr = lane % LPR, c0 = lr * V;
  const int hp = p.rot / 2 / V;
  const int partner = (lane - lr) + (kInter || c0 >= p.rot ? lr : (lr < hp ? lr + hp : lr - hp));
  __shared__ __align__(16) unsigned long long turns[kRot ? D / 2 : 1];
  if (kRot) {
    if (threadIdx.x < p.rot / 2) turns[threadIdx.x] = turn_fraction(p.freqs[threadIdx.x]);
    __syncthreads();
  }
  float acc[2][V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[0][e] = acc[1][e] = 0.f;
  const int h0 = blockIdx.y * p.heads_per, h1 = min(h0 + p.heads_per, p.H0 + p.H1);
  for (long long base = blockIdx.x * (long long)TPB; base < p.tokens; base += gridDim.x * (long long)TPB) {
    const long long token = base + threadIdx.x / LPR;
    const bool live = token < p.tokens;
    const long long tk = live ? token : 0;
    const int b = (int)(tk / p.N), n = (int)(tk % p.N);
    float cs[V], sn[V];
    if (kRot) angles<V, kInter, sizeof(T) == 4>(p, tk, n, c0, turns, cs, sn);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int Hi = i ? p.H1 : p.H0, off = i ? p.H0 : 0;
      const int a0 = max(h0 - off, 0), a1 = min(h1 - off, Hi);
      if (a0 >= a1) continue;
      float w[V];
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = p.w[i] != nullptr ? p.w[i][c0 + e] : 1.f;
      const T* xs = (const T*)p.x[i] + b * p.stride[i][0] + n * p.stride[i][1] + c0;
      T* ds = (T*)p.y[i] + b * p.dstride[i][0] + n * p.dstride[i][1] + c0;
      const T* gs = (const T*)p.dy[i] + ((long long)b * Hi * p.N + n) * D + c0;
      for (int hb = a0; hb < a1; hb += U) {
        uint4 rx[U], rg[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = min(hb + u, a1 - 1);
          rx[u] = __ldcs(reinterpret_cast<const uint4*>(xs + h * p.stride[i][2]));
          rg[u] = __ldcs(reinterpret_cast<const uint4*>(gs + (long long)h * p.N * D));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (hb + u >= a1) break;
          float x[V], dy[V], dx[V];
          Vec<T>::split(rx[u], x);
          Vec<T>::split(rg[u], dy);
          if (kRot) {                                 // turned back
            float dp[V];
            if (kInter) {
#pragma unroll
              for (int e = 0; e < V; ++e) dp[e] = dy[e ^ 1];
            } else {
              Vec<T>::split(swap(rg[u], partner), dp);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) dy[e] = fmaf(dy[e], cs[e], -dp[e] * sn[e]);
          }
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            ss = fmaf(x[e], x[e], ss);
            dx[e] = dy[e] * x[e];                     // (the weights' part, times r)
            dot = fmaf(dx[e], w[e], dot);
          }
          const float r = rsqrtf(fmaf(p.c, row_sum<LPR>(ss), p.eps));
          const float k = p.c * r * r * row_sum<LPR>(dot);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            if (live) acc[i][e] = fmaf(dx[e], r, acc[i][e]);
            dx[e] = r * fmaf(-x[e], k, dy[e] * w[e]);
          }
          if (live) *reinterpret_cast<uint4*>(ds + (hb + u) * p.dstride[i][2]) = Vec<T>::join(dx);
        }
      }
    }
  }
  if (p.part == nullptr) return;
  __shared__ float sm[NT * V];
  const long long cta = blockIdx.x + (long long)blockIdx.y * gridDim.x;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) sm[(threadIdx.x / LPR) * D + c0 + e] = acc[i][e];
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll 8
      for (int t = 0; t < TPB; ++t) s += sm[t * D + threadIdx.x];
      p.part[(cta * 2 + i) * D + threadIdx.x] = s;
    }
  }
}

// The CTAs' sums of the weights' gradients: a CTA takes 16 components of one
// weight, 64 threads each, which share the parts.
__global__ void __launch_bounds__(1024)
norm_weight_sums_kernel(const float* part, int ctas, int D, float* dw0, float* dw1) {
  __shared__ float sm[64][17];
  const int i = blockIdx.y, d = blockIdx.x * 16 + threadIdx.x % 16, t0 = threadIdx.x / 16;
  float* dst = i ? dw1 : dw0;
  if (dst == nullptr) return;
  float s = 0.f;
#pragma unroll 4
  for (int c = t0; c < ctas; c += 64) s += part[((long long)c * 2 + i) * D + d];
  sm[t0][threadIdx.x % 16] = s;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp >= 16) return;
  s = sm[lane][warp] + sm[lane + 32][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) dst[blockIdx.x * 16 + warp] = s;
}

NormKernelArgs kernel_args(const NormArgs& a) {
  NormKernelArgs p{};
  for (int i = 0; i < 2; ++i) {
    p.x[i] = a.x[i]; p.y[i] = a.y[i]; p.w[i] = a.w[i]; p.dy[i] = a.dy[i];
    for (int j = 0; j < 3; ++j) {
      p.stride[i][j] = a.stride[i][j];
      p.dstride[i][j] = a.dstride[i][j];
    }
  }
  p.positions = a.positions; p.freqs = a.freqs;
  p.N = a.N; p.H0 = a.H[0]; p.H1 = a.H[1]; p.rot = a.rot;
  p.tokens = (long long)a.B * a.N;
  p.c = a.l2 ? 1.f : 1.f / (float)a.d;
  p.eps = a.eps;
  return p;
}

// Heads that a CTA takes for each of its tokens: all, or half as often as that
// leaves at least `least` to a token's sines and gives no more than `want` CTAs.
int heads_per_cta(long long ctas, int heads, int least, long long want) {
  int per = heads;
  while ((per + 1) / 2 >= least && ctas * ((heads + per - 1) / per) < want) per = (per + 1) / 2;
  return per;
}
// Few tokens: down to 4 heads, until every SM has CTAs (64 tokens of 32 heads 3.3 us
// against 10 with all heads in a CTA, gradient of 512 tokens of 48 heads 8.3 against 18); many: a
// token's heads in halves while that gives a better last wave (16384 tokens of 48 heads
// 68 us, 71 with all in a CTA, 99 with 4; gradient 108, 115, 187).
int heads_per_cta(long long ctas, int heads) {
  const int per = heads_per_cta(ctas, heads, 4, 2 * kSlots);
  return per < heads ? per : heads_per_cta(ctas, heads, 20, 12 * kSlots);
}

// CTAs of the backward: at most a wave (two an SM), as many rounds for every
// CTA, each with a part of the weights' sums.
struct BackwardGrid { int x, y, per; };
BackwardGrid backward_grid(long long tokens, int heads, int d, int size) {
  const int tpb = NT / (d * size / 16);
  const long long ctas = (tokens + tpb - 1) / tpb;
  BackwardGrid g;
  g.per = heads_per_cta(ctas, heads);
  g.y = (heads + g.per - 1) / g.per;
  long long most = (2LL * kSlots + g.y - 1) / g.y;
  const long long rounds = (ctas + most - 1) / most;
  most = (ctas + rounds - 1) / rounds;
  g.x = (int)(ctas < most ? ctas : most);
  return g;
}

template <int D, typename T, bool kInter, bool kRot>
cudaError_t launch(const NormArgs& a, bool backward) {
  NormKernelArgs p = kernel_args(a);
  constexpr int LPR = D / Vec<T>::V, TPB = NT / LPR;
  const int heads = a.H[0] + a.H[1];
  const long long ctas = (p.tokens + TPB - 1) / TPB;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (!backward) {
    p.heads_per = heads_per_cta(ctas, heads);
    const int gy = (heads + p.heads_per - 1) / p.heads_per;
    if (gy > 65535) return cudaErrorInvalidConfiguration;
    norm_rotate_kernel<D, T, kInter, kRot><<<dim3((unsigned)ctas, gy), NT, 0, a.stream>>>(p);
  } else {
    const BackwardGrid g = backward_grid(p.tokens, heads, D, (int)sizeof(T));
    if (g.y > 65535) return cudaErrorInvalidConfiguration;
    p.heads_per = g.per;
    const bool sums = a.dw[0] != nullptr || a.dw[1] != nullptr;
    p.part = sums ? a.workspace : nullptr;
    for (int i = 0; i < 2; ++i) p.y[i] = a.dx[i];
    norm_rotate_backward_kernel<D, T, kInter, kRot><<<dim3(g.x, g.y), NT, 0, a.stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    note_launch();
    if (!sums) return cudaSuccess;
    norm_weight_sums_kernel<<<dim3(D / 16, 2), 1024, 0, a.stream>>>(p.part, g.x * g.y, D, a.dw[0], a.dw[1]);
  }
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

template <int D, typename T>
cudaError_t launch_t(const NormArgs& a, bool backward) {
  if (a.rot == 0) return launch<D, T, false, false>(a, backward);
  return a.interleaved ? launch<D, T, true, true>(a, backward) : launch<D, T, false, true>(a, backward);
}

cudaError_t dispatch(const NormArgs& a, bool backward) {
  const bool bf = a.dtype == LA_BF16;
  switch (a.d) {
    case 16: return bf ? launch_t<16, __nv_bfloat16>(a, backward) : launch_t<16, float>(a, backward);
    case 32: return bf ? launch_t<32, __nv_bfloat16>(a, backward) : launch_t<32, float>(a, backward);
    case 64: return bf ? launch_t<64, __nv_bfloat16>(a, backward) : launch_t<64, float>(a, backward);
    case 128: return bf ? launch_t<128, __nv_bfloat16>(a, backward) : launch_t<128, float>(a, backward);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t norm_rotate(const NormArgs& a) { return dispatch(a, false); }
cudaError_t norm_rotate_backward(const NormArgs& a) { return dispatch(a, true); }

size_t norm_rotate_backward_workspace(int B, int N, int Hq, int Hk, int d, la_dtype dtype) {
  const BackwardGrid g = backward_grid((long long)B * N, Hq + Hk, d, dtype == LA_BF16 ? 2 : 4);
  return sizeof(float) * 2 * (size_t)d * g.x * g.y;
}

}  // namespace la
