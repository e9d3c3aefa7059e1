// Verification of drafted tokens against the target's probabilities, from
// given random numbers.
//
// Chain (the draft's own distributions q_0 .. q_{T-1} known): token i, drawn
// from q_i, stands if all before it stand and u_i q_i(x_i) < p_i(x_i), i.e.
// with probability min(1, p_i(x_i) / q_i(x_i)). The token after the n that
// stand is drawn from max(p_n - q_n, 0) (normalised) where one fell, from p_n
// where none did: its law is then exactly the target's.
// Tree: at a context c (the committed state, or the last accepted node) a
// token is drawn from p_c with u_c; a child of c that holds it is accepted and
// becomes the context, else the token is the answer. Every token is a sample
// of the target's, whatever drafted the tree.
//
// A draw from weights w_0 .. w_{V-1} with u takes the smallest t with
// w_0 + ... + w_t > u (w_0 + ... + w_{V-1}). A vocabulary of 131072 has as
// many borders, and a border that moves by e changes an answer with
// probability e, so the sums need far more than fp32. fp64 would do, but its
// pipe gives a warp's addition once in 64 cycles here (64 chains over 131072
// tokens with the joins alone in fp64: 79 us): all sums are pairs of fp32
// words with the rounding error of every addition kept (about 46 bits). p - q
// is kept whole in the same way.
//
// One thread-block cluster per sequence: each CTA takes a contiguous part of
// the vocabulary, each warp a contiguous part of that, so that the joined
// sums are prefix sums in token order. The CTAs exchange their totals through
// distributed shared memory; the one whose part holds the answer finds the
// warp's part, splits that over its warps again and scans the last piece.
// Bound by latency up to a few sequences (row, exchange, search one after the
// other) and by HBM beyond. Barriers of the cluster stand where every CTA comes by:
// what they depend on is exchanged, not worked out by each CTA for itself.
#include "la_tree.cuh"

namespace la {

namespace {

constexpr int VT = 512;               // threads per CTA
constexpr int VW = VT / 32;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// Address of the same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return a;
}
__device__ __forceinline__ void peer_store(uint32_t addr, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t addr, int x) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}

// A number as the sum of two fp32 words, |l| at most half a step of h.
struct Pair {
  float h, l;
};

// (s, e): s + e = a + b exactly (Knuth's two-sum).
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  const float x = __fadd_rn(a, b);
  const float bb = __fsub_rn(x, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(x, bb)), __fsub_rn(b, bb));
  s = x;
}
__device__ __forceinline__ Pair normalised(float h, float l) {
  const float s = __fadd_rn(h, l);
  return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
// Sums of numbers that are not negative: 2^-46 of the sum.
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  float s, e;
  two_sum(a.h, b.h, s, e);
  return normalised(s, __fadd_rn(e, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ bool operator>(Pair a, Pair b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }
__device__ __forceinline__ Pair operator*(float u, Pair a) {
  const float p = __fmul_rn(u, a.h);
  return normalised(p, __fmaf_rn(u, a.l, __fmaf_rn(u, a.h, -p)));
}
__device__ __forceinline__ Pair warp_total(Pair x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Pair y = {__shfl_xor_sync(0xffffffffu, x.h, o), __shfl_xor_sync(0xffffffffu, x.l, o)};
    x = x + y;
  }
  return x;
}

// u * q < p for fp32 numbers, exactly: the product's rounding error decides a
// tie. Tiny numbers are scaled up first, so that the error does not underflow.
__device__ __forceinline__ bool stands(float u, float q, float p) {
  if (fabsf(q) < 0x1p-60f && fabsf(p) < 0x1p-60f) {
    q *= 0x1p60f;
    p *= 0x1p60f;
  }
  const float x = __fmul_rn(u, q);
  return x < p || (x == p && __fmaf_rn(u, q, -x) < 0.f);
}

// The weight of one token: p, or max(p - q, 0) (exact as a Pair). Anything not
// above zero (a NaN too) weighs nothing.
__device__ __forceinline__ Pair weight(float p) { return {p > 0.f ? p : 0.f, 0.f}; }
__device__ __forceinline__ Pair weight(float p, float q) {
  Pair w;
  two_sum(p, -q, w.h, w.l);
  if (!(w.h > 0.f)) w = {0.f, 0.f};
  return w;
}

struct VerifyShared {
  Pair warp_sum[VW], sub_sum[VW];
  Pair cta_sum[kMaxCluster];         // every CTA's total, in every CTA
  int answer[2];                     // token drawn, child entered
  int found;
  int par[kTreeMax], tok[kTreeMax];
};

// N consecutive values as one load (4 fp32 or 8 bf16).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ float get(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};

// The tokens of warp `w` of CTA `rank`, out of nc * VW parts in order: whole
// vector loads of a warp.
struct Part {
  int w0, w1;
  __device__ Part(int V, int rank, int nc, int w) {
    const int per = ((V + nc * VW - 1) / (nc * VW) + 255) & ~255;
    const long long lo = (long long)(rank * VW + w) * per;
    w0 = (int)min(lo, (long long)V);
    w1 = (int)min(lo + per, (long long)V);
  }
};

// This warp's sum of the weights of tokens [t0, t1). vec: every row starts on
// a 16-byte boundary (t0 and t1 are multiples of a load then, or t1 = V is).
template <typename T>
__device__ Pair span_total(const T* p, const T* q, int t0, int t1, bool vec) {
  const int lane = threadIdx.x & 31;
  float hi = 0.f, lo = 0.f;
  auto add = [&](Pair w) {
    float r;
    two_sum(hi, w.h, hi, r);
    lo += w.l + r;
  };
  constexpr int N = Vec<T>::N;
  if (vec) {
    if (q != nullptr) {
#pragma unroll 4
      for (int t = t0 + N * lane; t < t1; t += 32 * N) {
        Vec<T> x, y;
        x.load(p + t);
        y.load(q + t);
#pragma unroll
        for (int i = 0; i < N; ++i) add(weight(x.get(i), y.get(i)));
      }
    } else {
#pragma unroll 4
      for (int t = t0 + N * lane; t < t1; t += 32 * N) {
        Vec<T> x;
        x.load(p + t);
#pragma unroll
        for (int i = 0; i < N; ++i) add(weight(x.get(i)));
      }
    }
  } else if (q != nullptr) {
#pragma unroll 8
    for (int t = t0 + lane; t < t1; t += 32) add(weight(to_f32<T>(p[t]), to_f32<T>(q[t])));
  } else {
#pragma unroll 8
    for (int t = t0 + lane; t < t1; t += 32) add(weight(to_f32<T>(p[t])));
  }
  return warp_total(normalised(hi, lo));
}

// The row's total, the same in every CTA: the parts' sums, this CTA's own sent
// to every CTA of the cluster (one cluster barrier).
template <typename T>
__device__ Pair row_total(const T* p, const T* q, int V, bool vec, int rank, int nc, VerifyShared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Part part(V, rank, nc, warp);
  const Pair x = span_total(p, q, part.w0, part.w1, vec);
  if (lane == 0) sh.warp_sum[warp] = x;
  __syncthreads();
  if (threadIdx.x < nc) {
    Pair t = sh.warp_sum[0];
    for (int w = 1; w < VW; ++w) t = t + sh.warp_sum[w];
    const uint32_t to = peer(&sh.cta_sum[rank], threadIdx.x);
    peer_store(to, t.h);
    peer_store(to + 4, t.l);
  }
  __syncwarp();
  cluster_sync();
  Pair total = sh.cta_sum[0];
  for (int r = 1; r < nc; ++r) total = total + sh.cta_sum[r];
  return total;
}

// The first of n sums whose prefix (from `before`) passes `want`, `before`
// then being the prefix in front of it; the last positive one (and `end`)
// where none does, as rounding may have it.
__device__ __forceinline__ int pass(const Pair* sums, int n, Pair want, Pair& before, bool& end) {
  int last = 0;
  Pair sum = before;
  for (int i = 0; i < n; ++i) {
    const Pair c = sums[i];
    if (!(c.h > 0.f)) continue;
    last = i;
    const Pair next = sum + c;
    if (!end && next > want) {
      before = sum;
      return i;
    }
    sum = next;
  }
  end = true;
  return last;
}

// The token drawn with u from a row whose row_total is `total` > 0: returned
// by every thread of the CTA whose part holds it, -1 elsewhere.
template <typename T>
__device__ int draw(const T* p, const T* q, int V, bool vec, float u, Pair total, int rank, int nc, VerifyShared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Pair want = u * total;
  Pair before = {0.f, 0.f};
  bool end = false;
  if (pass(sh.cta_sum, nc, want, before, end) != rank) return -1;
  const int w = pass(sh.warp_sum, VW, want, before, end);
  // that warp's part again, over all warps
  const Part part(V, rank, nc, w);
  const int sub = ((part.w1 - part.w0 + VW - 1) / VW + 31) & ~31;
  {
    const int t0 = min(part.w0 + warp * sub, part.w1);
    const Pair x = span_total(p, q, t0, min(t0 + sub, part.w1), false);
    if (lane == 0) sh.sub_sum[warp] = x;
  }
  __syncthreads();
  const int m = pass(sh.sub_sum, VW, want, before, end);
  if (warp == m) {
    const int t0 = part.w0 + m * sub, t1 = min(t0 + sub, part.w1);
    int pick = -1;
    for (int t = t0; t < t1; t += 32) {
      Pair x = {0.f, 0.f};
      if (t + lane < t1) {
        const float a = to_f32<T>(p[t + lane]);
        x = q != nullptr ? weight(a, to_f32<T>(q[t + lane])) : weight(a);
      }
      const bool some = x.h > 0.f;
      const unsigned any = __ballot_sync(0xffffffffu, some);
      if (any == 0u) continue;
      pick = t + 31 - __clz(any);
      if (end) continue;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Pair y = {__shfl_up_sync(0xffffffffu, x.h, o), __shfl_up_sync(0xffffffffu, x.l, o)};
        if (lane >= o) x = x + y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, some && before + x > want);
      if (past != 0u) {
        pick = t + __ffs(past) - 1;
        break;
      }
      before = before + Pair{__shfl_sync(0xffffffffu, x.h, 31), __shfl_sync(0xffffffffu, x.l, 31)};
    }
    if (lane == 0) sh.found = pick;
  }
  __syncthreads();
  return sh.found;
}

template <typename T>
__global__ void __launch_bounds__(VT)
chain_kernel(const T* __restrict__ target, const T* __restrict__ draft, const int* __restrict__ tokens,
             const int* __restrict__ count, const float* __restrict__ uniform, int* __restrict__ accepted,
             int* __restrict__ next, int ntok, int V, int nc, bool vec) {
  __shared__ VerifyShared sh;
  const int rank = (int)cluster_rank(), b = blockIdx.x / nc, lane = threadIdx.x & 31;
  const T* pb = target + (long long)b * (ntok + 1) * V;
  const T* qb = draft + (long long)b * ntok * V;
  const int all = clamp_count(count, b, ntok);
  const float u = uniform[(long long)b * (ntok + 1) + ntok];
  cluster_arrive();                            // every CTA runs before one writes to another
  // the first token that falls (by every warp for itself: no barrier needed)
  int n = all;
  for (int i0 = 0; i0 < all && n == all; i0 += 32) {
    const int i = i0 + lane;
    bool ok = true;
    if (i < all) {
      const int x = tokens[(long long)b * ntok + i];
      ok = x >= 0 && x < V &&
           stands(uniform[(long long)b * (ntok + 1) + i], to_f32<T>(qb[(long long)i * V + x]), to_f32<T>(pb[(long long)i * V + x]));
    }
    const unsigned falls = __ballot_sync(0xffffffffu, !ok);
    if (falls != 0u) n = i0 + __ffs(falls) - 1;
  }
  const T* p = pb + (long long)n * V;
  const T* q = n < all ? qb + (long long)n * V : nullptr;
  cluster_wait();
  Pair total = row_total(p, q, V, vec, rank, nc, sh);
  if (!(total.h > 0.f)) {
    // nothing left to draw from (p <= q everywhere): from p itself
    cluster_sync();                            // the totals have been read
    q = nullptr;
    total = row_total(p, q, V, vec, rank, nc, sh);
  }
  // (a row with an infinite weight has a total that is no number)
  const bool some = total.h > 0.f && total.h <= 3.4e38f;
  const int t = some ? draw(p, q, V, vec, u, total, rank, nc, sh) : -1;
  if (threadIdx.x == 0) {
    if (rank == 0) accepted[b] = n;
    if (t >= 0 || (rank == 0 && !some)) next[b] = t;
  }
}

template <typename T>
__global__ void __launch_bounds__(VT)
tree_verify_kernel(const T* __restrict__ target, const int* __restrict__ tokens, const int* __restrict__ parent,
                   const int* __restrict__ count, const float* __restrict__ uniform, int* __restrict__ path,
                   int* __restrict__ accepted, int* __restrict__ next, int ntok, int V, int nc, bool vec) {
  __shared__ VerifyShared sh;
  const int rank = (int)cluster_rank(), b = blockIdx.x / nc, lane = threadIdx.x & 31;
  const T* pb = target + (long long)b * (ntok + 1) * V;
  const int all = clamp_count(count, b, ntok);
  cluster_arrive();                            // every CTA runs before one writes to another
  if (threadIdx.x < all) {
    sh.par[threadIdx.x] = tree_parent(parent + (long long)b * ntok, threadIdx.x);
    sh.tok[threadIdx.x] = tokens[(long long)b * ntok + threadIdx.x];
  }
  __syncwarp();
  cluster_wait();
  int at = -1, n = 0, token = -1;
  // a child comes after its parent, so that there are at most `ntok` steps down
  for (int step = 0; step <= ntok; ++step) {
    const T* p = pb + (long long)(at + 1) * V;
    const float u = uniform[(long long)b * (ntok + 1) + at + 1];
    const Pair total = row_total<T>(p, nullptr, V, vec, rank, nc, sh);
    token = -1;
    int child = -1;
    if (total.h > 0.f && total.h <= 3.4e38f) {
      const int t = draw<T>(p, nullptr, V, vec, u, total, rank, nc, sh);
      if (t >= 0 && threadIdx.x < 32) {
        // the first child that holds the token
        int hit = -1;
        for (int i0 = 0; i0 < all && hit < 0; i0 += 32) {
          const int i = i0 + lane;
          const unsigned m = __ballot_sync(0xffffffffu, i < all && i > at && sh.par[i] == at && sh.tok[i] == t);
          if (m != 0u) hit = i0 + __ffs(m) - 1;
        }
        if (lane < nc) {
          peer_store(peer(&sh.answer[0], lane), t);
          peer_store(peer(&sh.answer[1], lane), hit);
        }
      }
      __syncwarp();
      cluster_sync();
      token = sh.answer[0];
      child = sh.answer[1];
    }
    if (child < 0) break;
    if (rank == 0 && threadIdx.x == 0) path[(long long)b * ntok + n] = child;
    ++n;
    at = child;
  }
  if (rank == 0) {
    for (int i = n + threadIdx.x; i < ntok; i += VT) path[(long long)b * ntok + i] = -1;
    if (threadIdx.x == 0) {
      accepted[b] = n;
      next[b] = token;
    }
  }
}

// CTAs per sequence. One CTA goes through about 4096 tokens before its joins
// cost less than its sums; more than eight would need the non-portable size.
int cluster_size(int V) {
  int nc = 1;
  while (nc < kMaxCluster && V > 4096 * nc) nc *= 2;
  return nc;
}

template <typename... Params, typename... Values>
cudaError_t launch_cluster(void (*kern)(Params...), int B, int nc, cudaStream_t stream, Values... values) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(B * nc));
  cfg.blockDim = dim3(VT);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)nc;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(values)...);
}

template <typename T>
cudaError_t launch(const VerifyArgs& a) {
  const int nc = cluster_size(a.V);
  const bool vec = a.V % Vec<T>::N == 0;           // rows on 16-byte boundaries
  const T* p = (const T*)a.target;
  const cudaError_t e =
      a.draft != nullptr || a.parent == nullptr
          ? launch_cluster(chain_kernel<T>, a.B, nc, a.stream, p, (const T*)a.draft, a.tokens, a.count, a.uniform,
                           a.accepted, a.next, a.T, a.V, nc, vec)
          : launch_cluster(tree_verify_kernel<T>, a.B, nc, a.stream, p, a.tokens, a.parent, a.count, a.uniform, a.path,
                           a.accepted, a.next, a.T, a.V, nc, vec);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

cudaError_t verify(const VerifyArgs& a) {
  return a.dtype == LA_BF16 ? launch<__nv_bfloat16>(a) : launch<float>(a);
}

}  // namespace la
