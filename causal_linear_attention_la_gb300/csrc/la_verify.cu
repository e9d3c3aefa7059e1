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
// probability e, so the sums need far more than fp32: a lane sums in two fp32
// words (the rounding error of every addition kept, about 48 bits), the
// lanes' sums are joined in fp64 - the fp64 pipe is too slow for one addition
// per weight. p - q is likewise kept whole (the difference and its error).
//
// One thread-block cluster per sequence: each CTA takes a contiguous part of
// the vocabulary, each warp a contiguous part of that, so that the joined
// sums are prefix sums in token order; the CTAs exchange their totals through
// distributed shared memory, the one whose part holds the answer goes through
// the right warp's part again and tells the others. Every decision that the
// cluster's barriers depend on is taken by one CTA and sent to the rest.
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
__device__ __forceinline__ void peer_store(uint32_t addr, double x) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(x) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t addr, int x) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}

// (s, e): s + e = a + b exactly (Knuth's two-sum).
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}

// The weight of one token, as two fp32 words: p, or max(p - q, 0). Anything
// not above zero (a NaN too) weighs nothing.
template <typename T, bool kRest>
__device__ __forceinline__ void weight(const T* p, const T* q, long long t, float& s, float& e) {
  if constexpr (kRest) {
    two_sum(to_f32<T>(p[t]), -to_f32<T>(q[t]), s, e);
    if (!(s > 0.f)) s = e = 0.f;
  } else {
    s = to_f32<T>(p[t]);
    e = 0.f;
    if (!(s > 0.f)) s = 0.f;
  }
}

struct VerifyShared {
  double warp_sum[VW];
  double cta_sum[kMaxCluster];       // every CTA's total, in every CTA
  int answer[2];                     // token drawn, child entered
  int n;                             // chain: tokens that stand
  int par[kTreeMax], tok[kTreeMax];
};

__device__ __forceinline__ double warp_total(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// This CTA's part [c0, c1) of the V tokens and each warp's part of it.
struct Part {
  int w0, w1;
  __device__ Part(int V, int rank, int nc, int warp) {
    const int per = ((V + nc * VW - 1) / (nc * VW) + 31) & ~31;    // tokens per warp, whole lines
    const long long lo = (long long)(rank * VW + warp) * per;
    w0 = (int)min(lo, (long long)V);
    w1 = (int)min(lo + per, (long long)V);
  }
};

// Sums of this CTA's part, sent to every CTA of the cluster; returns the
// row's total (the same number in every CTA).
template <typename T, bool kRest>
__device__ double row_total(const T* p, const T* q, int V, int rank, int nc, VerifyShared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Part part(V, rank, nc, warp);
  float hi = 0.f, lo = 0.f;
#pragma unroll 8
  for (int t = part.w0 + lane; t < part.w1; t += 32) {
    float s, e, r;
    weight<T, kRest>(p, q, t, s, e);
    two_sum(hi, s, hi, r);
    lo += e + r;
  }
  const double x = warp_total((double)hi + (double)lo);
  if (lane == 0) sh.warp_sum[warp] = x;
  __syncthreads();
  if (threadIdx.x < nc) {
    double t = 0.0;
    for (int w = 0; w < VW; ++w) t += sh.warp_sum[w];
    peer_store(peer(&sh.cta_sum[rank], threadIdx.x), t);
  }
  __syncwarp();
  cluster_sync();
  double total = 0.0;
  for (int r = 0; r < nc; ++r) total += sh.cta_sum[r];
  return total;
}

// The token drawn with u, by warp 0 of the CTA whose part holds it (the other
// CTAs get -1): `total` > 0 from row_total on the same row.
template <typename T, bool kRest>
__device__ int draw(const T* p, const T* q, int V, float u, double total, int rank, int nc, const VerifyShared& sh) {
  const double want = (double)u * total;
  // the CTA: the first whose prefix passes `want`; rounding can leave none,
  // then the last one that weighs anything
  int owner = -1, last = 0;
  double before = 0.0, sum = 0.0;
  for (int r = 0; r < nc; ++r) {
    const double c = sh.cta_sum[r];
    if (c > 0.0) last = r;
    if (owner < 0 && sum + c > want) {
      owner = r;
      before = sum;
    }
    sum += c;
  }
  const bool none = owner < 0;
  if (none) owner = last;
  if (owner != rank || threadIdx.x >= 32) return -1;
  // the warp's part of it, in the same way
  int w = -1;
  last = 0;
  sum = before;
  for (int i = 0; i < VW; ++i) {
    const double c = sh.warp_sum[i];
    if (c > 0.0) last = i;
    if (!none && w < 0 && sum + c > want) {
      w = i;
      before = sum;
    }
    sum += c;
  }
  const bool end = w < 0;            // the last token with a weight, in that part
  if (end) w = last;
  const Part part(V, rank, nc, w);
  const int lane = threadIdx.x;
  int pick = -1;
  for (int t0 = part.w0; t0 < part.w1; t0 += 32) {
    float s = 0.f, e = 0.f;
    if (t0 + lane < part.w1) weight<T, kRest>(p, q, t0 + lane, s, e);
    const unsigned some = __ballot_sync(0xffffffffu, s > 0.f);
    if (some == 0u) continue;
    const int top = t0 + 31 - __clz(some);
    if (!end) {
      double x = (double)s + (double)e;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, s > 0.f && before + x > want);
      if (past != 0u) return t0 + __ffs(past) - 1;
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    pick = top;
  }
  return pick;
}

template <typename T>
__global__ void __launch_bounds__(VT)
chain_kernel(const T* __restrict__ target, const T* __restrict__ draft, const int* __restrict__ tokens,
             const int* __restrict__ count, const float* __restrict__ uniform, int* __restrict__ accepted,
             int* __restrict__ next, int ntok, int V, int nc) {
  __shared__ VerifyShared sh;
  const int rank = (int)cluster_rank(), b = blockIdx.x / nc;
  const T* pb = target + (long long)b * (ntok + 1) * V;
  const T* qb = draft + (long long)b * ntok * V;
  const int all = clamp_count(count, b, ntok);
  cluster_arrive();                            // every CTA runs before one writes to another
  int n = all;
  if (rank == 0 && threadIdx.x < 32) {
    // the first token that falls
    for (int i0 = 0; i0 < all && n == all; i0 += 32) {
      const int i = i0 + threadIdx.x;
      bool stands = true;
      if (i < all) {
        const int x = tokens[(long long)b * ntok + i];
        stands = x >= 0 && x < V;
        if (stands) {
          const float px = to_f32<T>(pb[(long long)i * V + x]), qx = to_f32<T>(qb[(long long)i * V + x]);
          // both products of two fp32 numbers are exact in fp64
          stands = (double)uniform[(long long)b * (ntok + 1) + i] * (double)qx < (double)px;
        }
      }
      const unsigned falls = __ballot_sync(0xffffffffu, !stands);
      if (falls != 0u) n = i0 + __ffs(falls) - 1;
    }
  }
  __syncwarp();
  cluster_wait();
  if (rank == 0 && threadIdx.x < nc) peer_store(peer(&sh.n, threadIdx.x), n);
  __syncwarp();
  cluster_sync();
  n = sh.n;
  const T* p = pb + (long long)n * V;
  const T* q = qb + (long long)n * V;
  const float u = uniform[(long long)b * (ntok + 1) + ntok];
  double total = 0.0;
  if (n < all) total = row_total<T, true>(p, q, V, rank, nc, sh);
  int t = -1;
  if (total > 0.0) {
    t = draw<T, true>(p, q, V, u, total, rank, nc, sh);
  } else {
    // none fell - or p <= q everywhere, where nothing is left to draw from
    if (n < all) cluster_sync();               // the totals have been read
    total = row_total<T, false>(p, q, V, rank, nc, sh);
    if (total > 0.0) t = draw<T, false>(p, q, V, u, total, rank, nc, sh);
  }
  if (threadIdx.x == 0) {
    if (rank == 0) accepted[b] = n;
    if (t >= 0) next[b] = t;
    if (rank == 0 && !(total > 0.0)) next[b] = -1;
  }
  __syncwarp();
  cluster_sync();                              // no CTA leaves while a peer may still write to it
}

template <typename T>
__global__ void __launch_bounds__(VT)
tree_verify_kernel(const T* __restrict__ target, const int* __restrict__ tokens, const int* __restrict__ parent,
                   const int* __restrict__ count, const float* __restrict__ uniform, int* __restrict__ path,
                   int* __restrict__ accepted, int* __restrict__ next, int ntok, int V, int nc) {
  __shared__ VerifyShared sh;
  const int rank = (int)cluster_rank(), b = blockIdx.x / nc;
  const T* pb = target + (long long)b * (ntok + 1) * V;
  const int all = clamp_count(count, b, ntok);
  if (threadIdx.x < all) {
    sh.par[threadIdx.x] = tree_parent(parent + (long long)b * ntok, threadIdx.x);
    sh.tok[threadIdx.x] = tokens[(long long)b * ntok + threadIdx.x];
  }
  if (threadIdx.x < kMaxCluster) sh.cta_sum[threadIdx.x] = 0.0;
  if (threadIdx.x == 0) sh.answer[0] = sh.answer[1] = -1;
  __syncwarp();
  cluster_sync();
  int at = -1, n = 0, token = -1;
  // a child comes after its parent, so that there are at most `ntok` steps down
  for (int step = 0; step <= ntok; ++step) {
    const T* p = pb + (long long)(at + 1) * V;
    const float u = uniform[(long long)b * (ntok + 1) + at + 1];
    const double total = row_total<T, false>(p, nullptr, V, rank, nc, sh);
    token = -1;
    int child = -1;
    if (total > 0.0) {
      const int t = draw<T, false>(p, nullptr, V, u, total, rank, nc, sh);
      if (threadIdx.x < 32 && __shfl_sync(0xffffffffu, t, 0) >= 0) {
        // the first child that holds the token
        int hit = -1;
        for (int i0 = 0; i0 < all && hit < 0; i0 += 32) {
          const int i = i0 + threadIdx.x;
          const unsigned m = __ballot_sync(0xffffffffu, i < all && i > at && sh.par[i] == at && sh.tok[i] == t);
          if (m != 0u) hit = i0 + __ffs(m) - 1;
        }
        if (threadIdx.x < nc) {
          peer_store(peer(&sh.answer[0], threadIdx.x), t);
          peer_store(peer(&sh.answer[1], threadIdx.x), hit);
        }
      }
      __syncwarp();
      cluster_sync();
      token = sh.answer[0];
      child = sh.answer[1];
    }
    if (child < 0) break;
    if (rank == 0 && threadIdx.x == 0) path[(long long)b * ntok + n] = child;
    __syncwarp();
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
  __syncwarp();
  cluster_sync();
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
  const T* p = (const T*)a.target;
  const cudaError_t e =
      a.draft != nullptr || a.parent == nullptr
          ? launch_cluster(chain_kernel<T>, a.B, nc, a.stream, p, (const T*)a.draft, a.tokens, a.count, a.uniform,
                           a.accepted, a.next, a.T, a.V, nc)
          : launch_cluster(tree_verify_kernel<T>, a.B, nc, a.stream, p, a.tokens, a.parent, a.count, a.uniform, a.path,
                           a.accepted, a.next, a.T, a.V, nc);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

cudaError_t verify(const VerifyArgs& a) {
  return a.dtype == LA_BF16 ? launch<__nv_bfloat16>(a) : launch<float>(a);
}

}  // namespace la
