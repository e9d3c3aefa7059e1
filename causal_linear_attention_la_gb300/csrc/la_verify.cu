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
// words, and p - q is kept whole in the same way. With u = 2^-24 a lane's sums
// over 16 values are off by 140 u^2 of themselves at most (the words' rounding
// errors are added up in fp32), a join of two pairs by 3 u^2; a lane joins 64
// such sums before they meet the rest. In all 2^-38 of the row's sum for up to
// 2^18 tokens, 2^-35 for 2^24, 2^-30 for 2^30 at worst; rows of random weights
// come out within 2^-48. (One plain fp32 sum of all of a lane's rounding errors
// had 2^-38 there with 4096 values a lane, 2^-25 with 32768.)
//
// One thread-block cluster per sequence: each CTA takes a contiguous part of
// the vocabulary, each warp a contiguous part of that, so that the joined
// sums are prefix sums in token order. Every warp sends its sum to all CTAs
// (distributed shared memory), one warp of each finds the part that holds the answer
// by one scan over all of them; the CTA that has it splits it over its warps
// again and scans the last piece. (Sums joined per CTA first, and added up one
// after the other, took as long as the rows: 31 us for the trees below.)
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
__device__ __forceinline__ void peer_store(uint32_t addr, int x) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}

// A number as the sum of two fp32 words, |l| at most half a step of h.
struct __align__(8) Pair {
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
__device__ __forceinline__ void peer_store(uint32_t addr, Pair x) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x.h), "f"(x.l) : "memory");
}
__device__ __forceinline__ Pair from_lane(Pair x, int lane) {
  return {__shfl_sync(0xffffffffu, x.h, lane), __shfl_sync(0xffffffffu, x.l, lane)};
}
// Sums over lanes 0 .. this one, for the first N lanes.
template <int N>
__device__ __forceinline__ Pair prefix(Pair x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < N; o <<= 1) {
    const Pair y = {__shfl_up_sync(0xffffffffu, x.h, o), __shfl_up_sync(0xffffffffu, x.l, o)};
    if (lane >= o) x = x + y;
  }
  return x;
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
// tie. Where p is tiny, both sides are scaled up first, so that neither a tie's
// product (it is near p) nor its error, 2^-48 of it at least, underflows. With q
// at 2^60 or more and p below 2^-60 there is no tie: u would be below 2^-120 and
// the product still 2^-89, which leaves its error room.
__device__ __forceinline__ bool stands(float u, float q, float p) {
  if (fabsf(p) < 0x1p-60f && fabsf(q) < 0x1p60f) {
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

// Where a draw with u ends up: the part (of nc * VW) that holds the answer, the
// sum of the parts before it, what the draw has to pass; `end`: rounding left
// no part, it is the last token with a weight in the last part that has one.
struct Found {
  Pair total, want, before;
  int part;
  bool end;
};

struct VerifyShared {
  Pair sums[kMaxCluster * VW];       // every warp's total, in every CTA of the cluster
  Pair sub_sum[VW];
  Found found_part;
  int piece;
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
  __device__ __forceinline__ void clear() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ float get(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  uint4 v;
  __device__ __forceinline__ void clear() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};

// The tokens of warp `w` of CTA `rank`, out of nc * VW parts in order, each a
// multiple of 32.
struct Part {
  int w0, w1;
  __device__ Part(int V, int rank, int nc, int w) {
    const int per = ((V + nc * VW - 1) / (nc * VW) + 31) & ~31;
    const long long lo = (long long)(rank * VW + w) * per;
    w0 = (int)min(lo, (long long)V);
    w1 = (int)min(lo + per, (long long)V);
  }
};

// This warp's sum of the weights of tokens [t0, t1), in groups of up to 16
// values and 64 groups (the precision above). vec: every row starts on
// a 16-byte boundary (t0 and t1 are multiples of a load then, or t1 = V is).
// Rows that start anywhere are read a value at a time, US loads in flight: 16
// for the tree (25.3 us for the trees below with 8, 24.0 with 16), 8 for the
// chain, which reads two rows and loses with the registers (17.2 and 17.9).
// (The children's rows brought into L2 during the search: a captured sequence
// of calls 24.0 -> 23.3 us, a call by itself 24.6 -> 26.6. Left out.)
template <int US, typename T>
__device__ Pair span_total(const T* p, const T* q, int t0, int t1, bool vec) {
  const int lane = threadIdx.x & 31;
  float hi = 0.f, lo = 0.f;
  auto add = [&](Pair w) {
    float r;
    two_sum(hi, w.h, hi, r);
    lo += w.l + r;
  };
  Pair group = {0.f, 0.f}, sum = {0.f, 0.f};
  int folds = 0;
  auto fold = [&] {
    group = group + normalised(hi, lo);
    hi = lo = 0.f;
    if ((++folds & 63) == 0) {
      sum = sum + group;
      group = {0.f, 0.f};
    }
  };
  // (batches of loads under their own bounds: a loop's remainder would wait for
  // every load by itself)
  constexpr int N = Vec<T>::N;
  if (vec) {
    constexpr int U = 4;
    for (int tb = t0 + N * lane; tb < t1; tb += U * 32 * N) {
      Vec<T> x[U], y[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int t = tb + i * 32 * N;
        x[i].clear();
        y[i].clear();
        if (t < t1) {
          x[i].load(p + t);
          if (q != nullptr) y[i].load(q + t);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (tb + i * 32 * N < t1) {
          if (q != nullptr) {
#pragma unroll
            for (int e = 0; e < N; ++e) add(weight(x[i].get(e), y[i].get(e)));
          } else {
#pragma unroll
            for (int e = 0; e < N; ++e) add(weight(x[i].get(e)));
          }
        }
        if ((i + 1) * N % 16 == 0) fold();
      }
    }
  } else {
    constexpr int U = US;
    for (int tb = t0 + lane; tb < t1; tb += U * 32) {
      float x[U], y[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int t = tb + i * 32;
        x[i] = y[i] = 0.f;
        if (t < t1) {
          x[i] = to_f32<T>(p[t]);
          if (q != nullptr) y[i] = to_f32<T>(q[t]);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) add(q != nullptr ? weight(x[i], y[i]) : weight(x[i]));
      fold();
    }
  }
  return warp_total(sum + group);
}

// The sums of all warps' parts of a row, in every CTA (one cluster barrier).
template <int US, typename T>
__device__ void row_sums(const T* p, const T* q, int V, bool vec, int rank, int nc, VerifyShared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Part part(V, rank, nc, warp);
  const Pair x = span_total<US>(p, q, part.w0, part.w1, vec);
  if (lane < nc) peer_store(peer(&sh.sums[rank * VW + warp], lane), x);
  __syncwarp();
  cluster_sync();
}

// By one warp, from row_sums: a lane takes PER sums in a row (nc / 2; one of 16
// for a single CTA).
template <int PER>
__device__ __forceinline__ Found find_part_warp(const VerifyShared& sh, int count, float u) {
  const int lane = threadIdx.x & 31;
  Pair c[PER], upto[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] = lane * PER + i < count ? sh.sums[lane * PER + i] : Pair{0.f, 0.f};
    upto[i] = i == 0 ? c[0] : upto[i - 1] + c[i];
  }
  const Pair through = prefix<32>(upto[PER - 1]);
  Found f;
  f.total = from_lane(through, 31);
  f.want = u * f.total;
  Pair front = {__shfl_up_sync(0xffffffffu, through.h, 1), __shfl_up_sync(0xffffffffu, through.l, 1)};
  if (lane == 0) front = {0.f, 0.f};
  // this lane's first sum that passes, and its last positive one
  int hit = -1, last = -1;
  Pair before = front;
#pragma unroll
  for (int i = PER - 1; i >= 0; --i)
    if (c[i].h > 0.f) {
      if (last < 0) last = i;
      if (front + upto[i] > f.want) {
        hit = i;
        before = i == 0 ? front : front + upto[i > 0 ? i - 1 : 0];
      }
    }
  const unsigned past = __ballot_sync(0xffffffffu, hit >= 0);
  const unsigned any = __ballot_sync(0xffffffffu, last >= 0);
  f.end = past == 0u;
  const int at = f.end ? (any != 0u ? 31 - __clz(any) : 0) : __ffs(past) - 1;
  f.part = at * PER + max(__shfl_sync(0xffffffffu, f.end ? last : hit, at), 0);
  f.before = from_lane(before, at);
  return f;
}

// By the CTA: one warp searches (the pair arithmetic of sixteen would queue up).
__device__ __forceinline__ Found find_part(VerifyShared& sh, int nc, float u) {
  if (threadIdx.x < 32) {
    const Found f = nc == 8 ? find_part_warp<4>(sh, nc * VW, u)
                    : nc == 4 ? find_part_warp<2>(sh, nc * VW, u) : find_part_warp<1>(sh, nc * VW, u);
    if (threadIdx.x == 0) sh.found_part = f;
  }
  __syncthreads();
  return sh.found_part;
}

// The token of a draw whose part this CTA has: that part again, over all warps.
// Returned to every thread.
template <typename T>
__device__ int draw(const T* p, const T* q, int V, const Found& f, int rank, int nc, VerifyShared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Part part(V, rank, nc, f.part % VW);
  const int sub = ((part.w1 - part.w0 + VW - 1) / VW + 31) & ~31;
  const int t0 = min(part.w0 + warp * sub, part.w1), t1 = min(t0 + sub, part.w1);
  auto token_weight = [&](int t) {
    if (t >= t1) return Pair{0.f, 0.f};
    const float a = to_f32<T>(p[t]);
    return q != nullptr ? weight(a, to_f32<T>(q[t])) : weight(a);
  };
  // (a piece of 32 tokens is scanned at once, a longer one summed first)
  Pair x = {0.f, 0.f}, upto = {0.f, 0.f}, sum;
  if (sub == 32) {
    x = token_weight(t0 + lane);
    upto = prefix<32>(x);
    sum = from_lane(upto, 31);
  } else {
    sum = span_total<8>(p, q, t0, t1, false);
  }
  if (lane == 0) sh.sub_sum[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    // the piece, and the sum in front of it
    const Pair c = lane < VW ? sh.sub_sum[lane] : Pair{0.f, 0.f};
    const Pair pieces = f.before + prefix<VW>(c);
    const bool some = lane < VW && c.h > 0.f;
    const unsigned past = __ballot_sync(0xffffffffu, some && pieces > f.want);
    const unsigned any = __ballot_sync(0xffffffffu, some);
    const bool end = f.end || past == 0u;
    const int m = end ? (any != 0u ? 31 - __clz(any) : 0) : __ffs(past) - 1;
    const Pair front = from_lane(pieces, m > 0 ? m - 1 : 0);
    if (lane == 0) {
      sh.piece = m;
      sh.found_part.before = m > 0 ? front : f.before;
      sh.found_part.end = end;
    }
  }
  __syncthreads();
  if (warp == sh.piece) {
    const Pair before = sh.found_part.before;
    Pair passed = {0.f, 0.f};                  // the piece's sum so far: joins of it are off by less than those of `before`
    const bool end = sh.found_part.end;
    int pick = -1;
    for (int t = t0; t < t1; t += 32) {
      if (sub != 32) {
        x = token_weight(t + lane);
        upto = prefix<32>(x);
      }
      const bool some = x.h > 0.f;
      const unsigned weighed = __ballot_sync(0xffffffffu, some);
      if (weighed == 0u) continue;
      pick = t + 31 - __clz(weighed);
      if (end) continue;
      const unsigned hit = __ballot_sync(0xffffffffu, some && before + (passed + upto) > f.want);
      if (hit != 0u) {
        pick = t + __ffs(hit) - 1;
        break;
      }
      passed = passed + from_lane(upto, 31);
    }
    if (lane == 0) sh.found = pick;
  }
  __syncthreads();
  return sh.found;
}

// A total that can be drawn from (an infinite weight, or more than fp32 holds,
// makes it infinite or no number).
__device__ __forceinline__ bool drawable(Pair total) { return total.h > 0.f && total.h <= 3.4e38f; }

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
  row_sums<8>(p, q, V, vec, rank, nc, sh);
  Found f = find_part(sh, nc, u);
  if (!(f.total.h > 0.f)) {
    // nothing left to draw from (p <= q everywhere): from p itself
    cluster_sync();                            // the sums have been read
    q = nullptr;
    row_sums<8>(p, q, V, vec, rank, nc, sh);
    f = find_part(sh, nc, u);
  }
  const bool some = drawable(f.total);
  const int t = some && f.part / VW == rank ? draw(p, q, V, f, rank, nc, sh) : -1;
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
    row_sums<16, T>(p, nullptr, V, vec, rank, nc, sh);
    const Found f = find_part(sh, nc, u);
    token = -1;
    int child = -1;
    if (drawable(f.total)) {
      const bool mine = f.part / VW == rank;
      const int t = mine ? draw<T>(p, nullptr, V, f, rank, nc, sh) : -1;
      if (mine && threadIdx.x < 32) {
        // the first child that holds the token (told in any case: a row that
        // changed since it was summed, by a caller's mistake, may give none, and
        // the others would go by what lies in their memory)
        int hit = -1;
        for (int i0 = 0; t >= 0 && i0 < all && hit < 0; i0 += 32) {
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

// CTAs per sequence: as many as keep 2048 tokens each and two CTAs per SM at
// most (64 chains over 131072 fp32 tokens, rows in L2: 8 CTAs 26 us, 4 20, 2 24,
// 1 36; 32 trees over 50021 bf16 tokens: 8 33 us, 4 32, 2 39, 1 52). More than
// eight would need the non-portable cluster size.
int cluster_size(int B, int V) {
  int nc = 1;
  while (nc < kMaxCluster && V > 2048 * nc && (long long)B * nc * 2 <= 2 * kSlots) nc *= 2;
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
  const int nc = cluster_size(a.B, a.V);
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
