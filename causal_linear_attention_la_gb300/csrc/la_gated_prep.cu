// The triangles of every chunk of the gated delta rule: P = scale D o q.k and
// T = (I + X diag(beta))^-1, X = D o k.k strictly below the diagonal (formulas
// and record layout: la_gated_mma.cuh). One CTA of four warps per chunk slot
// and key head; k.k and q.k by mma once for all heads of values that share them.
//
// The inverse, in blocks: a lane per column substitutes in the 8 x 8 blocks on the
// diagonal, then 2 x 2 blocks are joined three times,
//   [A 0; B C]^-1 = [A^-1 0; -C^-1 B A^-1 C^-1],
// to 16 in fp32 on the CUDA cores, to 32 and 64 by mma with operands split in high and
// low parts: there B lies in the accumulators that made it, as the operand that is
// wanted, and Y^T = (B A^-1)^T comes out as the next product's. What a record holds is
// written from registers wherever it lies there as a fragment, transposed by movmatrix.
// A key, decay or beta that is not finite leaves no output and no state behind
// it finite, but must reach none before it, which a product with a zero above a diagonal would
// do: from the first such token on the triangles are made as if there were none,
// and e^G is NaN instead.
//
// Sums of g are pairs of fp32 in units of log 2: a difference of two keeps its
// digits behind a token that forgets nearly all, and fp64 would take 64 cycles an
// addition. (All inverse steps on the CUDA cores and fp64 sums: 181 us for 256 heads of
// 2048 tokens.)
#include <type_traits>

#include "la_gated_mma.cuh"

namespace la {

namespace {

using namespace gmma;

constexpr int PT = 128;         // threads
constexpr int LD = C + 4, LA = 20;      // floats per row of T, and of the blocks of 16

constexpr int HB = 4;           // heads whose sums of g are made at once

template <int DK>
struct PrepSmem {
  union {
    struct { __align__(16) uint8_t k[C * DK * 2], q[C * DK * 2]; };
    struct {                          // once the products are done
      __align__(16) float a[C * LA];  // X diag(beta) in the 16 x 16 blocks on the diagonal, one under the other
      __align__(16) float t[C * LD];  // T
      __align__(16) float4 part[4 * 32];    // from warp 2 to warp 3
    };
  };
  float gs[HB][C], gl[HB][C], eg[HB][C], ec[HB][C], beta[HB][C];
  int first_k[4], first_g[HB];        // first tokens that are not finite: by block of 16, by head
};

struct PrepArgs {
  const __nv_bfloat16* q; const __nv_bfloat16* k;
  const float* g; const float* beta;
  const int* offsets;
  uint8_t* rec;
  int4* chunks;                       // backward
  int Hk, H, N, nseq;
  float scale;
};

// Four values of a 16 x 16 block as the B fragments of its two 8-column tiles.
__device__ __forceinline__ void store_frag(uint8_t* dst, int block, int lane, const uint4& v) {
  *reinterpret_cast<uint4*>(dst + block * 512 + lane * 16) = v;
}

__device__ __forceinline__ float power2(float x) {      // (off by 2^-22; zero below 2^-126)
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// A fragment of 8 x 8 bf16 values (row lane / 4, two columns), transposed
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

struct Pair { float hi, lo; };
__device__ __forceinline__ Pair add(const Pair& a, const Pair& b) {
  const float s = a.hi + b.hi, bb = s - a.hi;
  const float l = (a.lo + b.lo) + ((a.hi - (s - bb)) + (b.hi - bb));
  Pair r;
  r.hi = s + l;
  r.lo = l - (r.hi - s);
  return r;
}
__device__ __forceinline__ Pair log2_pair(float g) {
  g = g < -128.f ? -128.f : g;                 // exp(-128) is zero in fp32; NaN stays
  constexpr float kL = 1.44269504f, kR = 1.92596299e-8f;      // log2(e) in two parts
  Pair r;
  r.hi = g * kL;
  r.lo = fmaf(g, kL, -r.hi) + g * kR;
  return r;
}

template <int DK, bool kBackward>
__global__ void __launch_bounds__(PT, 4)          // (256 heads of 2048 tokens 121 us; three CTAs an SM 135, five 125)
gated_prep_kernel(const PrepArgs p) {
  extern __shared__ __align__(16) uint8_t raw[];
  PrepSmem<DK>& sm = *reinterpret_cast<PrepSmem<DK>*>(raw);
  constexpr int CH = DK / 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, tig = lane & 3;
  const int slot = blockIdx.x / p.Hk, hk = blockIdx.x % p.Hk;
  const ChunkRange c = chunk_range(p.offsets, p.nseq, slot, p.N, C);
  if (kBackward && hk == 0 && tid == 0) p.chunks[slot] = make_int4(c.b, c.row, c.n, 0);
  if (c.n <= 0) return;
  const long long krow = ((long long)c.b * p.Hk + hk) * p.N + c.row;
  load_tile<CH, PT>(smem_addr(sm.k), p.k + krow * DK, DK, c.n, tid);
  load_tile<CH, PT>(smem_addr(sm.q), p.q + krow * DK, DK, c.n, tid);
  cp_commit();
  const int group = p.H / p.Hk;
  // sums of g and what comes of them for heads hb .. hb + 3, one a warp, two tokens a lane
  auto sums = [&](int hb) {
    const int hh = hb + warp;
    if (hh >= group) return;
    const long long vrow = ((long long)c.b * p.H + hk * group + hh) * p.N + c.row;
    const int t = 2 * lane;
    const Pair zero = {0.f, 0.f};
    const Pair x0 = t < c.n ? log2_pair(p.g[vrow + t]) : zero, x1 = t + 1 < c.n ? log2_pair(p.g[vrow + t + 1]) : zero;
    Pair s = add(x0, x1);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      Pair y;
      y.hi = __shfl_up_sync(0xffffffffu, s.hi, o);
      y.lo = __shfl_up_sync(0xffffffffu, s.lo, o);
      if (lane >= o) s = add(y, s);
    }
    Pair last, before;
    last.hi = -__shfl_sync(0xffffffffu, s.hi, 31);
    last.lo = -__shfl_sync(0xffffffffu, s.lo, 31);
    // (not s - x1: behind a token that is not finite the one before it stays clean)
    before.hi = __shfl_up_sync(0xffffffffu, s.hi, 1);
    before.lo = __shfl_up_sync(0xffffffffu, s.lo, 1);
    if (lane == 0) before = zero;
    const Pair both[2] = {add(before, x0), s};
    int first = C;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sm.gs[warp][t + e] = both[e].hi;
      sm.gl[warp][t + e] = both[e].lo;
      sm.eg[warp][t + e] = exp2f(both[e].hi);
      sm.ec[warp][t + e] = exp2f(-((last.hi + both[e].hi) + (last.lo + both[e].lo)));
      const float b = t + e < c.n ? p.beta[vrow + t + e] : 0.f;
      sm.beta[warp][t + e] = b;
      if (first == C && !(both[e].hi < INFINITY && fabsf(b) < INFINITY)) first = t + e;
    }
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sm.first_g[warp] = first;
  };
  sums(0);
  cp_wait<0>();
  __syncthreads();
  // rows 16 warp .. + 15 of k.k, columns up to the diagonal block; of q.k the
  // same, or in the backward k.q, columns from the diagonal block on
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) kk[j][e] = qk[j][e] = 0.f;
  {
    const int i = lane >> 3, l = lane & 7;
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t ak[4], aq[4];
      const uint32_t at = tile_at<CH>(16 * warp + ((i & 1) << 3) + l, 2 * ks + (i >> 1));
      ldmatrix4(ak, smem_addr(sm.k) + at);
      if (!kBackward) ldmatrix4(aq, smem_addr(sm.q) + at);
#pragma unroll
      for (int jb = 0; jb < 4; ++jb) {
        const uint32_t bt = tile_at<CH>(16 * jb + ((i >> 1) << 3) + l, 2 * ks + (i & 1));
        uint32_t b[4];
        if (jb <= warp) {
          ldmatrix4(b, smem_addr(sm.k) + bt);
          mma(kk[2 * jb], ak, b[0], b[1]);
          mma(kk[2 * jb + 1], ak, b[2], b[3]);
          if (!kBackward) {
            mma(qk[2 * jb], aq, b[0], b[1]);
            mma(qk[2 * jb + 1], aq, b[2], b[3]);
          }
        }
        if (kBackward && jb >= warp) {
          ldmatrix4(b, smem_addr(sm.q) + bt);
          mma(qk[2 * jb], ak, b[0], b[1]);
          mma(qk[2 * jb + 1], ak, b[2], b[3]);
        }
      }
    }
  }
  {
    // k.k on the diagonal: rows g and g + 8 are in the lanes with tig = g / 2
    int first = C;
#pragma unroll
    for (int jb = 0; jb < 4; ++jb)
      if (jb == warp && tig == (g >> 1)) {
        const float x0 = (g & 1) ? kk[2 * jb][1] : kk[2 * jb][0], x1 = (g & 1) ? kk[2 * jb + 1][3] : kk[2 * jb + 1][2];
        first = !(x0 < INFINITY) ? 16 * warp + g : !(x1 < INFINITY) ? 16 * warp + g + 8 : C;
      }
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sm.first_k[warp] = first;
  }
  __syncthreads();
  const int first_k = min(min(sm.first_k[0], sm.first_k[1]), min(sm.first_k[2], sm.first_k[3]));
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      qk[j][e] *= p.scale;
      if (first_k < C && max(16 * warp + g + 8 * (e >> 1), 8 * j + 2 * tig + (e & 1)) >= first_k) kk[j][e] = qk[j][e] = 0.f;
    }
  for (int hh = 0; hh < group; ++hh) {
    const int h = hk * group + hh, hs = hh % HB;
    uint8_t* rec = p.rec + ((long long)slot * p.H + h) * (kBackward ? REC_BWD : REC_FWD);
    __syncthreads();                       // the previous head's readers are done
    if (hh > 0 && hs == 0) {
      sums(hh);
      __syncthreads();
    }
    const int first = min(first_k, sm.first_g[hs]);
    if (first < C) {
      if (tid >= first && tid < C) {
        sm.gs[hs][tid] = first > 0 ? sm.gs[hs][first - 1] : 0.f;
        sm.gl[hs][tid] = first > 0 ? sm.gl[hs][first - 1] : 0.f;
        sm.beta[hs][tid] = 0.f;
        sm.eg[hs][tid] = NAN;
      }
      if (tid < C) sm.ec[hs][tid] = 1.f;
      __syncthreads();
    }
    const float *gs = sm.gs[hs], *gl = sm.gl[hs], *beta = sm.beta[hs];
    float* vec = reinterpret_cast<float*>(rec + OFF_VEC);
    if (tid < C) {
      vec[tid] = sm.eg[hs][tid];
      vec[C + tid] = sm.ec[hs][tid];
      vec[2 * C + tid] = beta[tid];
      if (kBackward) {
        reinterpret_cast<float*>(rec + OFF_SUMS)[tid] = gs[tid];
        reinterpret_cast<float*>(rec + OFF_SUMS)[C + tid] = gl[tid];
      }
    }
    // T, as pairs of columns of a row, B[k = j][n = t], and for the backward pairs of rows of
    // a column
    auto store_t = [&](int block, const uint32_t (&hi)[4], const uint32_t (&lo)[4]) {
      store_frag(rec + FRAG, block, lane, make_uint4(hi[0], hi[1], hi[2], hi[3]));
      store_frag(rec, block, lane, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      if (kBackward) {
        store_frag(rec + OFF_REST, block, lane, make_uint4(transposed(hi[0]), transposed(hi[2]), transposed(hi[1]), transposed(hi[3])));
        store_frag(rec + OFF_REST + 2 * FRAG, block, lane,
                   make_uint4(transposed(lo[0]), transposed(lo[2]), transposed(lo[1]), transposed(lo[3])));
      }
    };
    const int t0 = 16 * warp + g;          // this lane's rows: t0, t0 + 8
    const float gt[2] = {gs[t0], gs[t0 + 8]}, lt[2] = {gl[t0], gl[t0 + 8]};
    float* a16 = sm.a + 16 * warp * LA;
    float* td = sm.t + 16 * warp * LD + 16 * warp;
    // X diag(beta): into sm.a on the diagonal, kept as fragments (pairs of columns) below
    uint32_t bh[6][2], bl[6][2];           // tiles 0 .. 3 (warps 2, 3) and the block beside the diagonal (1, 3); rows g, g + 8
    auto block = [&](int jb, auto diagonal) {
      uint32_t w[4], wl[4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int tile = 2 * jb + half, j = 8 * tile + 2 * tig;
        const float2 gj = *reinterpret_cast<const float2*>(gs + j), lj = *reinterpret_cast<const float2*>(gl + j);
        const float2 bj = *reinterpret_cast<const float2*>(beta + j);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int t = t0 + 8 * r;
          float d0 = power2((gt[r] - gj.x) + (lt[r] - lj.x)), d1 = power2((gt[r] - gj.y) + (lt[r] - lj.y));
          float p0 = 0.f, p1 = 0.f;
          if constexpr (decltype(diagonal)::value) {
            if (!kBackward) {
              p0 = j < t ? d0 * qk[tile][2 * r] : j == t ? qk[tile][2 * r] : 0.f;
              p1 = j + 1 < t ? d1 * qk[tile][2 * r + 1] : j + 1 == t ? qk[tile][2 * r + 1] : 0.f;
            }
            *reinterpret_cast<float2*>(&a16[(g + 8 * r) * LA + 8 * half + 2 * tig]) =
                make_float2(j < t ? d0 * kk[tile][2 * r] * bj.x : 0.f, j + 1 < t ? d1 * kk[tile][2 * r + 1] * bj.y : 0.f);
          } else {
            if (!kBackward) {
              p0 = d0 * qk[tile][2 * r];
              p1 = d1 * qk[tile][2 * r + 1];
            }
            const int at = jb == warp - 1 && (warp & 1) ? 4 + half : tile & 3;
            split2(d0 * kk[tile][2 * r] * bj.x, d1 * kk[tile][2 * r + 1] * bj.y, bh[at][r], bl[at][r]);
          }
          if (!kBackward) split2(p0, p1, w[2 * r + half], wl[2 * r + half]);
        }
      }
      if (!kBackward) {
        store_frag(rec + OFF_REST, block_of(warp, jb), lane, make_uint4(w[0], w[1], w[2], w[3]));
        store_frag(rec + OFF_REST + FRAG, block_of(warp, jb), lane, make_uint4(wl[0], wl[1], wl[2], wl[3]));
      }
    };
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      if (jb < warp) block(jb, std::false_type{});
      if (jb == warp) block(jb, std::true_type{});
    }
    if (kBackward) {
      // P^T: row j = t0 (+ 8) of k.q, columns t from the diagonal block on
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        if (tb < warp) continue;
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int tile = 2 * tb + half, t = 8 * tile + 2 * tig;
          const float2 gi = *reinterpret_cast<const float2*>(gs + t), li = *reinterpret_cast<const float2*>(gl + t);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int j = t0 + 8 * r;
            const float d0 = power2((gi.x - gt[r]) + (li.x - lt[r])), d1 = power2((gi.y - gt[r]) + (li.y - lt[r]));
            const float q0 = qk[tile][2 * r], q1 = qk[tile][2 * r + 1];
            split2(t > j ? d0 * q0 : t == j ? q0 : 0.f, t + 1 > j ? d1 * q1 : t + 1 == j ? q1 : 0.f, ph[2 * r + half], pl[2 * r + half]);
          }
        }
        store_frag(rec + OFF_REST + FRAG, block_of(tb, warp), lane, make_uint4(ph[0], ph[1], ph[2], ph[3]));
        store_frag(rec + OFF_REST + 3 * FRAG, block_of(tb, warp), lane, make_uint4(pl[0], pl[1], pl[2], pl[3]));
      }
    }
    __syncwarp();
    // blocks of 16 on the diagonal, each by its warp: 8 x 8 blocks, a lane per column
    {
      if (lane < 16) {
        const int sub = 8 * (lane >> 3), col = lane & 7;
        const float* as = a16 + sub * LA + sub;
        float* ts = td + sub * LD + sub;
        float x[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const float4 r0 = *reinterpret_cast<const float4*>(as + t * LA), r1 = *reinterpret_cast<const float4*>(as + t * LA + 4);
          const float r[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
          float s = t == col ? 1.f : 0.f;
#pragma unroll
          for (int l = 0; l < t; ++l)
            if (l >= col) s = fmaf(-r[l], x[l], s);
          x[t] = t >= col ? s : 0.f;
          ts[t * LD + col] = x[t];
        }
      }
      __syncwarp();
      const int i = lane >> 2, j = 2 * (lane & 3);
      float y0 = 0.f, y1 = 0.f;
#pragma unroll
      for (int l = 0; l < 8; l += 4) {
        const float4 b = *reinterpret_cast<const float4*>(&a16[(8 + i) * LA + l]);
        const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 t = *reinterpret_cast<const float2*>(td + (l + e) * LD + j);
          y0 = fmaf(bb[e], t.x, y0);
          y1 = fmaf(bb[e], t.y, y1);
        }
      }
      // row i of Y is in lanes 4 i .. 4 i + 3
      float z0 = 0.f, z1 = 0.f;
#pragma unroll
      for (int l = 0; l < 8; ++l) {
        const float v0 = __shfl_sync(0xffffffffu, y0, 4 * l + (lane & 3)), v1 = __shfl_sync(0xffffffffu, y1, 4 * l + (lane & 3));
        const float b = -td[(8 + i) * LD + 8 + l];
        if (l <= i) {
          z0 = fmaf(b, v0, z0);
          z1 = fmaf(b, v1, z1);
        }
      }
      *reinterpret_cast<float2*>(td + (8 + i) * LD + j) = make_float2(z0, z1);
      *reinterpret_cast<float2*>(td + i * LD + 8 + j) = make_float2(0.f, 0.f);
    }
    __syncwarp();
    uint32_t dh[4], dl[4];                 // this warp's block of T on the diagonal, pairs of columns
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = g + 8 * (e >> 1), j = 2 * tig + 8 * (e & 1);
      const float2 x = *reinterpret_cast<const float2*>(&td[t * LD + j]);
      split2(j <= t ? x.x : 0.f, j + 1 <= t ? x.y : 0.f, dh[e], dl[e]);
    }
    store_t(block_of(warp, warp), dh, dl);
    __syncthreads();
    // A^-T of the block of 16 at `at` as an A fragment: pairs of rows l of a column j
    auto column_pairs = [&](const float* at, int lb, int jb, uint32_t (&ah)[4], uint32_t (&al)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 16 * jb + g + 8 * (e & 1), l = 16 * lb + 2 * tig + 8 * (e >> 1);
        split2(l >= j ? at[l * LD + j] : 0.f, l + 1 >= j ? at[(l + 1) * LD + j] : 0.f, ah[e], al[e]);
      }
    };
    float f[4][4];                         // a block of T under construction, tiles 0 .. 3
    if (warp & 1) {
      // pairs of blocks of 16: Y^T = A^-T B^T, then -C^-1 Y
      float y[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[nt][e] = 0.f;
      uint32_t ah[4], al[4], yh[2][2], yl[2][2];
      column_pairs(sm.t + 16 * (warp - 1) * LD + 16 * (warp - 1), 0, 0, ah, al);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        mma(y[nt], ah, bh[4][nt], bh[5][nt]);
        mma(y[nt], al, bh[4][nt], bh[5][nt]);
        mma(y[nt], ah, bl[4][nt], bl[5][nt]);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) split2(-y[nt][2 * r], -y[nt][2 * r + 1], yh[r][nt], yl[r][nt]);
      // (C^-1 as an A fragment: rows g, g + 8, then the columns from 8 on)
      const uint32_t ch[4] = {dh[0], dh[2], dh[1], dh[3]}, cl[4] = {dl[0], dl[2], dl[1], dl[3]};
      uint32_t h4[4], l4[4];
#pragma unroll
      for (int jt = 0; jt < 2; ++jt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[jt][e] = 0.f;
        mma(f[jt], ch, yh[jt][0], yh[jt][1]);
        mma(f[jt], cl, yh[jt][0], yh[jt][1]);
        mma(f[jt], ch, yl[jt][0], yl[jt][1]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          split2(f[jt][2 * r], f[jt][2 * r + 1], h4[2 * r + jt], l4[2 * r + jt]);
          *reinterpret_cast<float2*>(&sm.t[(t0 + 8 * r) * LD + 16 * (warp - 1) + 8 * jt + 2 * tig]) = make_float2(f[jt][2 * r], f[jt][2 * r + 1]);
        }
      }
      store_t(block_of(warp, warp - 1), h4, l4);
    }
    __syncthreads();
    if (warp >= 2) {
      // blocks of 32. Y^T = A^-T B^T: rows j, columns this warp's 16 rows i of B
      float y[2][2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[m][nt][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (m > ks) continue;            // T is zero above its diagonal: l < j
          uint32_t ah[4], al[4];
          column_pairs(sm.t, ks, m, ah, al);
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            mma(y[m][nt], ah, bh[2 * ks][nt], bh[2 * ks + 1][nt]);
            mma(y[m][nt], al, bh[2 * ks][nt], bh[2 * ks + 1][nt]);
            mma(y[m][nt], ah, bl[2 * ks][nt], bl[2 * ks + 1][nt]);
          }
        }
      // this warp's part of -C^-1 Y: block rows rb, its own 16 of the sum
      uint32_t yh[4][2], yl[4][2];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) split2(-y[m][nt][2 * r], -y[m][nt][2 * r + 1], yh[2 * m + r][nt], yl[2 * m + r][nt]);
      auto times = [&](const uint32_t (&ah)[4], const uint32_t (&al)[4], float (&o)[4][4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
          mma(o[j], ah, yh[j][0], yh[j][1]);
          mma(o[j], al, yh[j][0], yh[j][1]);
          mma(o[j], ah, yl[j][0], yl[j][1]);
        }
      };
      const uint32_t ch[4] = {dh[0], dh[2], dh[1], dh[3]}, cl[4] = {dl[0], dl[2], dl[1], dl[3]};
      times(ch, cl, f);                    // C^-1's block on the diagonal: this warp's rows
      if (warp == 2) {
        // its block below, for warp 3's rows
        float o[4][4];
        uint32_t ah[4], al[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = *reinterpret_cast<const float2*>(&sm.t[(48 + g + 8 * (e & 1)) * LD + 32 + 2 * tig + 8 * (e >> 1)]);
          split2(v.x, v.y, ah[e], al[e]);
        }
        times(ah, al, o);
#pragma unroll
        for (int j = 0; j < 4; ++j) sm.part[32 * j + lane] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
      }
      asm volatile("bar.sync 1, 64;" ::: "memory");
      if (warp == 3) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 o = sm.part[32 * j + lane];
          f[j][0] += o.x; f[j][1] += o.y; f[j][2] += o.z; f[j][3] += o.w;
        }
      }
#pragma unroll
      for (int jb = 0; jb < 2; ++jb) {
        uint32_t h4[4], l4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tile = 2 * jb + (e & 1), r = 2 * (e >> 1);
          split2(f[tile][r], f[tile][r + 1], h4[e], l4[e]);
        }
        store_t(block_of(warp, jb), h4, l4);
      }
    }
  }
}

template <int DK, bool kBackward>
cudaError_t launch(const PrepArgs& p, long long slots, cudaStream_t stream) {
  auto kern = gated_prep_kernel<DK, kBackward>;
  const int smem = (int)sizeof(PrepSmem<DK>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(slots * p.Hk), PT, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

cudaError_t gated_prep(const GatedArgs& a, uint8_t* records, int4* chunks) {
  const bool backward = chunks != nullptr;
  PrepArgs p{};
  p.q = (const __nv_bfloat16*)a.q; p.k = (const __nv_bfloat16*)a.k; p.g = a.g; p.beta = a.beta; p.offsets = a.offsets;
  p.rec = records; p.chunks = chunks; p.Hk = a.Hk; p.H = a.H; p.N = a.N; p.nseq = a.nseq; p.scale = a.scale;
  const long long slots = chunk_slots(a.B, a.N, a.nseq, a.offsets != nullptr, C);
  if (slots == 0) return cudaSuccess;
  if (a.dk == 64) return backward ? launch<64, true>(p, slots, a.stream) : launch<64, false>(p, slots, a.stream);
  return backward ? launch<128, true>(p, slots, a.stream) : launch<128, false>(p, slots, a.stream);
}

}  // namespace la
