// The forward chains of the gated delta rule by pairs of warps: as la_gated_chain.cu
// (formulas, precision: la_gated_mma.cuh) where each SM gets one CTA, or where one long
// sequence is what the others end up waiting for.
//
// A pair has 16 columns m of the state. The chain warp holds S^T [16 x DK], accumulators of
// m16n8k16 (rows m, columns dk). Per chunk of 64 tokens:
//   1. (K S)^T                   A = S^T from the registers, B = K's rows
//   2. R^T = V^T - e^G (K S)^T   V by ldmatrix.trans, laid out as the accumulator
//   3. E^T = R^T T^T             B = T's fragments;  U = beta E
//   4. S^T = e^{G_C} S^T + (e^{G_C-G} U)^T K
// and leaves S's and U's fragments in shared memory for its helper warp, which a
// chunk later does what the chain need not wait for:
//   5. O^T = scale e^G (Q S)^T + U^T P^T, the outputs
// and the copies of later chunks, by TMA (by cp.async, 26 a thread and chunk, a twelfth more). A CTA is four pairs of one head that share a chunk's
// K, Q and triangles; a pair's warps share a sub-core, whose tensor pipe has the helper's
// products while the chain warp goes from one product to the next. One barrier a chunk.
// Rows behind a sequence's last token are zeros in shared memory and have beta = 0.
//
// What bounds it: the tensor pipe has 2.0 of a chunk's 2.9 us at d = 128 (504 products of
// 16 x 8 x 16 a chunk and 16 columns, two warps to a sub-core), the rest is the chain warp's way
// from product to product. (A warp with 32 columns halves the reads of K, Q, T and P but has
// no second warp beside it, and was slower at every size.)
#include "la_gated_mma.cuh"

namespace la {

namespace {

using namespace gmma;

using sm100::mbar_init;
using sm100::fence_mbar_init;
using sm100::mbar_arrive_expect_tx;
using sm100::mbar_drain;
using sm100::tma_load_3d;

constexpr int W = 4;                                 // pairs of a CTA

template <int DK>
struct PairSmem {
  static constexpr int TB = C * DK * 2;              // a tile of K or Q
  // for the chain: K, the CTA's columns of V, [T lo | T hi | vec]
  static constexpr int V = TB;
  static constexpr int R = V + C * W * 32;
  static constexpr int VA = OFF_VEC;          // vec in it
  static constexpr int RA = VA + VEC;
  static constexpr int up(int x) { return (x + 1023) / 1024 * 1024; }   // (the swizzle goes by the address)
  static constexpr int A_BYTES = R + RA, A = up(A_BYTES);
  // for the helpers: Q, [vec | P hi | P lo]
  static constexpr int RB = VEC + 2 * FRAG;
  static constexpr int B_BYTES = TB + RB, B = up(B_BYTES);
  // from a chain warp to its helper, two chunks': S^T's fragments, high and low, U's
  static constexpr int SF = DK / 16 * 512;
  static constexpr int X = 2 * SF + 2 * 4 * 512;
  static constexpr int AT_B = 2 * A, AT_X = AT_B + 2 * B;
  static constexpr int BARS = AT_X + 2 * W * X;      // two barriers, a flag
  static constexpr int TOTAL = BARS + 64;
  static_assert(TOTAL <= 227 * 1024 && SF >= C * 32, "shared memory");
};

struct PairArgs {
  const uint8_t* rec;
  const float* S_in; float* S_out;
  const int* offsets;
  __nv_bfloat16* out;
  int Hk, H, N, dv, nseq, nblk;
  float scale;
  int* status;
  int stall;                             // for tests: 16 bytes more than come, so that the waits run out
};

// Maps of [heads][rows][DK], of [heads][rows][dv], in boxes of 64 columns and 64 rows
struct PairMaps { CUtensorMap q, k, v; };

template <int DK>
__global__ void __launch_bounds__(64 * W, 1)
gated_pair_kernel(const PairArgs p, const __grid_constant__ PairMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using L = PairSmem<DK>;
  constexpr int NT = 32 * W, KS = DK / 16;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & (W - 1);
  const bool helper = threadIdx.x >= NT;
  const int g = lane >> 2, tig = lane & 3, mi = lane >> 3, ml = lane & 7;
  long long block = blockIdx.x;
  const int blk = (int)(block % p.nblk);
  block /= p.nblk;
  const int h = (int)(block % p.H), s = sequence_of(p.offsets, (int)(block / p.H), p.nseq, p.N);
  const SeqRange sq = seq_range(p.offsets, s, p.N, C);
  const int n = sq.n, nchunks = (n + C - 1) / C;
  const int m0 = blk * 16 * W + warp * 16;           // this pair's first column
  const uint32_t base = smem_addr(smem);

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BARS);
  volatile int* gave_up = reinterpret_cast<volatile int*>(smem + L::BARS + 32);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) mbar_init(&bars[i], 1);
    *gave_up = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (helper) {
    const int tid = threadIdx.x - NT;
    const int kh = sq.b * p.Hk + h / (p.H / p.Hk), vh = sq.b * p.H + h;
    const long long vrow = (long long)vh * p.N + sq.lo;
    const uint8_t* rec = p.rec + ((long long)sq.slot * p.H + h) * REC_FWD;
    // One thread asks for copies, in turn i: chunk i + 1 for the chain, whose buffer chunk
    // i - 1 had, and chunk i for the helpers, who are at chunk i - 1. They have landed at
    // turn i + 1's barrier; turns take two barriers one after the other.
    auto load = [&](int i) {
      const bool a = i + 1 < nchunks, b = i >= 0 && i < nchunks;
      uint64_t* bar = &bars[(i + 1) & 1];
      mbar_arrive_expect_tx(bar, (a ? L::A_BYTES : 0) + (b ? L::B_BYTES : 0) + (p.stall && i == -1 ? 16 : 0));
      if (a) {
        const int c = i + 1, t0 = sq.lo + c * C, at = (c & 1) * L::A;
#pragma unroll
        for (int x = 0; x < DK / 64; ++x) tma_load_3d(smem + at + x * C * 128, &maps.k, bar, 64 * x, t0, kh);
        tma_load_3d(smem + at + L::V, &maps.v, bar, blk * 16 * W, t0, vh);
        bulk_load(base + at + L::R, rec + (long long)c * p.H * REC_FWD, L::RA, bar);
      }
      if (b) {
        const int t0 = sq.lo + i * C, at = L::AT_B + (i & 1) * L::B;
#pragma unroll
        for (int x = 0; x < DK / 64; ++x) tma_load_3d(smem + at + x * C * 128, &maps.q, bar, 64 * x, t0, kh);
        bulk_load(base + at + L::TB, rec + (long long)i * p.H * REC_FWD + OFF_VEC, L::RB, bar);
      }
    };
    // Copies have whole boxes: rows behind the sequence's last token become zeros.
    auto clear = [&](int at, int boxes) {
      for (int x = 0; x < boxes; ++x)
        for (int j = tid; j < (C - n % C) * 8; j += NT)
          *reinterpret_cast<uint4*>(smem + at + x * C * 128 + n % C * 128 + j * 16) = make_uint4(0u, 0u, 0u, 0u);
    };
    bool ok = true;                                  // (once a wait gave up, none is begun and no copy asked for)
    int late = 0;
    if (tid == 0) load(-1);
    __nv_bfloat16* ob = p.out + vrow * p.dv + m0;
    for (int i = 0; i <= nchunks; ++i) {
      if (ok) {
        ok = mbar_drain(&bars[i & 1], (i >> 1) & 1, kWaitNs);
        late = i;
        if (!ok) *gave_up = 1;
      }
      if (n % C != 0 && i == nchunks - 1) clear((i & 1) * L::A, DK / 64 + 1);        // K and V
      if (n % C != 0 && i == nchunks) clear(L::AT_B + ((i - 1) & 1) * L::B, DK / 64);
      __syncthreads();                               // chunk i's copies are there, chunk i - 1's chain is done
      if (tid == 0 && ok) load(i);
      if (i == 0) continue;
      const int c = i - 1, t0 = c * C, cn = min(C, n - t0);
      const uint32_t sb = base + L::AT_B + (c & 1) * L::B;
      const uint8_t* rp = smem + L::AT_B + (c & 1) * L::B + L::TB;
      const float* EG = reinterpret_cast<const float*>(rp);
      uint8_t* xp = smem + L::AT_X + ((c & 1) * W + warp) * L::X;
      auto pfrag = [&](int lo, int b) { return *reinterpret_cast<const uint4*>(rp + VEC + lo * FRAG + b * 512 + lane * 16); };
      auto product = [&](float (&y)[8][4]) {         // (Q S)^T
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[j][e] = 0.f;
        uint4 a[2], d[2];                            // high and low parts
        uint32_t b[2][4][4];
        auto ask = [&](int ks) {
          a[ks & 1] = *reinterpret_cast<const uint4*>(xp + ks * 512 + lane * 16);
          d[ks & 1] = *reinterpret_cast<const uint4*>(xp + L::SF + ks * 512 + lane * 16);
#pragma unroll
          for (int t = 0; t < 4; ++t)
            ldmatrix4(b[ks & 1][t], sb + box_at(16 * t + ((mi >> 1) << 3) + ml, 2 * ks + (mi & 1)));
        };
        ask(0);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          if (ks + 1 < KS) ask(ks + 1);
          const uint32_t w[4] = {a[ks & 1].x, a[ks & 1].y, a[ks & 1].z, a[ks & 1].w};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            mma(y[2 * t], w, b[ks & 1][t][0], b[ks & 1][t][1]);
            mma(y[2 * t + 1], w, b[ks & 1][t][2], b[ks & 1][t][3]);
          }
          const uint32_t wl[4] = {d[ks & 1].x, d[ks & 1].y, d[ks & 1].z, d[ks & 1].w};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            mma(y[2 * t], wl, b[ks & 1][t][0], b[ks & 1][t][1]);
            mma(y[2 * t + 1], wl, b[ks & 1][t][2], b[ks & 1][t][3]);
          }
        }
      };
      float y[8][4];
      product(y);
      uint4 pf[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) pf[b] = pfrag(0, b);
      uint32_t u[4][4], ul[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint4 w = *reinterpret_cast<const uint4*>(xp + 2 * L::SF + t * 512 + lane * 16);
        const uint4 l = *reinterpret_cast<const uint4*>(xp + 2 * L::SF + 2048 + t * 512 + lane * 16);
        u[t][0] = w.x; u[t][1] = w.y; u[t][2] = w.z; u[t][3] = w.w;
        ul[t][0] = l.x; ul[t][1] = l.y; ul[t][2] = l.z; ul[t][3] = l.w;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 eg = *reinterpret_cast<const float2*>(EG + 8 * j + 2 * tig);
        y[j][0] *= p.scale * eg.x; y[j][1] *= p.scale * eg.y;
        y[j][2] *= p.scale * eg.x; y[j][3] *= p.scale * eg.y;
      }
#pragma unroll
      for (int jb = 0; jb < 4; ++jb)
#pragma unroll
        for (int tb = jb; tb < 4; ++tb) {
          const uint4 w = pf[block_of(tb, jb)], wl = pfrag(1, block_of(tb, jb));
          mma(y[2 * tb], u[jb], w.x, w.y);
          mma(y[2 * tb + 1], u[jb], w.z, w.w);
          mma(y[2 * tb], ul[jb], w.x, w.y);
          mma(y[2 * tb + 1], ul[jb], w.z, w.w);
          mma(y[2 * tb], u[jb], wl.x, wl.y);
          mma(y[2 * tb + 1], u[jb], wl.z, wl.w);
        }
      // A zero weight of a later token's row that is not finite would be NaN
      // for the tokens before it: such a chunk is done again, each token
      // with the rows behind it left out.
      if (__any_sync(0xffffffffu, not_finite(y))) {
        float qs[8][4];
        product(qs);
#pragma unroll 1
        for (int t = 0; t < cn; ++t) {
          const int tb = t >> 4;
          float o2[2][4];
          const float f = p.scale * EG[t];
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((j >> 1) == tb) o2[j & 1][e] = qs[j][e] * f;
#pragma unroll
          for (int jb = 0; jb < 4; ++jb) {
            if (jb > tb) continue;
            uint32_t a[4], b[4];
            rows_to(a, u[jb], jb, t, tig);
            rows_to(b, ul[jb], jb, t, tig);
            const uint4 w = pfrag(0, block_of(tb, jb)), wl = pfrag(1, block_of(tb, jb));
            mma(o2[0], a, w.x, w.y);
            mma(o2[1], a, w.z, w.w);
            mma(o2[0], b, w.x, w.y);
            mma(o2[1], b, w.z, w.w);
            mma(o2[0], a, wl.x, wl.y);
            mma(o2[1], a, wl.z, wl.w);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (8 * j + 2 * tig + (e & 1) == t) y[j][e] = o2[j & 1][e];
        }
      }
      // rows [token][16 columns] over S's fragments, then 16 bytes a lane
      __syncwarp();
      const uint32_t xa = smem_addr(xp);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        stmatrix4t(xa + tile_at<2>(16 * t + ((mi >> 1) << 3) + ml, mi & 1), pack2(y[2 * t][0], y[2 * t][1]),
                   pack2(y[2 * t][2], y[2 * t][3]), pack2(y[2 * t + 1][0], y[2 * t + 1][1]),
                   pack2(y[2 * t + 1][2], y[2 * t + 1][3]));
      __syncwarp();
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * r + (lane >> 1), half = lane & 1;
        if (t < cn && ok)
          *reinterpret_cast<uint4*>(ob + (long long)(t0 + t) * p.dv + 8 * half) =
              *reinterpret_cast<const uint4*>(xp + tile_at<2>(t, half));
      }
    }
    if (!ok) {
      mbar_drain(&bars[late & 1], (late >> 1) & 1, kWaitNs / 8);
      atomicExch(p.status, (int)LA_ERR_TIMEOUT);      // (any thread's: one may give up where the others just did not)
    }
    return;
  }

  float st[2 * KS][4];                               // S^T: tile j has dk 8j ..
  {
    const float* src = p.S_in == nullptr ? nullptr : p.S_in + ((long long)s * p.H + h) * DK * p.dv + m0 + g;
#pragma unroll
    for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        st[j][e] = src == nullptr ? 0.f : src[(long long)(8 * j + 2 * tig + (e & 1)) * p.dv + 8 * (e >> 1)];
  }
  __syncthreads();
  for (int i = 0; i < nchunks; ++i) {
    const int cn = min(C, n - i * C);
    const uint32_t sb = base + (i & 1) * L::A;
    const uint8_t* rp = smem + (i & 1) * L::A + L::R;
    const float* EG = reinterpret_cast<const float*>(rp + L::VA);
    const float* EC = EG + C;
    const float* BT = EG + 2 * C;
    uint8_t* xp = smem + L::AT_X + ((i & 1) * W + warp) * L::X;
    auto tfrag = [&](bool low, int b) {
      return *reinterpret_cast<const uint4*>(rp + (low ? 0 : FRAG) + b * 512 + lane * 16);
    };
    // 1. (K S)^T (fragments are asked for ahead of the stores, which no load may pass)
    float x[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[j][e] = 0.f;
    uint32_t kb[2][4][4], v[4][4];
    auto ask = [&](int ks) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        ldmatrix4(kb[ks & 1][t], sb + box_at(16 * t + ((mi >> 1) << 3) + ml, 2 * ks + (mi & 1)));
    };
    ask(0);
#pragma unroll
    for (int t = 0; t < 4; ++t) ldmatrix4t(v[t], sb + L::V + box_at(16 * t + ((mi >> 1) << 3) + ml, 2 * warp + (mi & 1)));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (ks + 1 < KS) ask(ks + 1);
      uint32_t ah[4], al[4];
      split2(st[2 * ks][0], st[2 * ks][1], ah[0], al[0]);
      split2(st[2 * ks][2], st[2 * ks][3], ah[1], al[1]);
      split2(st[2 * ks + 1][0], st[2 * ks + 1][1], ah[2], al[2]);
      split2(st[2 * ks + 1][2], st[2 * ks + 1][3], ah[3], al[3]);
      *reinterpret_cast<uint4*>(xp + ks * 512 + lane * 16) = make_uint4(ah[0], ah[1], ah[2], ah[3]);
      *reinterpret_cast<uint4*>(xp + L::SF + ks * 512 + lane * 16) = make_uint4(al[0], al[1], al[2], al[3]);
      const uint32_t (&b)[4][4] = kb[ks & 1];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        mma(x[2 * t], ah, b[t][0], b[t][1]);
        mma(x[2 * t + 1], ah, b[t][2], b[t][3]);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        mma(x[2 * t], al, b[t][0], b[t][1]);
        mma(x[2 * t + 1], al, b[t][2], b[t][3]);
      }
    }
    const float last = EG[C - 1];
    // 2. R^T, split
    uint32_t rh[4][4], rl[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {                  // e: A fragment a0 .. a3 = (tile 2t + e / 2, rows 8 (e % 2))
        const int j = 2 * t + (e >> 1), r = 2 * (e & 1);
        const float2 eg = *reinterpret_cast<const float2*>(EG + 8 * j + 2 * tig);
        split2(low_half(v[t][e]) - eg.x * x[j][r], high_half(v[t][e]) - eg.y * x[j][r + 1], rh[t][e], rl[t][e]);
      }
    }
    // 3. E^T
    float ev[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) ev[j][e] = 0.f;
#pragma unroll
    for (int jb = 0; jb < 4; ++jb)                   // (this way round neighbouring products are of different sums)
#pragma unroll
      for (int tb = jb; tb < 4; ++tb) {
        const uint4 th = tfrag(false, block_of(tb, jb));
        mma(ev[2 * tb], rh[jb], th.x, th.y);
        mma(ev[2 * tb + 1], rh[jb], th.z, th.w);
        const uint4 tl = tfrag(true, block_of(tb, jb));
        mma(ev[2 * tb], rl[jb], th.x, th.y);
        mma(ev[2 * tb + 1], rl[jb], th.z, th.w);
        mma(ev[2 * tb], rh[jb], tl.x, tl.y);
        mma(ev[2 * tb + 1], rh[jb], tl.z, tl.w);
      }
    if (__any_sync(0xffffffffu, not_finite(ev))) {   // as the outputs: no row reaches those before it
#pragma unroll 1
      for (int t = 0; t < cn; ++t) {
        const int tb = t >> 4;
        float e2[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
          if (jb > tb) continue;
          uint32_t a[4], b[4];
          rows_to(a, rh[jb], jb, t, tig);
          rows_to(b, rl[jb], jb, t, tig);
          const uint4 th = tfrag(false, block_of(tb, jb));
          mma(e2[0], a, th.x, th.y); mma(e2[1], a, th.z, th.w);
          const uint4 tl = tfrag(true, block_of(tb, jb));
          mma(e2[0], b, th.x, th.y); mma(e2[1], b, th.z, th.w);
          mma(e2[0], a, tl.x, tl.y); mma(e2[1], a, tl.z, tl.w);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * j + 2 * tig + (e & 1) == t) ev[j][e] = e2[j & 1][e];
      }
    }
    // U for the outputs, e^{G_C-G} U for the state
    uint32_t kt[2][KS][4];
    auto ask_t = [&](int t) {
#pragma unroll
      for (int k2 = 0; k2 < KS; ++k2)
        ldmatrix4t(kt[t & 1][k2], sb + box_at(16 * t + ((mi & 1) << 3) + ml, 2 * k2 + (mi >> 1)));
    };
    ask_t(0);
    uint32_t uh[4][4], ul[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t u[4], u2[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 2 * t + (e >> 1), r = 2 * (e & 1);
        const float2 b = *reinterpret_cast<const float2*>(BT + 8 * j + 2 * tig);
        const float2 ec = *reinterpret_cast<const float2*>(EC + 8 * j + 2 * tig);
        split2(b.x * ev[j][r], b.y * ev[j][r + 1], u[e], u2[e]);
        split2(b.x * ec.x * ev[j][r], b.y * ec.y * ev[j][r + 1], uh[t][e], ul[t][e]);
      }
      *reinterpret_cast<uint4*>(xp + 2 * L::SF + t * 512 + lane * 16) = make_uint4(u[0], u[1], u[2], u[3]);
      *reinterpret_cast<uint4*>(xp + 2 * L::SF + 2048 + t * 512 + lane * 16) = make_uint4(u2[0], u2[1], u2[2], u2[3]);
    }
    // 4. S^T
#pragma unroll
    for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) st[j][e] *= last;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t < 3) ask_t(t + 1);
#pragma unroll
      for (int k2 = 0; k2 < KS; ++k2) {
        mma(st[2 * k2], uh[t], kt[t & 1][k2][0], kt[t & 1][k2][1]);
        mma(st[2 * k2 + 1], uh[t], kt[t & 1][k2][2], kt[t & 1][k2][3]);
      }
#pragma unroll
      for (int k2 = 0; k2 < KS; ++k2) {
        mma(st[2 * k2], ul[t], kt[t & 1][k2][0], kt[t & 1][k2][1]);
        mma(st[2 * k2 + 1], ul[t], kt[t & 1][k2][2], kt[t & 1][k2][3]);
      }
    }
    __syncthreads();                                 // the helper has this chunk, the next one's copies are there
  }
  if (p.S_out != nullptr && !*gave_up) {
    float* dst = p.S_out + ((long long)s * p.H + h) * DK * p.dv + m0 + g;
#pragma unroll
    for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[(long long)(8 * j + 2 * tig + (e & 1)) * p.dv + 8 * (e >> 1)] = st[j][e];
  }
}

template <int DK>
cudaError_t launch(PairArgs p, const PairMaps& maps, cudaStream_t stream) {
  const long long grid = (long long)p.nseq * p.H * p.nblk;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto kern = gated_pair_kernel<DK>;
  const int smem = PairSmem<DK>::TOTAL;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)grid, 64 * W, smem, stream>>>(p, maps);
  e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

// d = 128: 64 heads of 4096 tokens (128 CTAs) 189 us against 352 by one warp for 16 columns;
// 80 heads (160) 373 against 354, 256 heads of 2048 (512) 376 against 355; d = 64, 1024
// heads of 1024: 239 against 214. Packed, 16384 rows, 32 heads: of twelve unlike sequences
// 342 against 356, of 40 like ones 428 against 399.
bool gated_pair_wanted(const GatedArgs& a) {
  return a.offsets != nullptr || (long long)a.nseq * a.H * (a.dv / (16 * W)) <= kSlots;
}

cudaError_t gated_pair_forward(const GatedArgs& a, const uint8_t* records) {
  PairArgs p{};
  PairMaps maps;
  const long long keys = (long long)a.B * a.Hk, heads = (long long)a.B * a.H;
  if (!gated_map(&maps.q, a.q, keys, a.N, a.dk, 64) || !gated_map(&maps.k, a.k, keys, a.N, a.dk, 64) ||
      !gated_map(&maps.v, a.v, heads, a.N, a.dv, 64))
    return cudaErrorInvalidValue;
  p.status = device_status_ptr();
  if (p.status == nullptr) return cudaErrorNotReady;
  p.stall = take_gated_timeout_test(0) ? 1 : 0;
  p.rec = records; p.offsets = a.offsets; p.S_in = a.S0; p.S_out = a.S_final; p.out = (__nv_bfloat16*)a.out;
  p.Hk = a.Hk; p.H = a.H; p.N = a.N; p.dv = a.dv; p.nseq = a.nseq; p.nblk = a.dv / (16 * W); p.scale = a.scale;
  return a.dk == 64 ? launch<64>(p, maps, a.stream) : launch<128>(p, maps, a.stream);
}

}  // namespace la
