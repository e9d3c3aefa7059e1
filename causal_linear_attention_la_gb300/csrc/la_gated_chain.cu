// The chains of the gated delta rule on the tensor cores: chunk after chunk of
// one head, the state in registers (formulas, precision and why mma.sync:
// la_gated_mma.cuh).
//
// A warp has 16 columns m of the state as S^T [16 x DK], accumulators of m16n8k16
// (rows m, columns dk). Per chunk of 64 tokens:
//   1. (K S)^T and (Q S)^T       A = S^T from the registers, split; B = K, Q rows
//   2. R^T = V^T - e^G (K S)^T   V by ldmatrix.trans, laid out as the accumulator
//   3. E^T = R^T T^T             A = R^T split, B = T's fragments
//   4. O^T = scale e^G (Q S)^T + U^T P^T
//   5. S^T = e^{G_C} S^T + (e^{G_C-G} U)^T K
// Rows behind a sequence's last token are zeros in shared memory and have beta = 0.
// A forward CTA is eight warps of one head (four, where two CTAs fit an SM or dv is 64), which
// share the chunk's K, Q and triangles in two buffers, the next chunk's copies in flight during
// a chunk (d = 128, 256 heads of 2048 tokens: 355 us by eight warps, 403 by four; dk = 64, dv =
// 128, 256 heads of 1024: 135 by eight, 126 by four). A backward CTA has four warps of each
// chain (64 heads of 4096 tokens: 394 us, by eight warps of one or the other 452; 128 heads of
// 1024 of dk = 128, dv = 64: 101, by four of one or the other 126).
// Bound: the latency of a warp's way from product to product, two warps to a sub-core; the
// tensor pipe has 73 % of the forward's time (504 products of 16 x 8 x 16 a chunk and 16 columns
// of d = 128) and 52 % of the backward's (800).
#include "la_gated_mma.cuh"

namespace la {

namespace {

using namespace gmma;

using sm100::mbar_init;
using sm100::fence_mbar_init;
using sm100::mbar_arrive_expect_tx;
using sm100::mbar_drain;
using sm100::tma_load_3d;

enum { kFwd = 0, kSave = 1, kRev = 2 };
// W: warps of a CTA
template <int DK, int MODE, int W>
struct ChainSmem {
  static constexpr int KB = C * DK * 2;             // a tile of K or Q
  static constexpr int VB = C * W * 32;             // the CTA's columns of V or dO
  // the part of the record that is wanted: all, [T lo | T hi | vec],
  // [vec | T^T hi | P^T hi | T^T lo | P^T lo]
  static constexpr int FROM = MODE == kRev ? OFF_VEC : 0;
  static constexpr int RB = (MODE == kFwd ? REC_FWD : MODE == kSave ? OFF_REST : OFF_SUMS) - FROM;
  static constexpr int RV = OFF_VEC - FROM;          // vec in it
  __host__ __device__ static constexpr int tri(int i) {   // T hi, T lo, P hi, P lo (reverse: T^T, P^T)
    return MODE == kRev ? VEC + (i == 1 ? 2 : i == 2 ? 1 : i) * FRAG
                        : i == 0 ? FRAG : i == 1 ? 0 : RV + VEC + (i - 2) * FRAG;
  }
  static constexpr int K = 0;
  static constexpr int Q = K + KB;
  static constexpr int V = Q + (MODE == kSave ? 0 : KB);
  static constexpr int R = V + VB;
  static constexpr int BYTES = R + RB;
  static constexpr int STAGE = (BYTES + 1023) / 1024 * 1024;            // (the swizzle goes by the address)
  static constexpr int OUT = 2 * STAGE;             // a warp's rows on their way out
  static constexpr int BARS = OUT + W * C * 32;     // two barriers, a flag
  static constexpr int TOTAL = BARS + 64;
};

struct ChainArgs {
  const void* v;                         // dO in reverse
  const uint8_t* rec; int rec_bytes;
  const float* S_in; float* S_out;
  const int* offsets;
  __nv_bfloat16* out;                    // O, E or dR rows [B,H,N,dv]
  __nv_bfloat16* out_lo;                 // E, dR: what that leaves out
  __nv_bfloat16* states;                 // [slot,H,dv,DK]: before each chunk (save), behind it (reverse)
  __nv_bfloat16* states_lo;              // what that leaves out
  int Hk, H, N, dv, nseq, nblk;
  float scale;
  int* status;
  int stall;                             // for tests: 16 bytes more than come, so that the waits run out
};

// Maps of [heads][rows][DK], of [heads][rows][dv], in boxes of 64 columns and 64 rows
struct ChainMaps { CUtensorMap q, k, v; };

template <int DK, int MODE, int W>
__device__ __forceinline__ void chain(const ChainArgs& p, const ChainMaps& maps, long long block, uint8_t* smem) {
  using L = ChainSmem<DK, MODE, W>;
  constexpr int NT = 32 * W, KS = DK / 16;
  const int tid = MODE == kFwd ? threadIdx.x : threadIdx.x % NT, lane = tid & 31, warp = tid >> 5;
  auto sync = [] {                                   // of the chain's warps
    if constexpr (MODE == kFwd) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"n"(MODE), "n"(NT) : "memory");
  };
  const int g = lane >> 2, tig = lane & 3, mi = lane >> 3, ml = lane & 7;
  const int blk = (int)(block % p.nblk);
  block /= p.nblk;
  const int h = (int)(block % p.H), s = sequence_of(p.offsets, (int)(block / p.H), p.nseq, p.N);
  const SeqRange sq = seq_range(p.offsets, s, p.N, C);
  const int n = sq.n, nchunks = (n + C - 1) / C;
  const int kh = sq.b * p.Hk + h / (p.H / p.Hk), vh = sq.b * p.H + h;
  const long long vrow = (long long)vh * p.N + sq.lo;
  const int m0 = blk * 16 * W + warp * 16;           // this warp's first column
  __nv_bfloat16* ob = p.out + vrow * p.dv + m0;
  __nv_bfloat16* ol = MODE == kFwd ? nullptr : p.out_lo + vrow * p.dv + m0;
  const uint32_t base = smem_addr(smem);
  uint8_t* rows = smem + L::OUT + warp * C * 32;
  const uint32_t rows_at = base + L::OUT + warp * C * 32;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BARS);
  volatile int* gave_up = reinterpret_cast<volatile int*>(smem + L::BARS + 32);
  if (tid == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    *gave_up = 0;
    fence_mbar_init();
  }

  auto chunk_of = [&](int i) { return MODE == kRev ? nchunks - 1 - i : i; };
  auto load = [&](int i) {                           // one thread's
    const int c = chunk_of(i), t0 = sq.lo + c * C;
    uint8_t* to = smem + (i & 1) * L::STAGE;
    uint64_t* bar = &bars[i & 1];
    mbar_arrive_expect_tx(bar, L::BYTES + (p.stall && i == 0 ? 16 : 0));
#pragma unroll
    for (int x = 0; x < DK / 64; ++x) {
      tma_load_3d(to + L::K + x * C * 128, &maps.k, bar, 64 * x, t0, kh);
      if (MODE != kSave) tma_load_3d(to + L::Q + x * C * 128, &maps.q, bar, 64 * x, t0, kh);
    }
#pragma unroll
    for (int x = 0; x < W / 4; ++x) tma_load_3d(to + L::V + x * C * 128, &maps.v, bar, blk * 16 * W + 64 * x, t0, vh);
    bulk_load(smem_addr(to) + L::R, p.rec + ((long long)(sq.slot + c) * p.H + h) * p.rec_bytes + L::FROM, L::RB, bar);
  };
  if (tid == 0 && nchunks > 0) load(0);

  float st[2 * KS][4];                               // S^T: tile j has dk 8j ..
  {
    const float* src = p.S_in == nullptr ? nullptr : p.S_in + ((long long)s * p.H + h) * DK * p.dv + m0 + g;
#pragma unroll
    for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        st[j][e] = src == nullptr ? 0.f : src[(long long)(8 * j + 2 * tig + (e & 1)) * p.dv + 8 * (e >> 1)];
  }

  // rows [token][16 columns] by way of this warp's part of shared memory, 16 bytes a lane:
  // rounded, and (backward) what that leaves out
  auto rows_out = [&](const float (&x)[8][4], int t0, int cn) {
#pragma unroll
    for (int part = 0; part < (MODE == kFwd ? 1 : 2); ++part) {
      __nv_bfloat16* to = part == 0 ? ob : ol;
      __syncwarp();
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t w[2][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2_out(x[2 * t + (e >> 1)][2 * (e & 1)], x[2 * t + (e >> 1)][2 * (e & 1) + 1], w[0][e], w[1][e]);
        stmatrix4t(rows_at + tile_at<2>(16 * t + ((mi >> 1) << 3) + ml, mi & 1), w[part][0], w[part][1], w[part][2], w[part][3]);
      }
      __syncwarp();
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * r + (lane >> 1), half = lane & 1;
        if (t < cn)
          *reinterpret_cast<uint4*>(to + (long long)(t0 + t) * p.dv + 8 * half) =
              *reinterpret_cast<const uint4*>(rows + tile_at<2>(t, half));
      }
    }
  };

  for (int i = 0; i < nchunks; ++i) {
    const int c = chunk_of(i), t0 = c * C, cn = min(C, n - t0);
    if (i == 0) sync();                              // the barriers are there
    if (!mbar_drain(&bars[i & 1], (i >> 1) & 1, kWaitNs)) *gave_up = 1;
    if (cn < C) {                                    // copies have whole boxes: rows behind the last become zeros
      uint8_t* to = smem + (i & 1) * L::STAGE;
      for (int x = 0; x < L::R / (C * 128); ++x)
        for (int j = tid; j < (C - cn) * 8; j += NT)
          *reinterpret_cast<uint4*>(to + x * C * 128 + cn * 128 + j * 16) = make_uint4(0u, 0u, 0u, 0u);
      sm100::fence_proxy_async_smem();               // (copies come here again)
    }
    sync();                                          // the copies are there; the other buffer's readers are done
    if (*gave_up) {
      mbar_drain(&bars[i & 1], (i >> 1) & 1, kWaitNs / 8);
      if (tid == 0) atomicExch(p.status, (int)LA_ERR_TIMEOUT);
      return;
    }
    if (tid == 0 && i + 1 < nchunks) load(i + 1);
    const uint32_t sb = base + (i & 1) * L::STAGE;
    const uint8_t* rp = smem + (i & 1) * L::STAGE + L::R;
    const float* vec = reinterpret_cast<const float*>(rp + L::RV);
    const float* EG = vec;
    const float* EC = vec + C;
    const float* BT = vec + 2 * C;
    auto frag = [&](int tri, int b) {                // block b of triangle `tri` of this mode's record
      return *reinterpret_cast<const uint4*>(rp + L::tri(tri) + b * 512 + lane * 16);
    };

    // the state as bf16 rows [dv][DK]: two lanes join 8 bytes of neighbouring tiles
    const long long at = MODE == kFwd ? 0 : (((long long)(sq.slot + c) * p.H + h) * p.dv + m0) * DK;
    const bool odd = tig & 1;
    auto join = [&](__nv_bfloat16* dst, int j, int r, uint32_t a, uint32_t b) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
      const uint2 w = odd ? make_uint2(got, b) : make_uint2(a, got);
      *reinterpret_cast<uint2*>(dst + at + (long long)(g + 8 * r) * DK + 8 * (j + odd) + 4 * (tig >> 1)) = w;
    };

    // 1. (K S)^T, and in the forward (Q S)^T
    float x[8][4], y[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[j][e] = y[j][e] = 0.f;
    uint32_t kb[2][4][4];
    auto ask = [&](int ks) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        ldmatrix4(kb[ks & 1][t], sb + L::K + box_at(16 * t + ((mi >> 1) << 3) + ml, 2 * ks + (mi & 1)));
    };
    ask(0);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t ah[4], al[4];
      split2(st[2 * ks][0], st[2 * ks][1], ah[0], al[0]);
      split2(st[2 * ks][2], st[2 * ks][3], ah[1], al[1]);
      split2(st[2 * ks + 1][0], st[2 * ks + 1][1], ah[2], al[2]);
      split2(st[2 * ks + 1][2], st[2 * ks + 1][3], ah[3], al[3]);
      const uint32_t (&b)[4][4] = kb[ks & 1];
      uint32_t bq[4][4];
      if (MODE == kFwd) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
          ldmatrix4(bq[t], sb + L::Q + box_at(16 * t + ((mi >> 1) << 3) + ml, 2 * ks + (mi & 1)));
      }
      if (ks + 1 < KS) ask(ks + 1);
      if (MODE != kFwd) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          join(p.states, 2 * ks, r, ah[r], ah[2 + r]);
          join(p.states_lo, 2 * ks, r, al[r], al[2 + r]);
        }
      }
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
      if (MODE == kFwd) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          mma(y[2 * t], ah, bq[t][0], bq[t][1]);
          mma(y[2 * t + 1], ah, bq[t][2], bq[t][3]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          mma(y[2 * t], al, bq[t][0], bq[t][1]);
          mma(y[2 * t + 1], al, bq[t][2], bq[t][3]);
        }
      }
    }

    const float last = EG[C - 1];
    if (MODE != kRev) {
      // 2. R^T, split
      uint32_t rh[4][4], rl[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t v[4];
        ldmatrix4t(v, sb + L::V + box_at(16 * t + ((mi >> 1) << 3) + ml, 2 * warp + (mi & 1)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {                // e: A fragment a0 .. a3 = (tile 2t + e / 2, rows 8 (e % 2))
          const int j = 2 * t + (e >> 1), r = 2 * (e & 1);
          const float2 eg = *reinterpret_cast<const float2*>(EG + 8 * j + 2 * tig);
          split2(low_half(v[e]) - eg.x * x[j][r], high_half(v[e]) - eg.y * x[j][r + 1], rh[t][e], rl[t][e]);
        }
      }
      // 3. E^T
      float ev[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) ev[j][e] = 0.f;
#pragma unroll
      for (int jb = 0; jb < 4; ++jb)                 // (this way round neighbouring products are of different sums)
#pragma unroll
        for (int tb = jb; tb < 4; ++tb) {
          const uint4 th = frag(0, block_of(tb, jb));
          mma(ev[2 * tb], rh[jb], th.x, th.y);
          mma(ev[2 * tb + 1], rh[jb], th.z, th.w);
          const uint4 tl = frag(1, block_of(tb, jb));
          mma(ev[2 * tb], rl[jb], th.x, th.y);
          mma(ev[2 * tb + 1], rl[jb], th.z, th.w);
          mma(ev[2 * tb], rh[jb], tl.x, tl.y);
          mma(ev[2 * tb + 1], rh[jb], tl.z, tl.w);
        }
      // 4. U and the outputs
      uint32_t u[4][4], ul[4][4];
      if (MODE == kFwd) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 b = *reinterpret_cast<const float2*>(BT + 8 * j + 2 * tig);
          const float2 eg = *reinterpret_cast<const float2*>(EG + 8 * j + 2 * tig);
          split2(b.x * ev[j][0], b.y * ev[j][1], u[j >> 1][2 * (j & 1)], ul[j >> 1][2 * (j & 1)]);
          split2(b.x * ev[j][2], b.y * ev[j][3], u[j >> 1][2 * (j & 1) + 1], ul[j >> 1][2 * (j & 1) + 1]);
          y[j][0] *= p.scale * eg.x; y[j][1] *= p.scale * eg.y;
          y[j][2] *= p.scale * eg.x; y[j][3] *= p.scale * eg.y;
        }
#pragma unroll
        for (int jb = 0; jb < 4; ++jb)
#pragma unroll
          for (int tb = jb; tb < 4; ++tb) {
            const uint4 w = frag(2, block_of(tb, jb)), wl = frag(3, block_of(tb, jb));
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
        float bad = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) bad = fmaf(0.f, ev[j][e], fmaf(0.f, y[j][e], bad));
        if (__any_sync(0xffffffffu, bad != 0.f)) {
#pragma unroll 1
          for (int t = 0; t < cn; ++t) {
            const int tb = t >> 4;
            float e2[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int jb = 0; jb < 4; ++jb) {
              if (jb > tb) continue;
              uint32_t a[4], b[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int j = 16 * jb + 8 * (e >> 1) + 2 * tig;
                const uint32_t keep = (j <= t ? 0xffffu : 0u) | (j + 1 <= t ? 0xffff0000u : 0u);
                a[e] = rh[jb][e] & keep;
                b[e] = rl[jb][e] & keep;
              }
              const uint4 th = frag(0, block_of(tb, jb));
              mma(e2[0], a, th.x, th.y); mma(e2[1], a, th.z, th.w);
              const uint4 tl = frag(1, block_of(tb, jb));
              mma(e2[0], b, th.x, th.y); mma(e2[1], b, th.z, th.w);
              mma(e2[0], a, tl.x, tl.y); mma(e2[1], a, tl.z, tl.w);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (8 * j + 2 * tig + (e & 1) == t) ev[j][e] = e2[j & 1][e];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 b = *reinterpret_cast<const float2*>(BT + 8 * j + 2 * tig);
            split2(b.x * ev[j][0], b.y * ev[j][1], u[j >> 1][2 * (j & 1)], ul[j >> 1][2 * (j & 1)]);
            split2(b.x * ev[j][2], b.y * ev[j][3], u[j >> 1][2 * (j & 1) + 1], ul[j >> 1][2 * (j & 1) + 1]);
          }
          // (Q S)^T again: a product of the state's columns with one query's row
          float qs[8][4];
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) qs[j][e] = 0.f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t ah[4], al[4], b[4];
            split2(st[2 * ks][0], st[2 * ks][1], ah[0], al[0]);
            split2(st[2 * ks][2], st[2 * ks][3], ah[1], al[1]);
            split2(st[2 * ks + 1][0], st[2 * ks + 1][1], ah[2], al[2]);
            split2(st[2 * ks + 1][2], st[2 * ks + 1][3], ah[3], al[3]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              ldmatrix4(b, sb + L::Q + box_at(16 * t + ((mi >> 1) << 3) + ml, 2 * ks + (mi & 1)));
              mma(qs[2 * t], ah, b[0], b[1]);
              mma(qs[2 * t + 1], ah, b[2], b[3]);
              mma(qs[2 * t], al, b[0], b[1]);
              mma(qs[2 * t + 1], al, b[2], b[3]);
            }
          }
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
              const uint4 w = frag(2, block_of(tb, jb)), wl = frag(3, block_of(tb, jb));
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
      }
      if constexpr (MODE == kFwd) rows_out(y, t0, cn); else rows_out(ev, t0, cn);
      // 5. S^T
      uint32_t kt[2][KS][4];
      auto ask_t = [&](int t) {
#pragma unroll
        for (int k2 = 0; k2 < KS; ++k2)
          ldmatrix4t(kt[t & 1][k2], sb + L::K + box_at(16 * t + ((mi & 1) << 3) + ml, 2 * k2 + (mi >> 1)));
      };
      ask_t(0);
#pragma unroll
      for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) st[j][e] *= last;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t uh[4], ul[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 2 * t + (e >> 1), r = 2 * (e & 1);
          const float2 b = *reinterpret_cast<const float2*>(BT + 8 * j + 2 * tig);
          const float2 ec = *reinterpret_cast<const float2*>(EC + 8 * j + 2 * tig);
          split2(b.x * ec.x * ev[j][r], b.y * ec.y * ev[j][r + 1], uh[e], ul[e]);
        }
        if (t < 3) ask_t(t + 1);
#pragma unroll
        for (int k2 = 0; k2 < KS; ++k2) {
          mma(st[2 * k2], uh, kt[t & 1][k2][0], kt[t & 1][k2][1]);
          mma(st[2 * k2 + 1], uh, kt[t & 1][k2][2], kt[t & 1][k2][3]);
        }
#pragma unroll
        for (int k2 = 0; k2 < KS; ++k2) {
          mma(st[2 * k2], ul, kt[t & 1][k2][0], kt[t & 1][k2][1]);
          mma(st[2 * k2 + 1], ul, kt[t & 1][k2][2], kt[t & 1][k2][3]);
        }
      }
    } else {
      // dU^T = (P^T dO)^T + e^{G_C-G} (K dS)^T
      uint32_t dof[4][4];                            // dO^T as A fragments
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t v[4];
        ldmatrix4t(v, sb + L::V + box_at(16 * t + ((mi >> 1) << 3) + ml, 2 * warp + (mi & 1)));
#pragma unroll
        for (int e = 0; e < 4; ++e) dof[t][e] = v[e];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 ec = *reinterpret_cast<const float2*>(EC + 8 * j + 2 * tig);
        x[j][0] *= ec.x; x[j][1] *= ec.y; x[j][2] *= ec.x; x[j][3] *= ec.y;
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb)
#pragma unroll
        for (int jb = 0; jb <= tb; ++jb) {
          const uint4 ph = frag(2, block_of(tb, jb));
          mma(x[2 * jb], dof[tb], ph.x, ph.y);
          mma(x[2 * jb + 1], dof[tb], ph.z, ph.w);
          const uint4 pl = frag(3, block_of(tb, jb));
          mma(x[2 * jb], dof[tb], pl.x, pl.y);
          mma(x[2 * jb + 1], dof[tb], pl.z, pl.w);
        }
      // dR^T = (beta dU)^T T
      uint32_t rh[4][4], rl[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 2 * t + (e >> 1), r = 2 * (e & 1);
          const float2 b = *reinterpret_cast<const float2*>(BT + 8 * j + 2 * tig);
          split2(b.x * x[j][r], b.y * x[j][r + 1], rh[t][e], rl[t][e]);
        }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[j][e] = 0.f;
#pragma unroll
      for (int tb = 0; tb < 4; ++tb)
#pragma unroll
        for (int jb = 0; jb <= tb; ++jb) {
          const uint4 th = frag(0, block_of(tb, jb));
          mma(y[2 * jb], rh[tb], th.x, th.y);
          mma(y[2 * jb + 1], rh[tb], th.z, th.w);
          const uint4 tl = frag(1, block_of(tb, jb));
          mma(y[2 * jb], rl[tb], th.x, th.y);
          mma(y[2 * jb + 1], rl[tb], th.z, th.w);
          mma(y[2 * jb], rh[tb], tl.x, tl.y);
          mma(y[2 * jb + 1], rh[tb], tl.z, tl.w);
        }
      rows_out(y, t0, cn);
      // dS^T = e^{G_C} dS^T + (scale e^G dO)^T Q - (e^G dR)^T K
#pragma unroll
      for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) st[j][e] *= last;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t qh[4], ql[4], kh[4], kl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 2 * t + (e >> 1), r = 2 * (e & 1);
          const float2 eg = *reinterpret_cast<const float2*>(EG + 8 * j + 2 * tig);
          split2(p.scale * eg.x * low_half(dof[t][e]), p.scale * eg.y * high_half(dof[t][e]), qh[e], ql[e]);
          split2(-eg.x * y[j][r], -eg.y * y[j][r + 1], kh[e], kl[e]);
        }
#pragma unroll
        for (int k4 = 0; k4 < KS; k4 += 4) {
          uint32_t b[4][4], d[4][4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t at = box_at(16 * t + ((mi & 1) << 3) + ml, 2 * (k4 + x) + (mi >> 1));
            ldmatrix4t(b[x], sb + L::Q + at);
            ldmatrix4t(d[x], sb + L::K + at);
          }
#pragma unroll
          for (int part = 0; part < 4; ++part)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t (&w)[4] = part & 1 ? d[x] : b[x];
              const uint32_t (&f)[4] = part == 0 ? qh : part == 1 ? kh : part == 2 ? ql : kl;
              mma(st[2 * (k4 + x)], f, w[0], w[1]);
              mma(st[2 * (k4 + x) + 1], f, w[2], w[3]);
            }
        }
      }
    }
  }
  if (p.S_out != nullptr) {
    float* dst = p.S_out + ((long long)s * p.H + h) * DK * p.dv + m0 + g;
#pragma unroll
    for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[(long long)(8 * j + 2 * tig + (e & 1)) * p.dv + 8 * (e >> 1)] = st[j][e];
  }
}

template <int DK, int W>
__global__ void __launch_bounds__(32 * W)
gated_chain_kernel(const ChainArgs p, const __grid_constant__ ChainMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  chain<DK, kFwd, W>(p, maps, blockIdx.x, smem);
}

// Both chains of the backward of the same columns side by side in a CTA (they need nothing
// of each other): four warps each.
template <int DK>
struct ChainsSmem {
  static constexpr int SAVE = (ChainSmem<DK, kRev, 4>::TOTAL + 1023) / 1024 * 1024;
  static constexpr int TOTAL = SAVE + ChainSmem<DK, kSave, 4>::TOTAL;
  static_assert(TOTAL <= 227 * 1024, "shared memory");
};
template <int DK>
__global__ void __launch_bounds__(256)
gated_chains_kernel(const ChainArgs rev, const __grid_constant__ ChainMaps rmaps, const ChainArgs save,
                    const __grid_constant__ ChainMaps smaps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (threadIdx.x < 128) chain<DK, kRev, 4>(rev, rmaps, blockIdx.x, smem);
  else chain<DK, kSave, 4>(save, smaps, blockIdx.x, smem + ChainsSmem<DK>::SAVE);
}

// W: of the forward
template <int DK, int W>
cudaError_t launch(const GatedArgs& a, ChainArgs f, const ChainArgs* save) {
  f.nblk = a.dv / (16 * (save != nullptr ? 4 : W));
  const long long grid = (long long)f.nseq * f.H * f.nblk;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const long long keys = (long long)a.B * a.Hk, heads = (long long)a.B * a.H;
  ChainMaps m, ms;
  if (!gated_map(&m.q, a.q, keys, a.N, DK, 64) || !gated_map(&m.k, a.k, keys, a.N, DK, 64) || !gated_map(&m.v, f.v, heads, a.N, a.dv, 64))
    return cudaErrorInvalidValue;
  f.status = device_status_ptr();
  if (f.status == nullptr) return cudaErrorNotReady;
  f.stall = take_gated_timeout_test(0) ? 1 : 0;
  cudaError_t e;
  if (save == nullptr) {
    auto kern = gated_chain_kernel<DK, W>;
    const int smem = ChainSmem<DK, kFwd, W>::TOTAL;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)grid, 32 * W, smem, a.stream>>>(f, m);
  } else {
    ChainArgs b = *save;
    b.nblk = f.nblk;
    b.status = f.status;
    b.stall = f.stall;
    ms = m;
    if (!gated_map(&ms.v, b.v, heads, a.N, a.dv, 64)) return cudaErrorInvalidValue;
    auto kern = gated_chains_kernel<DK>;
    constexpr int smem = ChainsSmem<DK>::TOTAL;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)grid, 256, smem, a.stream>>>(f, m, b, ms);
  }
  e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t dispatch(const GatedArgs& a, const ChainArgs& f, const ChainArgs* save) {
  if (a.dk == 64) return launch<64, 4>(a, f, save);
  return a.dv == 128 ? launch<128, 8>(a, f, save) : launch<128, 4>(a, f, save);
}

ChainArgs chain_args(const GatedArgs& a, const uint8_t* rec, int rec_bytes) {
  ChainArgs p{};
  p.v = a.v; p.rec = rec; p.rec_bytes = rec_bytes; p.offsets = a.offsets;
  p.Hk = a.Hk; p.H = a.H; p.N = a.N; p.dv = a.dv; p.nseq = a.nseq; p.scale = a.scale;
  return p;
}

}  // namespace

cudaError_t gated_chain_forward(const GatedArgs& a, const uint8_t* records) {
  ChainArgs p = chain_args(a, records, REC_FWD);
  p.S_in = a.S0; p.S_out = a.S_final; p.out = (__nv_bfloat16*)a.out;
  return dispatch(a, p, nullptr);
}

cudaError_t gated_chain_backward(const GatedArgs& a, const uint8_t* records, const ChainOut& o) {
  ChainArgs r = chain_args(a, records, REC_BWD), s = r;
  r.v = a.dout; r.S_in = a.dS; r.S_out = a.dS0; r.out = (__nv_bfloat16*)a.dv_; r.out_lo = o.dr_lo;
  r.states = o.dstates; r.states_lo = o.dstates_lo;
  s.S_in = a.S0; s.out = o.e; s.out_lo = o.e_lo; s.states = o.states; s.states_lo = o.states_lo;
  return dispatch(a, r, &s);
}

}  // namespace la
