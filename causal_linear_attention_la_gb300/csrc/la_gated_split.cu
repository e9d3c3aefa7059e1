// The chains of the gated delta rule for few heads: as la_gated_chain.cu (formulas,
// precision: la_gated_mma.cuh), with the work on 16 columns of a state spread over
// eight warps of a CTA, so that a chunk takes less time.
//
// Four chain warps share the columns m of the state: warp kw has S^T [16 x DK/4], a
// quarter of the keys' components, as accumulators of m16n8k16. Per chunk:
//   1. its share of (K S)^T           A = S^T from the registers
//   2. the shares meet in shared memory; from here on warp kw has the 16 tokens of
//      block kw:  R^T = V^T - e^G (K S)^T
//   3. E^T = R^T T^T over the blocks up to its own, U = beta E
//   4. S^T = e^{G_C} S^T + (e^{G_C-G} U)^T K, its quarter again
// (backward the same with dS, dO and the transposed triangles.) Results of a step are
// the next one's A fragments as they lie in registers, and go through shared memory as such.
// Four helper warps do what the chain need not wait for: the copies of later
// chunks by TMA (by cp.async their 100 instructions a chunk took 1300 cycles, more than
// half of the chain's time), (Q S)^T + U^T P^T and the outputs of the chunk before (a chain warp leaves its
// split S and U as fragments), in the backward P^T dO and the states that are kept. One
// barrier of all eight warps a chunk, two of the chain warps alone.
#include <cudaTypedefs.h>

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
constexpr int NH = 128;                              // helper threads, as many chain threads

template <int DK, int MODE>
struct SplitSmem {
  static constexpr int TB = C * DK * 2;              // a tile of K or Q
  static constexpr int VB = C * 32;                  // 16 columns of V or dO
  static constexpr int up(int x) { return (x + 1023) / 1024 * 1024; }   // (the swizzle goes by the address)
  // copies for the chain: K, (forward: V, backward: Q), T's triangles, vec
  static constexpr int TRI = 2 * FRAG;
  static constexpr int A_X = TB;                     // V or Q
  static constexpr int A_T = A_X + (MODE == kRev ? TB : VB);
  static constexpr int A_VEC = A_T + TRI;
  static constexpr int A_BYTES = A_VEC + VEC, A = up(A_BYTES);
  // and for the helpers: Q and P; backward dO and P^T's triangles; vec
  static constexpr int B_P = MODE == kRev ? VB : TB;
  static constexpr int B_VEC = B_P + TRI;
  static constexpr int B_BYTES = MODE == kSave ? 0 : B_VEC + VEC, B = up(B_BYTES);
  // between the warps
  static constexpr int SHARES = 0;                   // [to][from, without itself][2 tiles][lane] float4
  static constexpr int FR = SHARES + 12 * 1024;      // R's fragments [block][hi, lo][lane] 16 bytes
  static constexpr int FU = FR + 4096;               // and those of e^{G_C-G} U, or -e^G dR
  static constexpr int ROWS = FU + 4096;             // two chunks' U, E or dR: [hi, lo][block][lane] 16 bytes
  static constexpr int ROWB = 4096;
  static constexpr int SF = ROWS + 2 * ROWB;         // two chunks' S^T: [hi, lo][DK / 16][lane] 16 bytes
  static constexpr int SFB = 2 * (DK / 16) * 512;
  static constexpr int PRE = SF + 2 * SFB;           // backward, three chunks': P^T dO [block][2][lane] float4,
  static constexpr int PREB = MODE == kRev ? 4096 + 4096 : 0;   // fragments of scale e^G dO
  static constexpr int OUT = PRE + 3 * PREB;         // helper warps' rows on their way out
  static constexpr int BARS = OUT + 4 * 512;         // four barriers, a flag
  static constexpr int X = up(BARS + 64);
  static constexpr int total(int depth) { return X + (3 + depth) * A + (2 + depth) * B; }
  static constexpr int DEPTH = total(1) <= 227 * 1024 ? 1 : 0;  // chunks of copies in flight beside the next one's
  static constexpr int TOTAL = total(DEPTH);
  static_assert(TOTAL <= 227 * 1024, "shared memory");
};

struct SplitArgs {
  const __nv_bfloat16* q; const __nv_bfloat16* k; const __nv_bfloat16* v;   // v: dO in reverse
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

// Maps of [heads][rows][DK] in boxes of 64 columns and 64 rows, of [heads][rows][dv] in boxes of 16
struct SplitMaps { CUtensorMap q, k, v; };

__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

template <int DK, int MODE, bool ORDER>
__device__ __forceinline__ void split_chain(const SplitArgs& p, const SplitMaps& maps, long long block, uint8_t* smem) {
  using L = SplitSmem<DK, MODE>;
  constexpr int KS = DK / 64, SA = 3 + L::DEPTH, SB = 2 + L::DEPTH;
  const int tid = threadIdx.x, lane = tid & 31, kw = (tid >> 5) & 3;
  const bool helper = tid >= NH;
  const int g = lane >> 2, tig = lane & 3, mi = lane >> 3, ml = lane & 7;
  const int blk = (int)(block % p.nblk);
  block /= p.nblk;
  const int h = (int)(block % p.H), r = (int)(block / p.H);
  const int s = ORDER ? sequence_of(p.offsets, r, p.nseq, p.N) : r;
  const SeqRange sq = seq_range(p.offsets, s, p.N, C);
  const int n = sq.n, nchunks = (n + C - 1) / C;
  const long long vrow = ((long long)sq.b * p.H + h) * p.N + sq.lo;
  const int m0 = blk * 16;
  __nv_bfloat16* ob = p.out + vrow * p.dv + m0;
  __nv_bfloat16* ol = MODE == kFwd ? nullptr : p.out_lo + vrow * p.dv + m0;
  const uint32_t base = smem_addr(smem);
  const uint32_t a0 = base + L::X, b0 = a0 + SA * L::A;
  auto chunk_of = [&](int i) { return MODE == kRev ? nchunks - 1 - i : i; };
  auto quad = [&](int off) { return reinterpret_cast<uint4*>(smem + off) + lane; };

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BARS);
  volatile int* gave_up = reinterpret_cast<volatile int*>(smem + L::BARS + 32);
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) mbar_init(&bars[i], 1);
    *gave_up = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (helper) {
    const int ht = tid - NH;
    const int kh = sq.b * p.Hk + h / (p.H / p.Hk), vh = sq.b * p.H + h;
    // one thread asks for copies, of group `seq`: a barrier each, four in turn
    auto boxes = [&](uint32_t to, const CUtensorMap* map, int t0, uint64_t* bar) {
#pragma unroll
      for (int b = 0; b < DK / 64; ++b) tma_load_3d(smem + (to - base) + b * C * 128, map, bar, 64 * b, sq.lo + t0, kh);
    };
    auto bytes_a = [&](int i) { return i < nchunks ? L::A_BYTES : 0; };
    auto bytes_b = [&](int i) { return i < nchunks ? L::B_BYTES : 0; };
    auto load_a = [&](int i, uint64_t* bar) {
      if (i >= nchunks) return;
      const int c = chunk_of(i), t0 = c * C;
      const uint32_t to = a0 + (i % SA) * L::A;
      boxes(to, &maps.k, t0, bar);
      if (MODE == kRev) boxes(to + L::A_X, &maps.q, t0, bar);
      else tma_load_3d(smem + (to - base) + L::A_X, &maps.v, bar, m0, sq.lo + t0, vh);
      const uint8_t* rec = p.rec + ((long long)(sq.slot + c) * p.H + h) * p.rec_bytes;
      if (MODE != kRev) {                            // [T lo | T hi | vec]
        bulk_load(to + L::A_T, rec, L::TRI + VEC, bar);
      } else {                                       // T^T hi, T^T lo, vec
        bulk_load(to + L::A_T, rec + OFF_REST, FRAG, bar);
        bulk_load(to + L::A_T + FRAG, rec + OFF_REST + 2 * FRAG, FRAG, bar);
        bulk_load(to + L::A_VEC, rec + OFF_VEC, VEC, bar);
      }
    };
    auto load_b = [&](int i, uint64_t* bar) {
      if (MODE == kSave || i >= nchunks) return;
      const int c = chunk_of(i), t0 = c * C;
      const uint32_t to = b0 + (i % SB) * L::B;
      const uint8_t* rec = p.rec + ((long long)(sq.slot + c) * p.H + h) * p.rec_bytes;
      if (MODE == kFwd) {
        boxes(to, &maps.q, t0, bar);
        bulk_load(to + L::B_P, rec + OFF_REST, L::TRI, bar);
      } else {
        tma_load_3d(smem + (to - base), &maps.v, bar, m0, sq.lo + t0, vh);
        bulk_load(to + L::B_P, rec + OFF_REST + FRAG, FRAG, bar);
        bulk_load(to + L::B_P + FRAG, rec + OFF_REST + 3 * FRAG, FRAG, bar);
      }
      bulk_load(to + L::B_VEC, rec + OFF_VEC, VEC, bar);
    };
    // Copies have whole boxes: rows behind the sequence's last token become zeros.
    auto clear = [&](uint32_t to, int piece, int rows0) {         // rows of `piece` 16-byte pieces
      for (int j = ht; j < (C - rows0) * piece; j += NH)
        *reinterpret_cast<uint4*>(smem + (to - base) + rows0 * piece * 16 + j * 16) = make_uint4(0u, 0u, 0u, 0u);
    };
    auto clear_a = [&](int i) {
      if (i >= nchunks) return;
      const int m = n - chunk_of(i) * C;
      if (m >= C) return;
      const uint32_t to = a0 + (i % SA) * L::A;
#pragma unroll
      for (int b = 0; b < DK / 64; ++b) {
        clear(to + b * C * 128, 8, m);
        if (MODE == kRev) clear(to + L::A_X + b * C * 128, 8, m);
      }
      if (MODE != kRev) clear(to + L::A_X, 2, m);
      sm100::fence_proxy_async_smem();               // (copies come here again)
    };
    auto clear_b = [&](int i) {
      if (MODE == kSave || i >= nchunks) return;
      const int m = n - chunk_of(i) * C;
      if (m >= C) return;
      const uint32_t to = b0 + (i % SB) * L::B;
      if (MODE == kRev) {
        clear(to, 2, m);
      } else {
#pragma unroll
        for (int b = 0; b < DK / 64; ++b) clear(to + b * C * 128, 8, m);
      }
      sm100::fence_proxy_async_smem();
    };
    bool ok = true;
    int late = 0;
    // (once a wait gave up, none is begun and no copy asked for)
    auto landed = [&](int seq) {
      if (!ok) return;
      ok = mbar_drain(&bars[seq & 3], (seq >> 2) & 1, kWaitNs);
      late = seq;
    };
    // backward: of chunk i, P^T dO of block kw and the fragments of scale e^G dO
    auto pre = [&](int i) {
      if (MODE != kRev || i >= nchunks) return;
      const uint32_t st = b0 + (i % SB) * L::B;
      const uint8_t* sp = smem + (st - base);
      float d1[2][4], d2[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) d1[j][e] = d2[j][e] = 0.f;
      uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        if (tb < kw) continue;
        uint32_t a[4];
        ldmatrix4t(a, st + tile_at<2>(16 * tb + ((mi >> 1) << 3) + ml, mi & 1));
        if (tb == kw) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = a[e];
        }
        const uint4 ph = *reinterpret_cast<const uint4*>(sp + L::B_P + block_of(tb, kw) * 512 + lane * 16);
        mma(d1[0], a, ph.x, ph.y);
        mma(d1[1], a, ph.z, ph.w);
        const uint4 pl = *reinterpret_cast<const uint4*>(sp + L::B_P + FRAG + block_of(tb, kw) * 512 + lane * 16);
        mma(d2[0], a, pl.x, pl.y);
        mma(d2[1], a, pl.z, pl.w);
      }
      const int at = L::PRE + (i % 3) * L::PREB;
      float4* to = reinterpret_cast<float4*>(smem + at) + kw * 64 + lane;
      to[0] = make_float4(d1[0][0] + d2[0][0], d1[0][1] + d2[0][1], d1[0][2] + d2[0][2], d1[0][3] + d2[0][3]);
      to[32] = make_float4(d1[1][0] + d2[1][0], d1[1][1] + d2[1][1], d1[1][2] + d2[1][2], d1[1][3] + d2[1][3]);
      uint32_t qh[4], ql[4];
      const float* vec = reinterpret_cast<const float*>(sp + L::B_VEC);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 eg = *reinterpret_cast<const float2*>(vec + 16 * kw + 8 * (e >> 1) + 2 * tig);
        split2(p.scale * eg.x * low_half(v[e]), p.scale * eg.y * high_half(v[e]), qh[e], ql[e]);
      }
      *quad(at + 4096 + kw * 1024) = make_uint4(qh[0], qh[1], qh[2], qh[3]);
      *quad(at + 4096 + kw * 1024 + 512) = make_uint4(ql[0], ql[1], ql[2], ql[3]);
    };
    // Copies that are asked for behind the barrier of chunk i: the chain's of chunk
    // i + 2 + DEPTH, over those of chunk i - 1; the helpers' of chunk i + 1 + DEPTH, or
    // (backward, where they prepare chunk i + 2 during chunk i) i + 3 + DEPTH. They have
    // landed at the barrier of chunk i + 1 + DEPTH, behind which the chain goes on to chunk
    // i + 2 + DEPTH.
    constexpr int BA = MODE == kRev ? 3 : 1;
    constexpr int B0 = MODE == kRev ? SB : 1 + L::DEPTH;          // the helpers' first chunks
    if (ht == 0) {
      uint32_t bytes = p.stall ? 16 : 0;
      for (int i = 0; i < 2 + L::DEPTH; ++i) bytes += bytes_a(i);
      for (int i = 0; i < B0; ++i) bytes += bytes_b(i);
      mbar_arrive_expect_tx(&bars[0], bytes);
      for (int i = 0; i < 2 + L::DEPTH; ++i) load_a(i, &bars[0]);
      for (int i = 0; i < B0; ++i) load_b(i, &bars[0]);
    }
    landed(0);
    for (int i = 0; i < 2 + L::DEPTH; ++i) clear_a(i);
    for (int i = 0; i < B0; ++i) clear_b(i);
    bar_sync(1, NH);
    if (MODE == kRev) {
      pre(0);
      bar_sync(1, NH);                               // chunk 0's rows have been read
      if (ht == 0) {
        mbar_arrive_expect_tx(&bars[1], bytes_b(SB));
        load_b(SB, &bars[1]);
      }
      pre(1);
      landed(1);
      clear_b(SB);
    } else if (ht == 0) {
      mbar_arrive_expect_tx(&bars[1], 0);
    }
    bar_sync(0, 2 * NH);                             // chunk 0's copies are there
    for (int i = 0; i < nchunks; ++i) {
      const int c = chunk_of(i), t0 = c * C, cn = min(C, n - t0);
      bar_sync(0, 2 * NH);                           // chunk i: S^T and the rows are there, chunk i - 1 is done with
      if (ht == 0 && ok) {
        uint64_t* bar = &bars[(i + 2) & 3];
        mbar_arrive_expect_tx(bar, bytes_a(i + 2 + L::DEPTH) + bytes_b(i + BA + L::DEPTH));
        load_a(i + 2 + L::DEPTH, bar);
        load_b(i + BA + L::DEPTH, bar);
      }
      const uint8_t* sf = smem + L::SF + (i & 1) * L::SFB;
      if (MODE != kFwd) {
        // the state as bf16 rows [dv][DK]: two lanes join 8 bytes of neighbouring tiles
        const long long at = (((long long)(sq.slot + c) * p.H + h) * p.dv + m0) * DK;
        const bool odd = tig & 1;
        auto dump = [&](__nv_bfloat16* dst, int part) {
#pragma unroll
          for (int k = kw; k < DK / 16; k += 4) {
            const uint4 f = *reinterpret_cast<const uint4*>(sf + (part * (DK / 16) + k) * 512 + lane * 16);
            const uint32_t lo8[2] = {f.x, f.y}, hi8[2] = {f.z, f.w};      // components 16 k .. + 7, + 8 .. + 15; rows g, g + 8
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? lo8[r] : hi8[r], 1);
              *reinterpret_cast<uint2*>(dst + at + (long long)(g + 8 * r) * DK + 16 * k + 8 * odd + 4 * (tig >> 1)) =
                  odd ? make_uint2(got, hi8[r]) : make_uint2(lo8[r], got);
            }
          }
        };
        dump(p.states, 0);
        dump(p.states_lo, 1);
      }
      uint4 row4;
      {
        const uint8_t* rows = smem + L::ROWS + (i & 1) * L::ROWB;
        row4 = *reinterpret_cast<const uint4*>(rows + kw * 512 + lane * 16);
        if (MODE == kFwd) {
          const uint32_t st = b0 + (i % SB) * L::B;
          const uint8_t* sp = smem + (st - base);
          float y[2][4], z[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[j][e] = z[j][e] = 0.f;
#pragma unroll
          for (int k = 0; k < DK / 16; ++k) {
            const uint4 f = *reinterpret_cast<const uint4*>(sf + k * 512 + lane * 16);
            const uint4 f2 = *reinterpret_cast<const uint4*>(sf + (DK / 16 + k) * 512 + lane * 16);
            const uint32_t a[4] = {f.x, f.y, f.z, f.w}, a2[4] = {f2.x, f2.y, f2.z, f2.w};
            uint32_t b[4];
            ldmatrix4(b, st + box_at(16 * kw + ((mi >> 1) << 3) + ml, 2 * k + (mi & 1)));
            mma(y[0], a, b[0], b[1]);
            mma(y[1], a, b[2], b[3]);
            mma(z[0], a2, b[0], b[1]);
            mma(z[1], a2, b[2], b[3]);
          }
          const float* vec = reinterpret_cast<const float*>(sp + L::B_VEC);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 eg = *reinterpret_cast<const float2*>(vec + 16 * kw + 8 * j + 2 * tig);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[j][e] = (y[j][e] + z[j][e]) * (p.scale * ((e & 1) ? eg.y : eg.x));
          }
          const uint4 row2 = *reinterpret_cast<const uint4*>(rows + 2048 + kw * 512 + lane * 16);
          const uint32_t u[4] = {row4.x, row4.y, row4.z, row4.w}, u2[4] = {row2.x, row2.y, row2.z, row2.w};
          auto times = [&](float (&o)[2][4], const uint32_t (&a)[4], const uint32_t (&a2)[4], int jb) {
            const uint8_t* pp = sp + L::B_P + block_of(kw, jb) * 512 + lane * 16;
            const uint4 w = *reinterpret_cast<const uint4*>(pp), w2 = *reinterpret_cast<const uint4*>(pp + FRAG);
            mma(o[0], a, w.x, w.y);
            mma(o[1], a, w.z, w.w);
            mma(o[0], a2, w.x, w.y);
            mma(o[1], a2, w.z, w.w);
            mma(o[0], a, w2.x, w2.y);
            mma(o[1], a, w2.z, w2.w);
          };
#pragma unroll
          for (int jb = 0; jb < 3; ++jb) {
            if (jb >= kw) continue;
            const uint4 f = *reinterpret_cast<const uint4*>(rows + jb * 512 + lane * 16);
            const uint4 f2 = *reinterpret_cast<const uint4*>(rows + 2048 + jb * 512 + lane * 16);
            const uint32_t a[4] = {f.x, f.y, f.z, f.w}, a2[4] = {f2.x, f2.y, f2.z, f2.w};
            times(y, a, a2, jb);
          }
          // a zero weight of a later token's row that is not finite would be NaN for
          // the tokens before it: then each token with the rows behind it left out
          float bad = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) bad = fmaf(0.f, low_half(u2[e]), fmaf(0.f, high_half(u2[e]), bad));   // (a high part stops at the largest number)
          if (!__any_sync(0xffffffffu, bad != 0.f)) {
            times(y, u, u2, kw);
          } else {
            float o[2][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              z[0][e] = y[0][e];
              z[1][e] = y[1][e];
            }
#pragma unroll 1
            for (int t = 0; t < 16; ++t) {
              uint32_t a[4], a2[4];
              rows_to(a, u, 0, t, tig);
              rows_to(a2, u2, 0, t, tig);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[0][e] = z[0][e];
                o[1][e] = z[1][e];
              }
              times(o, a, a2, kw);
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (8 * j + 2 * tig + (e & 1) == t) y[j][e] = o[j][e];
            }
          }
          row4 = make_uint4(pack2(y[0][0], y[0][1]), pack2(y[0][2], y[0][3]), pack2(y[1][0], y[1][1]), pack2(y[1][2], y[1][3]));
        }
      }
      // rows [token][16 columns] of block kw, 16 bytes a lane: rounded, and (backward) what that leaves out
#pragma unroll
      for (int part = 0; part < (MODE == kFwd ? 1 : 2); ++part) {
        const uint32_t to = base + L::OUT + kw * 512;
        if (part == 1) row4 = *reinterpret_cast<const uint4*>(smem + L::ROWS + (i & 1) * L::ROWB + 2048 + kw * 512 + lane * 16);
        stmatrix4t(to + tile_at<2>(((mi >> 1) << 3) + ml, mi & 1), row4.x, row4.y, row4.z, row4.w);
        __syncwarp();
        const int r = lane >> 1, half = lane & 1, t = 16 * kw + r;
        const uint4 w = *reinterpret_cast<const uint4*>(smem + L::OUT + kw * 512 + tile_at<2>(r, half));
        if (t < cn && ok) *reinterpret_cast<uint4*>((part ? ol : ob) + (long long)(t0 + t) * p.dv + 8 * half) = w;
        __syncwarp();
      }
      pre(i + 2);
      if (i >= L::DEPTH) {
        landed(i + 2 - L::DEPTH);
        clear_a(i + 2);
        clear_b(i + BA);
      }
    }
    if (L::DEPTH && nchunks > 0) landed(nchunks + 1);
    if (!ok) {
      // copies in flight end before shared memory is released
      *gave_up = 1;
      for (int q = late; q < late + 2; ++q) mbar_drain(&bars[q & 3], (q >> 2) & 1, kWaitNs / 8);
      atomicExch(p.status, (int)LA_ERR_TIMEOUT);     // (any thread's: one may give up where the others just did not)
    }
    bar_sync(0, 2 * NH);
    return;
  }

  // ------------------------------ chain warps ------------------------------
  float4* shares = reinterpret_cast<float4*>(smem + L::SHARES);
  float st[2 * KS][4];                               // S^T: tile j has dk = kw DK / 4 + 8 j ..
  {
    const float* src = p.S_in == nullptr ? nullptr : p.S_in + (((long long)s * p.H + h) * DK + kw * (DK / 4)) * p.dv + m0 + g;
#pragma unroll
    for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        st[j][e] = src == nullptr ? 0.f : src[(long long)(8 * j + 2 * tig + (e & 1)) * p.dv + 8 * (e >> 1)];
  }
  bar_sync(0, 2 * NH);
  // (fragments are asked for as soon as their copies are there, ahead of the barrier before their use)
  uint32_t kf[KS][4][4];                             // K's rows, for the next chunk's first product
  auto ask_k = [&](int i) {
    const uint32_t sa = a0 + (i % SA) * L::A;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        ldmatrix4(kf[ks][t], sa + box_at(16 * t + ((mi >> 1) << 3) + ml, kw * (DK / 32) + 2 * ks + (mi & 1)));
  };
  if (nchunks > 0) ask_k(0);
  for (int i = 0; i < nchunks; ++i) {
    const uint32_t sa = a0 + (i % SA) * L::A;
    const uint8_t* ap = smem + (sa - base);
    const float* vec = reinterpret_cast<const float*>(ap + L::A_VEC);
    auto frag = [&](int lo, int b) {                 // (T lo is the first in a record)
      const int off = (MODE == kRev ? lo : 1 - lo) * FRAG;
      return *reinterpret_cast<const uint4*>(ap + L::A_T + off + b * 512 + lane * 16);
    };
    float2 eg[2], ec[2], bt[2];                      // of this lane's four tokens of block kw
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float* at = vec + 16 * kw + 8 * j + 2 * tig;
      eg[j] = *reinterpret_cast<const float2*>(at);
      ec[j] = *reinterpret_cast<const float2*>(at + C);
      bt[j] = *reinterpret_cast<const float2*>(at + 2 * C);
    }
    const float last = vec[C - 1];
    uint32_t v[4];                                   // V^T of block kw, or (backward) P^T dO
    float4 d[2];
    if (MODE == kRev) {
      const float4* from = reinterpret_cast<const float4*>(smem + L::PRE + (i % 3) * L::PREB) + kw * 64 + lane;
      d[0] = from[0];
      d[1] = from[32];
    } else {
      ldmatrix4t(v, sa + L::A_X + tile_at<2>(16 * kw + ((mi >> 1) << 3) + ml, mi & 1));
    }
    // 1. this warp's share of (K S)^T
    float x[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[j][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t ah[4], al[4];
      const uint32_t (&b)[4][4] = kf[ks];
      split2(st[2 * ks][0], st[2 * ks][1], ah[0], al[0]);
      split2(st[2 * ks][2], st[2 * ks][3], ah[1], al[1]);
      split2(st[2 * ks + 1][0], st[2 * ks + 1][1], ah[2], al[2]);
      split2(st[2 * ks + 1][2], st[2 * ks + 1][3], ah[3], al[3]);
      const int sf = L::SF + (i & 1) * L::SFB + (kw * KS + ks) * 512;
      *quad(sf) = make_uint4(ah[0], ah[1], ah[2], ah[3]);
      *quad(sf + (DK / 16) * 512) = make_uint4(al[0], al[1], al[2], al[3]);
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
    // 2. to the warps of their blocks
    float xs[2][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t == kw) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xs[0][e] = x[2 * t][e];
          xs[1][e] = x[2 * t + 1][e];
        }
      } else {
        float4* to = shares + (t * 3 + ((kw - t + 4) & 3) - 1) * 64 + lane;
        to[0] = make_float4(x[2 * t][0], x[2 * t][1], x[2 * t][2], x[2 * t][3]);
        to[32] = make_float4(x[2 * t + 1][0], x[2 * t + 1][1], x[2 * t + 1][2], x[2 * t + 1][3]);
      }
    }
    uint4 th[4], tl[4];                              // T's fragments
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (MODE == kRev ? b < kw : b > kw) continue;
      const int at = MODE == kRev ? block_of(b, kw) : block_of(kw, b);
      th[b] = frag(0, at);
      tl[b] = frag(1, at);
    }
#pragma unroll
    for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) st[j][e] *= last;
    bar_sync(2, NH);
#pragma unroll
    for (int f = 0; f < 3; ++f)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 a = shares[(kw * 3 + f) * 64 + j * 32 + lane];
        xs[j][0] += a.x; xs[j][1] += a.y; xs[j][2] += a.z; xs[j][3] += a.w;
      }
    uint32_t rh[4], rl[4];                           // R^T, or (beta dU)^T
    if (MODE == kRev) {
      const float dd[2][4] = {{d[0].x, d[0].y, d[0].z, d[0].w}, {d[1].x, d[1].y, d[1].z, d[1].w}};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = e >> 1, r = 2 * (e & 1);
        split2(bt[j].x * fmaf(ec[j].x, xs[j][r], dd[j][r]), bt[j].y * fmaf(ec[j].y, xs[j][r + 1], dd[j][r + 1]), rh[e], rl[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {                  // e: a0 .. a3 = (tile e / 2, rows 8 (e % 2))
        const int j = e >> 1, r = 2 * (e & 1);
        split2(low_half(v[e]) - eg[j].x * xs[j][r], high_half(v[e]) - eg[j].y * xs[j][r + 1], rh[e], rl[e]);
      }
    }
    *quad(L::FR + kw * 1024) = make_uint4(rh[0], rh[1], rh[2], rh[3]);
    *quad(L::FR + kw * 1024 + 512) = make_uint4(rl[0], rl[1], rl[2], rl[3]);
    bar_sync(2, NH);
    // 3. E^T, or dR^T: three sums, for the latency of an accumulator
    float ev[2][4], e1[2][4], e2[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) ev[j][e] = e1[j][e] = e2[j][e] = 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (MODE == kRev ? b < kw : b > kw) continue;
      const uint4 f = *quad(L::FR + b * 1024);
      const uint32_t a[4] = {f.x, f.y, f.z, f.w};
      mma(ev[0], a, th[b].x, th[b].y);
      mma(ev[1], a, th[b].z, th[b].w);
      const uint4 f2 = *quad(L::FR + b * 1024 + 512);
      const uint32_t a2[4] = {f2.x, f2.y, f2.z, f2.w};
      mma(e1[0], a2, th[b].x, th[b].y);
      mma(e1[1], a2, th[b].z, th[b].w);
      mma(e2[0], a, tl[b].x, tl[b].y);
      mma(e2[1], a, tl[b].z, tl[b].w);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) ev[j][e] += e1[j][e] + e2[j][e];
    if (MODE == kFwd) {
      // as for the outputs: a block with a row that is not finite is done again
      float bad = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) bad = fmaf(0.f, ev[j][e], bad);
      if (__any_sync(0xffffffffu, bad != 0.f)) {
        // (the same three sums, so that the other columns keep their bits)
        float low[3][2][4];
        auto add = [&](float (&o)[3][2][4], const uint32_t (&a)[4], const uint32_t (&a2)[4], int b) {
          const uint4 h4 = frag(0, block_of(kw, b));
          mma(o[0][0], a, h4.x, h4.y);
          mma(o[0][1], a, h4.z, h4.w);
          const uint4 l4 = frag(1, block_of(kw, b));
          mma(o[1][0], a2, h4.x, h4.y);
          mma(o[1][1], a2, h4.z, h4.w);
          mma(o[2][0], a, l4.x, l4.y);
          mma(o[2][1], a, l4.z, l4.w);
        };
#pragma unroll
        for (int z = 0; z < 24; ++z) low[z >> 3][(z >> 2) & 1][z & 3] = 0.f;
        for (int b = 0; b < kw; ++b) {
          const uint4 f = *quad(L::FR + b * 1024), f2 = *quad(L::FR + b * 1024 + 512);
          const uint32_t a[4] = {f.x, f.y, f.z, f.w}, a2[4] = {f2.x, f2.y, f2.z, f2.w};
          add(low, a, a2, b);
        }
#pragma unroll 1
        for (int t = 0; t < 16; ++t) {
          float o[3][2][4];
          uint32_t a[4], a2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 8 * (e >> 1) + 2 * tig;
            const uint32_t keep = (j <= t ? 0xffffu : 0u) | (j + 1 <= t ? 0xffff0000u : 0u);
            a[e] = rh[e] & keep;
            a2[e] = rl[e] & keep;
          }
#pragma unroll
          for (int z = 0; z < 24; ++z) o[z >> 3][(z >> 2) & 1][z & 3] = low[z >> 3][(z >> 2) & 1][z & 3];
          add(o, a, a2, kw);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (8 * j + 2 * tig + (e & 1) == t) ev[j][e] = o[0][j][e] + (o[1][j][e] + o[2][j][e]);
        }
      }
    }
    {
      uint32_t uh[4], ul[4], w[4], w2[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = e >> 1, r = 2 * (e & 1);
        if (MODE == kRev) {
          split2(-eg[j].x * ev[j][r], -eg[j].y * ev[j][r + 1], uh[e], ul[e]);
          split2_out(ev[j][r], ev[j][r + 1], w[e], w2[e]);
        } else {
          const float u0 = bt[j].x * ev[j][r], u1 = bt[j].y * ev[j][r + 1];
          split2(ec[j].x * u0, ec[j].y * u1, uh[e], ul[e]);
          if (MODE == kFwd) split2(u0, u1, w[e], w2[e]);
          else split2_out(ev[j][r], ev[j][r + 1], w[e], w2[e]);
        }
      }
      *quad(L::FU + kw * 1024) = make_uint4(uh[0], uh[1], uh[2], uh[3]);
      *quad(L::FU + kw * 1024 + 512) = make_uint4(ul[0], ul[1], ul[2], ul[3]);
      *quad(L::ROWS + (i & 1) * L::ROWB + kw * 512) = make_uint4(w[0], w[1], w[2], w[3]);
      *quad(L::ROWS + (i & 1) * L::ROWB + 2048 + kw * 512) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
    }
    // 4. this warp's quarter of the state
    uint32_t kt[4][KS][4], qt[MODE == kRev ? 4 : 1][KS][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int row = 16 * t + ((mi & 1) << 3) + ml, ch = kw * (DK / 32) + (mi >> 1);
#pragma unroll
      for (int k2 = 0; k2 < KS; ++k2) {
        ldmatrix4t(kt[t][k2], sa + box_at(row, ch + 2 * k2));
        if (MODE == kRev) ldmatrix4t(qt[t][k2], sa + L::A_X + box_at(row, ch + 2 * k2));
      }
    }
    uint4 f[4], f2[4];
    auto ask = [&](int from) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        f[t] = *quad(from + t * 1024);
        f2[t] = *quad(from + t * 1024 + 512);
      }
    };
    auto add = [&](const uint32_t (&tile)[4][KS][4]) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t ah[4] = {f[t].x, f[t].y, f[t].z, f[t].w};
#pragma unroll
        for (int k2 = 0; k2 < KS; ++k2) {
          mma(st[2 * k2], ah, tile[t][k2][0], tile[t][k2][1]);
          mma(st[2 * k2 + 1], ah, tile[t][k2][2], tile[t][k2][3]);
        }
        const uint32_t al[4] = {f2[t].x, f2[t].y, f2[t].z, f2[t].w};
#pragma unroll
        for (int k2 = 0; k2 < KS; ++k2) {
          mma(st[2 * k2], al, tile[t][k2][0], tile[t][k2][1]);
          mma(st[2 * k2 + 1], al, tile[t][k2][2], tile[t][k2][3]);
        }
      }
    };
    if constexpr (MODE == kRev) {
      ask(L::PRE + (i % 3) * L::PREB + 4096);
      add(qt);
    }
    bar_sync(0, 2 * NH);
    if (i + 1 < nchunks) ask_k(i + 1);
    ask(L::FU);
    add(kt);
  }
  bar_sync(0, 2 * NH);
  if (p.S_out != nullptr && !*gave_up) {
    float* dst = p.S_out + (((long long)s * p.H + h) * DK + kw * (DK / 4)) * p.dv + m0 + g;
#pragma unroll
    for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[(long long)(8 * j + 2 * tig + (e & 1)) * p.dv + 8 * (e >> 1)] = st[j][e];
  }
}

// ORDER: packed sequences (where it is not wanted its registers cost 1 % of the time)
template <int DK, bool ORDER>
__global__ void __launch_bounds__(2 * NH, 1)
gated_split_kernel(const SplitArgs p, const __grid_constant__ SplitMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  split_chain<DK, kFwd, ORDER>(p, maps, blockIdx.x, smem);
}

// Both chains of the backward in one launch (order: second_chain).
template <int DK>
__global__ void __launch_bounds__(2 * NH, 1)
gated_splits_kernel(const SplitArgs rev, const __grid_constant__ SplitMaps rmaps, const SplitArgs save,
                    const __grid_constant__ SplitMaps smaps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  unsigned number;
  if (second_chain(blockIdx.x, gridDim.x, rev.offsets != nullptr, rev.nblk * rev.H, number)) split_chain<DK, kSave, true>(save, smaps, number, smem);
  else split_chain<DK, kRev, true>(rev, rmaps, number, smem);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult qr;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) != cudaSuccess ||
        qr != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

bool make_maps(SplitMaps* m, const SplitArgs& a, int B, int dk) {
  return gated_map(&m->q, a.q, (long long)B * a.Hk, a.N, dk, 64) && gated_map(&m->k, a.k, (long long)B * a.Hk, a.N, dk, 64) &&
         gated_map(&m->v, a.v, (long long)B * a.H, a.N, a.dv, 16);
}

template <int DK>
cudaError_t launch(SplitArgs f, int B, const SplitArgs* save, cudaStream_t stream) {
  f.nblk = f.dv / 16;
  const long long grid = (long long)f.nseq * f.H * f.nblk * (save != nullptr ? 2 : 1);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  constexpr int kF = SplitSmem<DK, kFwd>::TOTAL, kR = SplitSmem<DK, kRev>::TOTAL, kS = SplitSmem<DK, kSave>::TOTAL;
  cudaError_t e;
  SplitMaps fm, bm;
  if (!make_maps(&fm, f, B, DK) || (save != nullptr && !make_maps(&bm, *save, B, DK))) return cudaErrorInvalidValue;
  f.status = device_status_ptr();
  if (f.status == nullptr) return cudaErrorNotReady;
  f.stall = take_gated_timeout_test(0) ? 1 : 0;
  if (save == nullptr) {
    auto kern = f.offsets != nullptr ? gated_split_kernel<DK, true> : gated_split_kernel<DK, false>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kF);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)grid, 2 * NH, kF, stream>>>(f, fm);
  } else {
    SplitArgs b = *save;
    b.nblk = f.nblk;
    b.status = f.status;
    b.stall = f.stall;
    constexpr int smem = kR > kS ? kR : kS;
    auto kern = gated_splits_kernel<DK>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)grid, 2 * NH, smem, stream>>>(f, fm, b, bm);
  }
  e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t dispatch(const SplitArgs& f, const SplitArgs* save, int B, int dk, cudaStream_t stream) {
  return dk == 64 ? launch<64>(f, B, save, stream) : launch<128>(f, B, save, stream);
}

SplitArgs split_args(const GatedArgs& a, const uint8_t* rec, int rec_bytes) {
  SplitArgs p{};
  p.q = (const __nv_bfloat16*)a.q; p.k = (const __nv_bfloat16*)a.k; p.v = (const __nv_bfloat16*)a.v;
  p.rec = rec; p.rec_bytes = rec_bytes; p.offsets = a.offsets;
  p.Hk = a.Hk; p.H = a.H; p.N = a.N; p.dv = a.dv; p.nseq = a.nseq; p.scale = a.scale;
  return p;
}

}  // namespace

bool gated_map(CUtensorMap* m, const void* ptr, long long heads, int N, int d, int cols) {
  const auto enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)heads};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)N * d * 2};
  const cuuint32_t box[3] = {(cuuint32_t)cols, (cuuint32_t)gmma::C, 1}, es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 16 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One of these CTAs has an SM for itself and takes 1.3 us a chunk of d = 128 (backward, the
// reverse chain and the one that keeps the states, 1.4 each); pairs of warps take 2.9, but four
// share an SM, and both chains of four column groups of the backward 6.1 (d = 64: 4.3). 4096
// tokens of d = 128, forward: 16 heads (128 CTAs here) 81 us against 188, 32 heads 166 against
// 188, 64 heads 330 against 189; backward: 19 heads (304) 179 against 390, 32 heads 349 against
// 390, 64 heads 625 against 394; 1024 tokens, d = 64, 256 heads (2048) 289 against 137. Packed
// sequences are taken to have one of half their rows, of more than eight one of 4 / nseq of
// them: 16 heads of 16384 rows, 12 unlike ones, 308 against 190, 40 like ones 449 against 226;
// backward of 12 heads of 8192 rows, d = 64, nine unlike ones 116 against 222, 40 like ones
// 233 against 81.
bool gated_split_wanted(const GatedArgs& a, bool backward) {
  const long long groups = (long long)a.H * (a.dv / 16) * (backward ? 2 : 1);
  const long long most = (backward ? a.dk == 128 ? 4 : 3 : 2) * kSlots;
  if (a.offsets == nullptr || a.nseq <= 2) return groups * a.nseq <= most;
  return groups * (a.nseq > 8 ? a.nseq : 8) <= 4 * most;
}

cudaError_t gated_split_forward(const GatedArgs& a, const uint8_t* records) {
  SplitArgs p = split_args(a, records, REC_FWD);
  p.S_in = a.S0; p.S_out = a.S_final; p.out = (__nv_bfloat16*)a.out;
  return dispatch(p, nullptr, a.B, a.dk, a.stream);
}

cudaError_t gated_split_backward(const GatedArgs& a, const uint8_t* records, const ChainOut& o) {
  SplitArgs r = split_args(a, records, REC_BWD), s = r;
  r.v = (const __nv_bfloat16*)a.dout; r.S_in = a.dS; r.S_out = a.dS0; r.out = (__nv_bfloat16*)a.dv_; r.out_lo = o.dr_lo;
  r.states = o.dstates; r.states_lo = o.dstates_lo;
  s.S_in = a.S0; s.out = o.e; s.out_lo = o.e_lo; s.states = o.states; s.states_lo = o.states_lo;
  return dispatch(r, &s, a.B, a.dk, a.stream);
}

}  // namespace la
