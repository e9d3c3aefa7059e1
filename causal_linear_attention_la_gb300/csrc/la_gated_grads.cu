// Gradients of the gated delta rule that sum over the values, chunk by chunk on
// the tensor cores (tcgen05), from the states before each chunk (S_0), their gradients
// behind it (dS), E and dR as the chains left them (formulas: la_gated_simt.cu,
// notation: la_gated_mma.cuh):
//   N_tj = -D_tj (dR_t.E_j) (j < t),   W_tj = scale D_tj (dO_t.E_j) (j <= t),
//   dK = -e^G (dR S_0^T) + beta (e^{G_C-G} E dS^T + N^T K + W^T Q) + (N beta) K
//   dQ = scale e^G (dO S_0^T) + (W beta) K
// Every sum that dbeta and dg want is a product of a row with k or q:
//   dbeta_t = k_t.(e^{G_C-G} E dS^T + N^T K + W^T Q)_t
//   dG_t = q_t.dQ_t + k_t.(-e^G dR S_0^T + (N beta) K)_t - beta_t dbeta_t,
// plus, at the chunk's end, sum_t beta_t k_t.(e^{G_C-G} E dS^T)_t + e^{G_C} S_0.dS; dg
// is the sum from each token to the end. A pair (t, j) adds what it takes away in that
// sum, once from row t and once from column j, and where keys are alike the others cancel
// too: S_0, dS, E, dR, N, W and N beta, W beta are bf16 high and low parts, a product's lo lo left
// out (rounded once each, dg was off by 3e-3 of its two-norm with independent keys, by up to
// 1.5e-1 with cosines of 0.9 between them).
// Products (M = 128, A and B in shared memory with the 128-byte swizzle, fp32 in
// tensor memory; a lane is a token's row: lanes 0-63 of dK, 64-127 of dQ):
//   1. [dR; dO] E^T                 [128 x 64], the low part of dR in columns of its own,
//   2. [dR; dO] S_0^T, [E; .] dS^T  [128 x DK]  since dO has none
//   3. [N; W] beta K, [N; W]^T [K; Q]
// (lanes 64-127 of what sums dR's low part, E dS^T and the transposed product are unused).
//
// Bound: HBM (240 KB a chunk and head at d = 128, the two states 128 of them: 150 us for 64
// heads of 4096 tokens) and the way from load to product to product of one CTA of 16 warps per
// SM, which goes through the chunks (276 us; the products have 5400 of a chunk's 20000 cycles).
// A key head's heads of values follow each other, so that dQ and dK of shared heads are summed
// in registers, in a fixed order. The states come in pieces of 64 values, the next head's
// while N and W are multiplied; its rows then take the place of N and W.
#include "la_gated_mma.cuh"

namespace la {

namespace {

using namespace gmma;
using namespace sm100;

constexpr int NT = 512;
constexpr uint64_t kWaitNs = 2000000000ull;       // bound of every wait for the tensor cores

// 32 lanes x 16 consecutive 32-bit columns of tensor memory.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

template <int DK, int DV>
struct GradSmem {
  // Boxes of 64 columns. Rows [E hi; E lo; dR lo; dR hi; dO]: what product takes as its 128
  // rows starts at any of them.
  static constexpr int KBOX = 128 * 128, RBOX = 320 * 128;
  static constexpr int KQB = (DK / 64) * KBOX;       // [K; Q]
  static constexpr int ROWB = (DV / 64) * RBOX;
  static constexpr int kEh = 0, kEl = 64 * 128, kRl = 128 * 128, kRh = 192 * 128;
  // a piece of a state: 64 values of its high and of its low part, rows dv
  static constexpr int PART = (DK / 64) * 8192, PIECE = 2 * PART;
  static constexpr int NP = 2 * (DV / 64);           // pieces a head: S_0, dS, S_0, dS
  // over a head's rows after step 2: [N; W] high and low, [N; W] beta high and low
  static constexpr int TILE = 16384, WSIZE = 4 * TILE;
  static constexpr int KQ = 0;
  static constexpr int ROWS = KQ + KQB;
  static constexpr int PIECES = ROWS + (ROWB > WSIZE ? ROWB : WSIZE);
  static constexpr int VECB = 5 * C * 4;             // e^G, e^{G_C-G}, beta, G high and low; two heads'
  static constexpr int REST = 4096 + 2 * VECB + 128;
  static constexpr int SLOTS = PIECES + NP * PIECE + REST <= 227 * 1024 ? NP : 3;
  static constexpr int SUMS = PIECES + SLOTS * PIECE;         // the rows' sums
  static constexpr int VECS = SUMS + 4096;
  static constexpr int CTRL = VECS + 2 * VECB;       // barriers, tensor memory's address, a flag, 16 sums
  static constexpr int TOTAL = CTRL + 128;
  // columns of tensor memory: dR hi and dO, dR lo times S_0; E dS^T; the same two times E; step 3
  static constexpr int D1 = 0, D1B = 128, D2 = 256, D3 = 384, D3B = 448, D5A = 384, D5B = 128;
  static_assert(TOTAL <= 227 * 1024, "shared memory");
  static_assert(SLOTS == NP || NP == 4, "the fourth piece takes the first one's place");
};

struct GradArgs {
  const __nv_bfloat16* q; const __nv_bfloat16* k; const __nv_bfloat16* dout; const __nv_bfloat16* dr;
  ChainOut c;
  const uint8_t* rec;
  const int4* chunks;                                // of every slot: its batch entry, first row, number of tokens
  __nv_bfloat16* dq; __nv_bfloat16* dk; __nv_bfloat16* dg; __nv_bfloat16* dbeta;
  int Hk, H, N;
  unsigned units;                                    // chunk slots x key heads
  float scale;
  int* status;
  int stall;                             // for tests: the first product never counts as done
};

struct Unit {
  unsigned u;
  int slot, hk, b, row, n;
};

// 16-byte piece c of row r in boxes of 64 columns
__device__ __forceinline__ uint32_t box_at(int r, int c, int box) {
  return (uint32_t)((c >> 3) * box + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// 64 rows of CH pieces into rows r0 .. of boxes, n of them there, the rest zeros
template <int CH>
__device__ __forceinline__ void load_box(uint32_t dst, int r0, int box, const __nv_bfloat16* src, int n, int tid) {
#pragma unroll
  for (int i = 0; i < C * CH / NT; ++i) {
    const int j = tid + i * NT, r = j / CH, c = j % CH;
    cp16(dst + box_at(r0 + r, c, box), src + (r < n ? r : 0) * (CH * 8) + c * 8, r < n);
  }
}

template <int DK, int DV>
__global__ void __launch_bounds__(NT, 1)
gated_grads_tc_kernel(const GradArgs p) {
  using L = GradSmem<DK, DV>;
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int KCH = DK / 8, VCH = DV / 8, HC = DK / 4;     // HC: columns of a warp's quarter
  constexpr int FIRST = L::SLOTS < L::NP ? L::SLOTS : L::NP;  // pieces asked for ahead
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_addr(smem);
  const int group = p.H / p.Hk;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::CTRL);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::CTRL + 40);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::CTRL + 44);
  float* dots = reinterpret_cast<float*>(smem + L::CTRL + 64);

  auto unit_at = [&](unsigned u) {                   // the next unit with tokens from u on
    Unit x;
    for (;; u += gridDim.x) {
      x.u = u;
      if (u >= p.units) break;
      x.slot = (int)(u / (unsigned)p.Hk);
      x.hk = (int)(u % (unsigned)p.Hk);
      const int4 c = __ldg(p.chunks + x.slot);
      x.b = c.x; x.row = c.y; x.n = c.z;
      if (x.n > 0) break;
    }
    return x;
  };
  auto load_keys = [&](const Unit& x) {
    const long long r = (((long long)x.b * p.Hk + x.hk) * p.N + x.row) * DK;
    load_box<KCH>(base + L::KQ, 0, L::KBOX, p.k + r, x.n, tid);
    load_box<KCH>(base + L::KQ, 64, L::KBOX, p.q + r, x.n, tid);
    cp_commit();
  };
  auto load_rows = [&](const Unit& x, int hh, int buf) {
    const int h = x.hk * group + hh;
    const long long r = (((long long)x.b * p.H + h) * p.N + x.row) * DV;
    const __nv_bfloat16* const src[5] = {p.c.e, p.c.e_lo, p.c.dr_lo, p.dr, p.dout};
#pragma unroll
    for (int i = 0; i < 5; ++i) load_box<VCH>(base + L::ROWS, 64 * i, L::RBOX, src[i] + r, x.n, tid);
    const uint8_t* rec = p.rec + ((long long)x.slot * p.H + h) * REC_BWD;
    load_bytes<VEC, NT>(base + L::VECS + buf * L::VECB, rec + OFF_VEC, tid);
    load_bytes<2 * C * 4, NT>(base + L::VECS + buf * L::VECB + VEC, rec + OFF_SUMS, tid);
    cp_commit();
  };
  // piece j of a head (S_0 or dS, values 64 (j / 2) ..), in slot (turn + j) % SLOTS
  auto at_piece = [&](unsigned turn, int j) { return L::PIECES + (int)((turn + j) % L::SLOTS) * L::PIECE; };
  auto load_piece = [&](const Unit& x, int hh, unsigned turn, int j) {
    const long long at = (((long long)x.slot * p.H + x.hk * group + hh) * DV + 64 * (j >> 1)) * DK;
    const __nv_bfloat16* hi = ((j & 1) ? p.c.dstates : p.c.states) + at;
    const __nv_bfloat16* lo = ((j & 1) ? p.c.dstates_lo : p.c.states_lo) + at;
    const uint32_t to = base + at_piece(turn, j);
#pragma unroll
    for (int i = 0; i < 64 * KCH / NT; ++i) {
      const int e = tid + i * NT;
      const uint32_t off = box_at(e / KCH, e % KCH, 8192);
      cp16(to + off, hi + e * 8, true);
      cp16(to + L::PART + off, lo + e * 8, true);
    }
    cp_commit();
  };

  Unit x = unit_at(blockIdx.x);
  if (x.u >= p.units) return;
  int hh = 0;
  load_keys(x);
  load_rows(x, 0, 0);
  for (int j = 0; j < FIRST; ++j) load_piece(x, 0, 0, j);
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) mbar_init(&bars[i], i == 0 && p.stall ? 2 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;

  const int quad = warp & 3, part = warp >> 2, row = 32 * quad + lane;
  const bool kside = quad < 2;                       // rows of dK; else of dQ
  const bool issuer = tid == NT - 32;                // of products: a thread of the side with fewer results to read
  const int t = row & 63;
  const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
  uint8_t* wt = smem + L::ROWS;
  float acc[HC];
  bool ok = true;
  int nhead = 0;
  unsigned turn = 0;
  // One thread's: the products with piece j, accumulated over the pieces.
  auto products = [&](int j) {
    constexpr uint32_t id = make_idesc_bf16(128, DK, false, true);      // the states' rows are the sum's index
    const uint32_t rows = base + L::ROWS + (j >> 1) * L::RBOX;
    const uint64_t hi = make_sdesc(base + at_piece(turn, j), 8192, 1024, kSwizzle128B);
    const uint64_t lo = sdesc_add(hi, L::PART);
    const uint64_t a = make_sdesc(rows + ((j & 1) ? L::kEh : L::kRh), 16, 1024, kSwizzle128B);
    const uint64_t al = make_sdesc(rows + ((j & 1) ? L::kEl : L::kRl), 16, 1024, kSwizzle128B);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t d = tmem + ((j & 1) ? L::D2 : L::D1), dl = (j & 1) ? d : tmem + L::D1B;
      const bool more = j > 1 || k > 0;
      mma_ss(d, sdesc_add(a, k * 32), sdesc_add(hi, k * 2048), id, more);
      mma_ss(d, sdesc_add(a, k * 32), sdesc_add(lo, k * 2048), id, true);
      mma_ss(dl, sdesc_add(al, k * 32), sdesc_add(hi, k * 2048), id, (j & 1) ? true : more);
    }
  };
  // S_0 . dS over values 64 i .., high times high and what that leaves out
  auto dot_of = [&](int i) {
    float d = 0.f;
    auto add8 = [&](const uint4& a, const uint4& b) {
      d = fmaf(low_half(a.x), low_half(b.x), fmaf(high_half(a.x), high_half(b.x), d));
      d = fmaf(low_half(a.y), low_half(b.y), fmaf(high_half(a.y), high_half(b.y), d));
      d = fmaf(low_half(a.z), low_half(b.z), fmaf(high_half(a.z), high_half(b.z), d));
      d = fmaf(low_half(a.w), low_half(b.w), fmaf(high_half(a.w), high_half(b.w), d));
    };
    const uint8_t *s0 = smem + at_piece(turn, 2 * i), *ds = smem + at_piece(turn, 2 * i + 1);
#pragma unroll
    for (int e = 0; e < L::PART / 16 / NT; ++e) {
      const int at = (tid + e * NT) * 16;
      const uint4 a = *reinterpret_cast<const uint4*>(s0 + at), al = *reinterpret_cast<const uint4*>(s0 + L::PART + at);
      const uint4 b = *reinterpret_cast<const uint4*>(ds + at), bl = *reinterpret_cast<const uint4*>(ds + L::PART + at);
      add8(a, b);
      add8(al, b);
      add8(a, bl);
    }
    return d;
  };
  while (true) {
    const uint32_t parity = nhead & 1;
    const float* vec = reinterpret_cast<const float*>(smem + L::VECS + parity * L::VECB);
    const float *EG = vec, *EC = vec + C, *BT = vec + 2 * C, *GS = vec + 3 * C, *GL = vec + 4 * C;
    // the next head, or the next chunk's first
    Unit nx = x;
    int nh = hh + 1;
    if (nh == group) {
      nx = unit_at(x.u + gridDim.x);
      nh = 0;
    }
    const bool more = nx.u < p.units;
    cp_wait<0>();
    fence_proxy_async_smem();
    __syncthreads();
    if (issuer) {
      tc_fence_after();
      if (FIRST < L::NP) {                           // its slot is wanted first
        products(0);
        tc_commit(&bars[3]);
      }
      // 1. [dR; dO] E^T
      constexpr uint32_t id = make_idesc_bf16(128, 64, false, false);
      const uint64_t a = make_sdesc(base + L::ROWS + L::kRh, 16, 1024, kSwizzle128B);
      const uint64_t al = make_sdesc(base + L::ROWS + L::kRl, 16, 1024, kSwizzle128B);
      const uint64_t b = make_sdesc(base + L::ROWS + L::kEh, 16, 1024, kSwizzle128B);
      const uint64_t bl = make_sdesc(base + L::ROWS + L::kEl, 16, 1024, kSwizzle128B);
#pragma unroll
      for (int k = 0; k < DV / 16; ++k) {
        const uint32_t off = (k >> 2) * L::RBOX + (k & 3) * 32;
        mma_ss(tmem + L::D3, sdesc_add(a, off), sdesc_add(b, off), id, k > 0);
        mma_ss(tmem + L::D3, sdesc_add(a, off), sdesc_add(bl, off), id, true);
        mma_ss(tmem + L::D3B, sdesc_add(al, off), sdesc_add(b, off), id, k > 0);
      }
      tc_commit(&bars[0]);
      // 2. with the states
      if (FIRST == L::NP) {
        for (int j = 0; j < FIRST; ++j) products(j);
        tc_commit(&bars[1]);
      }
    }
    float dot0 = dot_of(0);
    if (FIRST < L::NP) {
      ok = ok && mbar_wait(&bars[3], parity, abort_flag, kWaitNs);
      __syncthreads();                               // (all have read it, too)
      load_piece(x, hh, turn, FIRST);
      if (issuer)
        for (int j = 1; j < FIRST; ++j) products(j);
    }
    // N or W of this row, columns j = 16 part ..
    const float eg = EG[t], ec = EC[t], bt = BT[t], gs = GS[t], gl = GL[t];
    float nw[16];
    ok = ok && mbar_wait(&bars[0], parity, abort_flag, kWaitNs);
    tc_fence_after();
    {
      uint32_t v[16], w[16];
      tmem_ld16(lanes + L::D3 + 16 * part, v);
      if (kside) tmem_ld16(lanes + L::D3B + 16 * part, w);
      tmem_ld_wait();
      const float f = kside ? -1.f : p.scale;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j0 = 16 * part + 4 * i;
        const float4 g4 = *reinterpret_cast<const float4*>(GS + j0), l4 = *reinterpret_cast<const float4*>(GL + j0);
        const float gj[4] = {g4.x, g4.y, g4.z, g4.w}, lj[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float d;
          asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"((gs - gj[e]) + (gl - lj[e])));
          const float y = f * (kside ? __uint_as_float(v[4 * i + e]) + __uint_as_float(w[4 * i + e]) : __uint_as_float(v[4 * i + e]));
          nw[4 * i + e] = j0 + e < t ? d * y : j0 + e == t && !kside ? y : 0.f;
        }
      }
    }
    if (FIRST < L::NP) {
      cp_wait<0>();
      fence_proxy_async_smem();
      __syncthreads();
      if (issuer) {
        products(FIRST);
        tc_commit(&bars[1]);
      }
      dot0 += dot_of(1);
    } else if (L::NP == 4) {
      dot0 += dot_of(1);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot0 += __shfl_xor_sync(0xffffffffu, dot0, o);
    if (lane == 0) dots[warp] = dot0;
    ok = ok && mbar_wait(&bars[1], parity, abort_flag, kWaitNs);
    tc_fence_after();
    if (hh == 0) {
#pragma unroll
      for (int i = 0; i < HC; ++i) acc[i] = 0.f;
    }
    // This row of K or Q against the products: sums of the row's products, factors after
    // the sums. dR's low part times S_0 first, whose columns step 3 takes.
    float d1 = 0.f, d3 = 0.f, d5 = 0.f, d2 = 0.f;
    const uint8_t* xr = smem + L::KQ;
    const float f1 = kside ? -eg : p.scale * eg, f3 = bt * ec;
    auto against = [&](uint32_t cols, float f, float& sum) {
#pragma unroll
      for (int c0 = 0; c0 < HC; c0 += 16) {
        uint32_t v[16];
        tmem_ld16(lanes + cols + part * HC + c0, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 r4 = *reinterpret_cast<const uint4*>(xr + box_at(row, (part * HC + c0) / 8 + i, L::KBOX));
          const uint32_t r[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = __uint_as_float(v[8 * i + e]);
            acc[c0 + 8 * i + e] = fmaf(f, a, acc[c0 + 8 * i + e]);
            sum = fmaf((e & 1) ? high_half(r[e >> 1]) : low_half(r[e >> 1]), a, sum);
          }
        }
      }
    };
    if (kside) against(L::D1B, f1, d1);
    __syncthreads();                                 // (E, dR, dO and the states have been read by all)
    // [N; W] and [N; W] beta by rows, as they are multiplied from both sides
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 bj = *reinterpret_cast<const float2*>(BT + 16 * part + 2 * i);
        split2(nw[2 * i] * (b ? bj.x : 1.f), nw[2 * i + 1] * (b ? bj.y : 1.f), hi[i], lo[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t at = 2 * b * L::TILE + box_at(row, 2 * part + i, 0);
        *reinterpret_cast<uint4*>(wt + at) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
        *reinterpret_cast<uint4*>(wt + L::TILE + at) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (issuer) {
      // 3. [N; W] beta K and [N; W]^T [K; Q]: tokens are the sum's index
      tc_fence_after();
      constexpr uint32_t id = make_idesc_bf16(128, DK, false, true), idt = make_idesc_bf16(128, DK, true, true);
      const uint64_t dkq = make_sdesc(base + L::KQ, L::KBOX, 1024, kSwizzle128B);
#pragma unroll
      for (int lo = 0; lo < 2; ++lo) {
        const uint64_t a = make_sdesc(base + L::ROWS + (2 + lo) * L::TILE, 16, 1024, kSwizzle128B);
        // (rows 64 .. 127 of the transposed: the next tile's, into the unused lanes)
        const uint64_t at = make_sdesc(base + L::ROWS + lo * L::TILE, L::TILE, 1024, kSwizzle128B);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_ss(tmem + L::D5A, sdesc_add(a, k * 32), sdesc_add(dkq, k * 2048), id, lo > 0 || k > 0);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ss(tmem + L::D5B, sdesc_add(at, k * 2048), sdesc_add(dkq, k * 2048), idt, lo > 0 || k > 0);
      }
      tc_commit(&bars[2]);
    }
    if (more)
      for (int j = 0; j < FIRST; ++j) load_piece(nx, nh, turn + L::NP, j);
    against(L::D1, f1, d1);
    if (kside) against(L::D2, f3, d3);
    ok = ok && mbar_wait(&bars[2], parity, abort_flag, kWaitNs);
    tc_fence_after();
    if (more) load_rows(nx, nh, parity ^ 1);         // over N and W
    against(L::D5A, 1.f, d2);
    if (kside) against(L::D5B, bt, d5);
    tc_fence_before();
    float* sums = reinterpret_cast<float*>(smem + L::SUMS);      // [quarter][f1 d1 + d2 of both sides, d3, d5]
    sums[part * 256 + row] = fmaf(f1, d1, d2);
    if (kside) {
      sums[part * 256 + 128 + t] = ec * d3;
      sums[part * 256 + 192 + t] = d5;
    }
    // a wait that gave up: nobody stores, all leave
    if (!__syncthreads_and(ok)) break;
    const int n = x.n;
    // dQ and dK by way of shared memory (over K and Q), so that a warp stores whole rows
    if (hh == group - 1) {
#pragma unroll
      for (int i = 0; i < HC / 8; ++i)
        *reinterpret_cast<uint4*>(smem + L::KQ + box_at(row, part * (HC / 8) + i, L::KBOX)) =
            make_uint4(pack2(acc[8 * i], acc[8 * i + 1]), pack2(acc[8 * i + 2], acc[8 * i + 3]),
                       pack2(acc[8 * i + 4], acc[8 * i + 5]), pack2(acc[8 * i + 6], acc[8 * i + 7]));
      __syncthreads();
    }
    if (warp == 0) {
      // dg and dbeta, two tokens a lane
      float2 v[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        v[z] = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 o = *reinterpret_cast<const float2*>(sums + w * 256 + 64 * z + 2 * lane);
          v[z].x += o.x;
          v[z].y += o.y;
        }
      }
      const float2 b2 = *reinterpret_cast<const float2*>(BT + 2 * lane);
      const float b[2] = {b2.x, b2.y}, s0[2] = {v[0].x + v[1].x, v[0].y + v[1].y}, s3[2] = {v[2].x, v[2].y}, s5[2] = {v[3].x, v[3].y};
      float xg[2], xb[2], ws = lane < NT / 32 ? EG[C - 1] * dots[lane] : 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        xb[e] = s3[e] + s5[e];
        ws += b[e] * s3[e];
        xg[e] = s0[e] - b[e] * xb[e];
      }
      // from each token to the end, and what the end's sum carries (ws) for all
      float s = xg[0] + xg[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, s, o);
        ws += __shfl_xor_sync(0xffffffffu, ws, o);
        if (lane + o < 32) s += y;
      }
      float behind = __shfl_down_sync(0xffffffffu, s, 1);
      if (lane == 31) behind = 0.f;
      const long long at = ((long long)x.b * p.H + x.hk * group + hh) * p.N + x.row;
      const float out[2] = {s + ws, behind + xg[1] + ws};
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * lane + e < n) {
          p.dg[at + 2 * lane + e] = __float2bfloat16_rn(out[e]);
          p.dbeta[at + 2 * lane + e] = __float2bfloat16_rn(xb[e]);
        }
    } else if (hh == group - 1) {
      const long long at = (((long long)x.b * p.Hk + x.hk) * p.N + x.row) * DK;
      for (int i = tid - 32; i < 2 * C * KCH; i += NT - 32) {
        const int r = i / KCH, c = i % KCH;
        if ((r & 63) < n)
          *reinterpret_cast<uint4*>((r < 64 ? p.dk : p.dq) + at + (r & 63) * DK + c * 8) =
              *reinterpret_cast<const uint4*>(smem + L::KQ + box_at(r, c, L::KBOX));
      }
    }
    if (!more) break;
    __syncthreads();                                 // the sums and the rows on their way out have been read
    if (nh == 0) load_keys(nx);
    x = nx; hh = nh;
    turn += L::NP;
    ++nhead;
  }
  // copies and products in flight end before shared and tensor memory are released
  cp_wait<0>();
  if (*abort_flag) {
    if (issuer) {
      mbar_init(&bars[4], 1);
      fence_mbar_init();
      tc_commit(&bars[4]);
      mbar_drain(&bars[4], 0, kWaitNs);
      atomicExch(p.status, (int)LA_ERR_TIMEOUT);
    }
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int DK, int DV>
cudaError_t launch(const GradArgs& p, cudaStream_t stream) {
  auto kern = gated_grads_tc_kernel<DK, DV>;
  const int smem = GradSmem<DK, DV>::TOTAL;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(p.units < kSlots ? p.units : kSlots);
  kern<<<grid, NT, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Parts { size_t rec, chunks, rows, states; };
Parts parts(int B, int H, int N, int dk, int dv, int nseq, bool packed, bool backward) {
  const long long slots = chunk_slots(B, N, nseq, packed, C);
  Parts s;
  s.rec = up256((size_t)slots * H * (backward ? REC_BWD : REC_FWD));
  s.chunks = backward ? up256((size_t)slots * sizeof(int4)) : 0;
  s.rows = up256((size_t)B * H * N * dv * 2);
  s.states = up256((size_t)slots * H * dk * dv * 2);
  return s;
}

}  // namespace

size_t mma_gated_forward_workspace(int B, int H, int N, int dk, int dv, int nseq, bool packed) {
  return parts(B, H, N, dk, dv, nseq, packed, false).rec;
}

size_t mma_gated_backward_workspace(int B, int H, int N, int dk, int dv, int nseq, bool packed) {
  const Parts s = parts(B, H, N, dk, dv, nseq, packed, true);
  return s.rec + s.chunks + 3 * s.rows + 4 * s.states;
}

cudaError_t mma_gated_forward(const GatedArgs& a) {
  const cudaError_t e = gated_prep(a, (uint8_t*)a.workspace, nullptr);
  if (e != cudaSuccess) return e;
  const uint8_t* records = (const uint8_t*)a.workspace;
  if (gated_split_wanted(a, false)) return gated_split_forward(a, records);
  return gated_pair_wanted(a) ? gated_pair_forward(a, records) : gated_chain_forward(a, records);
}

cudaError_t mma_gated_backward(const GatedArgs& a) {
  const Parts s = parts(a.B, a.H, a.N, a.dk, a.dv, a.nseq, a.offsets != nullptr, true);
  uint8_t* ws = (uint8_t*)a.workspace;
  int4* chunks = (int4*)(ws + s.rec);
  uint8_t* at = ws + s.rec + s.chunks;
  auto take = [&](size_t bytes) {
    __nv_bfloat16* x = (__nv_bfloat16*)at;
    at += bytes;
    return x;
  };
  ChainOut o;
  o.e = take(s.rows); o.e_lo = take(s.rows); o.dr_lo = take(s.rows);
  o.states = take(s.states); o.states_lo = take(s.states); o.dstates = take(s.states); o.dstates_lo = take(s.states);
  cudaError_t err = gated_prep(a, ws, chunks);
  if (err != cudaSuccess) return err;
  err = gated_split_wanted(a, true) ? gated_split_backward(a, ws, o) : gated_chain_backward(a, ws, o);
  if (err != cudaSuccess) return err;
  GradArgs p{};
  p.q = (const __nv_bfloat16*)a.q; p.k = (const __nv_bfloat16*)a.k; p.dout = (const __nv_bfloat16*)a.dout;
  p.dr = (const __nv_bfloat16*)a.dv_; p.c = o; p.rec = ws; p.chunks = chunks;
  p.dq = (__nv_bfloat16*)a.dq; p.dk = (__nv_bfloat16*)a.dk_; p.dg = (__nv_bfloat16*)a.dg; p.dbeta = (__nv_bfloat16*)a.dbeta;
  p.Hk = a.Hk; p.H = a.H; p.N = a.N; p.scale = a.scale;
  p.status = device_status_ptr();
  if (p.status == nullptr) return cudaErrorNotReady;
  p.stall = take_gated_timeout_test(1) ? 1 : 0;
  p.units = (unsigned)(chunk_slots(a.B, a.N, a.nseq, a.offsets != nullptr, C) * a.Hk);
  if (p.units == 0) return cudaSuccess;
  if (a.dk == 64) return a.dv == 64 ? launch<64, 64>(p, a.stream) : launch<64, 128>(p, a.stream);
  return a.dv == 64 ? launch<128, 64>(p, a.stream) : launch<128, 128>(p, a.stream);
}

}  // namespace la
