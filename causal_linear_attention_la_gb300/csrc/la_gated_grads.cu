// Gradients of the gated delta rule that sum over the values, chunk by chunk on
// the tensor cores (tcgen05), from the states before each chunk (S_0), their gradients
// behind it (dS), E and dR as the chains left them (formulas: la_gated_simt.cu,
// notation: la_gated_mma.cuh):
//   N_tj = -D_tj (dR_t.E_j) beta_j (j < t),   W_tj = scale D_tj (dO_t.E_j) beta_j (j <= t),
//   dK = -e^G (dR S_0^T) + e^{G_C-G} beta (E dS^T) + N K + N^T K + W^T Q
//   dQ = scale e^G (dO S_0^T) + W K
// Every sum that dbeta and dg want is a product of a row with k or q:
//   dbeta_t = k_t.(e^{G_C-G} E dS^T)_t + k_t.(N^T K + W^T Q)_t / beta_t
//   dG_t = q_t.dQ_t + k_t.(-e^G dR S_0^T + N K)_t - beta_t dbeta_t,
// plus, at the chunk's end, sum_t beta_t k_t.(e^{G_C-G} E dS^T)_t + e^{G_C} S_0.dS; dg
// is the sum from each token to the end. A pair (t, j) adds what it takes away in that
// sum, once from row t and once from column j: both come from the same bf16 values of N and W, so that
// it leaves nothing. (Rounded apart, the pairs' differences were 9e-3 of dg.) Where
// |beta_j| < 2^-30 column j has 2^-30 in its place in N^T and W^T, whose row j
// then counts beta_j 2^30 times (a power of two near the others' sizes: with 2^-100 gradients
// of 1e-9 fell below bf16's normal numbers).
// Products (M = 128, A and B in shared memory with the 128-byte swizzle, fp32 in
// tensor memory; a lane is a token's row: lanes 0-63 of dK, 64-127 of dQ):
//   1. [dR; dO] E^T                 [128 x 64]
//   2. [E; dR] dS^T, [dR; dO] S_0^T [128 x DK]   (lanes 64-127 of the first unused)
//   3. [N; W] K, [N^T W^T] [K; Q]   [128 x DK]   (lanes 64-127 of the second unused)
// 2048 cycles of the tensor pipe at d = 128. Operands are bf16 (one rounding each of S_0, dS,
// E, dR, N and W); sums are fp32.
//
// Bound: HBM (150 KB a chunk and head at d = 128, the two states 64 of them). One
// CTA of 16 warps per SM goes through the chunks; a key head's heads of values follow
// each other, so that dQ and dK of shared heads are summed in registers, in a
// fixed order. The next head's rows are on their way from the start of a head on, its
// states from the end of step 2. (The same products by mma.sync took 282 us for 64
// heads of 4096 tokens: fragments through the shared-memory pipe and barriers.)
#include "la_gated_mma.cuh"

namespace la {

namespace {

using namespace gmma;
using namespace sm100;

constexpr int NT = 512;
constexpr uint64_t kWaitNs = 2000000000ull;       // bound of every wait for the tensor cores
constexpr float kTiny = 9.313225746154785e-10f, kHuge = 1073741824.f;   // 2^-30, 2^30

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
  static constexpr int KBOX = 128 * 128, RBOX = 192 * 128, SBOX = DV * 128;   // boxes of 64 columns
  static constexpr int KQB = (DK / 64) * KBOX;       // [K; Q]
  static constexpr int ROWB = (DV / 64) * RBOX;      // [E; dR; dO]
  static constexpr int SB = (DK / 64) * SBOX;        // a state, rows dv
  static constexpr int KQ = 0;                       // two units'
  static constexpr int ROWS = KQ + 2 * KQB;          // two heads'
  static constexpr int S0 = ROWS + 2 * ROWB;
  static constexpr int DS = S0 + SB;
  // [N; W] 16 KB, [N^T W^T] 16 KB (the product reads the 8 KB behind it as rows that
  // nobody uses), then the rows' sums: over a head's rows after step 2 where they fit
  static constexpr int WSIZE = 32768 + 8192;
  static constexpr bool kOver = ROWB >= WSIZE;
  static constexpr int WEXTRA = DS + SB;
  static constexpr int VECS = WEXTRA + (kOver ? 0 : WSIZE);   // two heads' e^G, e^{G_C-G}, beta, G high and low
  static constexpr int CTRL = VECS + 2 * 5 * C * 4;           // barriers, tensor memory's address, flags, 16 sums
  static constexpr int TOTAL = CTRL + 128;
  static constexpr int D1 = 0, D2 = 128, D5A = 256, D5B = 384, D3 = 384;      // columns of tensor memory
  static_assert(TOTAL <= 227 * 1024, "shared memory");
};

struct GradArgs {
  const __nv_bfloat16* q; const __nv_bfloat16* k; const __nv_bfloat16* dout; const __nv_bfloat16* e;
  const __nv_bfloat16* dr; const __nv_bfloat16* states; const __nv_bfloat16* dstates;
  const __nv_bfloat16* states_lo; const __nv_bfloat16* dstates_lo;     // or null
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
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_addr(smem);
  const int group = p.H / p.Hk;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::CTRL);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::CTRL + 32);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::CTRL + 40);
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
  auto load_rows = [&](const Unit& x, int hh, int buf, int kbuf) {
    if (hh == 0) {
      const long long r = (((long long)x.b * p.Hk + x.hk) * p.N + x.row) * DK;
      const uint32_t to = base + L::KQ + kbuf * L::KQB;
      load_box<KCH>(to, 0, L::KBOX, p.k + r, x.n, tid);
      load_box<KCH>(to, 64, L::KBOX, p.q + r, x.n, tid);
    }
    const int h = x.hk * group + hh;
    const long long r = (((long long)x.b * p.H + h) * p.N + x.row) * DV;
    const uint32_t to = base + L::ROWS + buf * L::ROWB;
    load_box<VCH>(to, 0, L::RBOX, p.e + r, x.n, tid);
    load_box<VCH>(to, 64, L::RBOX, p.dr + r, x.n, tid);
    load_box<VCH>(to, 128, L::RBOX, p.dout + r, x.n, tid);
    const uint8_t* rec = p.rec + ((long long)x.slot * p.H + h) * REC_BWD;
    load_bytes<VEC, NT>(base + L::VECS + buf * 5 * C * 4, rec + off_vec(true), tid);
    load_bytes<2 * C * 4, NT>(base + L::VECS + buf * 5 * C * 4 + VEC, rec + OFF_SUMS, tid);
    cp_commit();
  };
  auto load_states = [&](const Unit& x, int hh) {
    const long long at = ((long long)x.slot * p.H + x.hk * group + hh) * DK * DV;
#pragma unroll
    for (int i = 0; i < DV * KCH / NT; ++i) {
      const int j = tid + i * NT;
      cp16(base + L::DS + box_at(j / KCH, j % KCH, L::SBOX), p.dstates + at + j * 8, true);
      cp16(base + L::S0 + box_at(j / KCH, j % KCH, L::SBOX), p.states + at + j * 8, true);
    }
    cp_commit();
  };

  Unit x = unit_at(blockIdx.x);
  if (x.u >= p.units) return;
  int hh = 0, buf = 0, kbuf = 0;
  load_rows(x, 0, 0, 0);
  load_states(x, 0);
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) mbar_init(&bars[i], i == 0 && p.stall ? 2 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;

  const int quad = warp & 3, part = warp >> 2, row = 32 * quad + lane;
  const bool kside = quad < 2;                       // rows of dK; else of dQ
  const int t = row & 63;
  const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
  float acc[HC];
  bool ok = true;
  int nhead = 0;
  while (true) {
    const uint32_t kq = base + L::KQ + kbuf * L::KQB, rows = base + L::ROWS + buf * L::ROWB;
    const float* vec = reinterpret_cast<const float*>(smem + L::VECS + buf * 5 * C * 4);
    const float *EG = vec, *EC = vec + C, *BT = vec + 2 * C, *GS = vec + 3 * C, *GL = vec + 4 * C;
    const uint32_t parity = nhead & 1;
    uint8_t* wt = smem + (L::kOver ? L::ROWS + buf * L::ROWB : L::WEXTRA);
    const uint32_t wa = smem_addr(wt);

    cp_wait<1>();                                    // this head's rows; its states may be on their way
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      // 1. [dR; dO] E^T
      tc_fence_after();
      constexpr uint32_t id = make_idesc_bf16(128, 64, false, false);
      const uint64_t da = make_sdesc(rows + 64 * 128, 16, 1024, kSwizzle128B), db = make_sdesc(rows, 16, 1024, kSwizzle128B);
#pragma unroll
      for (int k = 0; k < DV / 16; ++k) {
        const uint32_t off = (k >> 2) * L::RBOX + (k & 3) * 32;
        mma_ss(tmem + L::D3, sdesc_add(da, off), sdesc_add(db, off), id, k > 0);
      }
      tc_commit(&bars[0]);
    }
    // the next head, or the next chunk's first
    Unit nx = x;
    int nh = hh + 1, nk = kbuf;
    if (nh == group) {
      nx = unit_at(x.u + gridDim.x);
      nh = 0;
      nk ^= 1;
    }
    const bool more = nx.u < p.units;
    if (more) load_rows(nx, nh, buf ^ 1, nk);
    if (more) cp_wait<1>(); else cp_wait<0>();       // this head's states
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      // 2. [E; dR] dS^T and [dR; dO] S_0^T: the states' rows are the sum's index
      constexpr uint32_t id = make_idesc_bf16(128, DK, false, true);
      const uint64_t de = make_sdesc(rows, 16, 1024, kSwizzle128B), dr = make_sdesc(rows + 64 * 128, 16, 1024, kSwizzle128B);
      const uint64_t ds = make_sdesc(base + L::DS, L::SBOX, 1024, kSwizzle128B);
      const uint64_t s0 = make_sdesc(base + L::S0, L::SBOX, 1024, kSwizzle128B);
#pragma unroll
      for (int k = 0; k < DV / 16; ++k)
        mma_ss(tmem + L::D2, sdesc_add(de, (k >> 2) * L::RBOX + (k & 3) * 32), sdesc_add(ds, k * 2048), id, k > 0);
#pragma unroll
      for (int k = 0; k < DV / 16; ++k)
        mma_ss(tmem + L::D1, sdesc_add(dr, (k >> 2) * L::RBOX + (k & 3) * 32), sdesc_add(s0, k * 2048), id, k > 0);
      tc_commit(&bars[1]);
    }
    float dot0 = 0.f;                                // S_0 . dS
    auto add8 = [&](const uint4& a, const uint4& b) {
      dot0 = fmaf(low_half(a.x), low_half(b.x), fmaf(high_half(a.x), high_half(b.x), dot0));
      dot0 = fmaf(low_half(a.y), low_half(b.y), fmaf(high_half(a.y), high_half(b.y), dot0));
      dot0 = fmaf(low_half(a.z), low_half(b.z), fmaf(high_half(a.z), high_half(b.z), dot0));
      dot0 = fmaf(low_half(a.w), low_half(b.w), fmaf(high_half(a.w), high_half(b.w), dot0));
    };
#pragma unroll 4
    for (int i = 0; i < DK * DV / 8 / NT; ++i)
      add8(*reinterpret_cast<const uint4*>(smem + L::S0 + (tid + i * NT) * 16),
           *reinterpret_cast<const uint4*>(smem + L::DS + (tid + i * NT) * 16));
    if (p.states_lo != nullptr) {
      const long long at = ((long long)x.slot * p.H + x.hk * group + hh) * DK * DV;
#pragma unroll 2
      for (int i = 0; i < DV * KCH / NT; ++i) {
        const int j = tid + i * NT;
        const uint32_t pos = box_at(j / KCH, j % KCH, L::SBOX);
        const uint4 a = *reinterpret_cast<const uint4*>(p.states_lo + at + j * 8);
        const uint4 b = *reinterpret_cast<const uint4*>(p.dstates_lo + at + j * 8);
        add8(*reinterpret_cast<const uint4*>(smem + L::S0 + pos), b);
        add8(a, *reinterpret_cast<const uint4*>(smem + L::DS + pos));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot0 += __shfl_xor_sync(0xffffffffu, dot0, o);
    if (lane == 0) dots[warp] = dot0;
    // N or W of this row, columns j = 16 part .., as bf16
    const float eg = EG[t], ec = EC[t], bt = BT[t], gs = GS[t], gl = GL[t];
    uint32_t w16[8];
    ok = ok && mbar_wait(&bars[0], parity, abort_flag, kWaitNs);
    tc_fence_after();
    {
      uint32_t v[16];
      tmem_ld16(lanes + L::D3 + 16 * part, v);
      tmem_ld_wait();
      const float f = kside ? -1.f : p.scale;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j0 = 16 * part + 4 * i;
        const float4 g4 = *reinterpret_cast<const float4*>(GS + j0), l4 = *reinterpret_cast<const float4*>(GL + j0);
        const float4 b4 = *reinterpret_cast<const float4*>(BT + j0);
        const float gj[4] = {g4.x, g4.y, g4.z, g4.w}, lj[4] = {l4.x, l4.y, l4.z, l4.w}, bj[4] = {b4.x, b4.y, b4.z, b4.w};
        float a[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float d;
          asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"((gs - gj[e]) + (gl - lj[e])));
          const float w = f * bj[e] * __uint_as_float(v[4 * i + e]);
          a[e] = j0 + e < t ? d * w : j0 + e == t && !kside ? w : 0.f;
        }
        w16[2 * i] = pack2(a[0], a[1]);
        w16[2 * i + 1] = pack2(a[2], a[3]);
      }
    }
    ok = ok && mbar_wait(&bars[1], parity, abort_flag, kWaitNs);
    tc_fence_after();
    // (a barrier: the states, E, dR and dO have been read by all)
    const bool tiny = __syncthreads_or(fabsf(bt) < kTiny);
    if (more) load_states(nx, nh);
    // [N; W] by rows, [N^T W^T] by columns
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint4*>(wt + box_at(row, 2 * part + i, 0)) =
          make_uint4(w16[4 * i], w16[4 * i + 1], w16[4 * i + 2], w16[4 * i + 3]);
    if (tiny) {
      uint32_t v[16];
      tmem_ld16(lanes + L::D3 + 16 * part, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = 16 * part + i;
        if (!(fabsf(BT[j]) < kTiny)) continue;
        float d;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"((gs - GS[j]) + (gl - GL[j])));
        const float w = (kside ? -kTiny : kTiny * p.scale) * __uint_as_float(v[i]);
        const uint32_t one = pack2(j < t ? d * w : j == t && !kside ? w : 0.f, 0.f);
        w16[i >> 1] = (i & 1) ? (w16[i >> 1] & 0xffffu) | (one << 16) : (w16[i >> 1] & 0xffff0000u) | one;
      }
    }
    {
      uint8_t* to = wt + 16384 + (kside ? 0 : 8192) + 2 * (t & 7);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = 16 * part + i;
        const uint32_t w = w16[i >> 1];
        *reinterpret_cast<uint16_t*>(to + j * 128 + (((t >> 3) ^ (j & 7)) << 4)) = (uint16_t)((i & 1) ? w >> 16 : w);
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      // 3. [N; W] K and [N^T W^T] [K; Q]: tokens are the sum's index
      tc_fence_after();
      constexpr uint32_t id = make_idesc_bf16(128, DK, false, true);
      const uint64_t dw = make_sdesc(wa, 16, 1024, kSwizzle128B), dt = make_sdesc(wa + 16384, 16, 1024, kSwizzle128B);
      const uint64_t dkq = make_sdesc(kq, L::KBOX, 1024, kSwizzle128B);
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_ss(tmem + L::D5A, sdesc_add(dw, k * 32), sdesc_add(dkq, k * 2048), id, k > 0);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma_ss(tmem + L::D5B, sdesc_add(dt, (k >> 2) * 8192 + (k & 3) * 32), sdesc_add(dkq, k * 2048), id, k > 0);
      tc_commit(&bars[2]);
    }
    // this row of K or Q against what has come so far
    if (hh == 0) {
#pragma unroll
      for (int i = 0; i < HC; ++i) acc[i] = 0.f;
    }
    // (sums of the row's products, factors after the sums)
    float d1 = 0.f, d3 = 0.f, d5 = 0.f, d2 = 0.f;
    const uint8_t* xr = smem + (kq - base);
    const float f1 = kside ? -eg : p.scale * eg, f3 = bt * ec;
#pragma unroll
    for (int c0 = 0; c0 < HC; c0 += 16) {
      uint32_t v[16], w[16];
      tmem_ld16(lanes + L::D1 + part * HC + c0, v);
      if (kside) tmem_ld16(lanes + L::D2 + part * HC + c0, w);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 r4 = *reinterpret_cast<const uint4*>(xr + box_at(row, (part * HC + c0) / 8 + i, L::KBOX));
        const uint32_t r[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xv = (e & 1) ? high_half(r[e >> 1]) : low_half(r[e >> 1]), a = __uint_as_float(v[8 * i + e]);
          float& y = acc[c0 + 8 * i + e];
          y = fmaf(f1, a, y);
          d1 = fmaf(xv, a, d1);
          if (kside) {
            const float b = __uint_as_float(w[8 * i + e]);
            y = fmaf(f3, b, y);
            d3 = fmaf(xv, b, d3);
          }
        }
      }
    }
    ok = ok && mbar_wait(&bars[2], parity, abort_flag, kWaitNs);
    tc_fence_after();
    const float f5 = fabsf(bt) < kTiny ? bt * kHuge : 1.f;
#pragma unroll
    for (int c0 = 0; c0 < HC; c0 += 16) {
      uint32_t v[16], w[16];
      tmem_ld16(lanes + L::D5A + part * HC + c0, v);
      if (kside) tmem_ld16(lanes + L::D5B + part * HC + c0, w);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 r4 = *reinterpret_cast<const uint4*>(xr + box_at(row, (part * HC + c0) / 8 + i, L::KBOX));
        const uint32_t r[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xv = (e & 1) ? high_half(r[e >> 1]) : low_half(r[e >> 1]), a = __uint_as_float(v[8 * i + e]);
          float& y = acc[c0 + 8 * i + e];
          y += a;
          d2 = fmaf(xv, a, d2);
          if (kside) {
            const float b = __uint_as_float(w[8 * i + e]);
            y = fmaf(f5, b, y);
            d5 = fmaf(xv, b, d5);
          }
        }
      }
    }
    tc_fence_before();
    float* sums = reinterpret_cast<float*>(wt + 32768);        // [quarter][d1 of both sides, d3, d5]
    sums[part * 256 + row] = fmaf(f1, d1, d2);
    if (kside) {
      sums[part * 256 + 128 + t] = ec * d3;
      sums[part * 256 + 192 + t] = d5;
    }
    // a wait that gave up: nobody stores, all leave
    if (!__syncthreads_and(ok)) break;
    const int n = x.n;
    // dQ and dK by way of shared memory (over N and W), so that a warp stores whole rows
    if (hh == group - 1) {
#pragma unroll
      for (int i = 0; i < HC / 8; ++i)
        *reinterpret_cast<uint4*>(wt + box_at(row, part * (HC / 8) + i, 16384)) =
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
        const bool small = fabsf(b[e]) < kTiny;
        xb[e] = s3[e] + __fdividef(s5[e], small ? kTiny : b[e]);
        const float w = b[e] * s3[e];
        ws += w;
        xg[e] = s0[e] - w - (small ? b[e] * kHuge * s5[e] : s5[e]);
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
              *reinterpret_cast<const uint4*>(wt + box_at(r, c, 16384));
      }
    }
    if (!more) break;
    x = nx; hh = nh; kbuf = nk; buf ^= 1;
    ++nhead;
  }
  // copies and products in flight end before shared and tensor memory are released
  cp_wait<0>();
  if (*abort_flag) {
    if (tid == 0) {
      mbar_init(&bars[3], 1);
      fence_mbar_init();
      tc_commit(&bars[3]);
      mbar_drain(&bars[3], 0, kWaitNs);
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

// A chunk's and head's dg share one product, e^{G_C} S_0.dS, of dk dv terms: with
// both factors rounded to bf16 it is off by about 2^-9 of the root of its squared terms'
// sum, as much as the product itself where they cancel. Over many chunks and
// heads that stays near 2^-9 of dg's 2-norm; with few of them the states' low parts are
// kept for it too: largest of 12 draws 4.5e-3 of dg's norm against 5.6e-3 at 4 heads
// of 512 tokens (32 chunks), the same 3.7e-3 at 64 chunks, where it costs a tenth of the time.
constexpr long long kFewChunks = 64;

struct Parts { size_t rec, e, states, chunks; bool lo; };
Parts parts(int B, int H, int N, int dk, int dv, int nseq, bool packed, bool backward) {
  const long long slots = chunk_slots(B, N, nseq, packed, C);
  Parts s;
  s.rec = up256((size_t)slots * H * (backward ? REC_BWD : REC_FWD));
  s.chunks = backward ? up256((size_t)slots * sizeof(int4)) : 0;
  s.e = up256((size_t)B * H * N * dv * 2);
  s.states = up256((size_t)slots * H * dk * dv * 2);
  // (the size query does not know whether one batch entry is packed)
  s.lo = chunk_slots(B, N, nseq, B == 1, C) * H <= kFewChunks;
  return s;
}

}  // namespace

size_t mma_gated_forward_workspace(int B, int H, int N, int dk, int dv, int nseq, bool packed) {
  return parts(B, H, N, dk, dv, nseq, packed, false).rec;
}

size_t mma_gated_backward_workspace(int B, int H, int N, int dk, int dv, int nseq, bool packed) {
  const Parts s = parts(B, H, N, dk, dv, nseq, packed, true);
  return s.rec + s.chunks + s.e + (s.lo ? 4 : 2) * s.states;
}

cudaError_t mma_gated_forward(const GatedArgs& a) {
  const cudaError_t e = gated_prep(a, (uint8_t*)a.workspace, nullptr, true);
  if (e != cudaSuccess) return e;
  const uint8_t* records = (const uint8_t*)a.workspace;
  if (gated_split_wanted(a, false)) return gated_split_forward(a, records);
  return gated_pair_wanted(a) ? gated_pair_forward(a, records) : gated_chain_forward(a, records);
}

cudaError_t mma_gated_backward(const GatedArgs& a) {
  const Parts s = parts(a.B, a.H, a.N, a.dk, a.dv, a.nseq, a.offsets != nullptr, true);
  uint8_t* ws = (uint8_t*)a.workspace;
  int4* chunks = (int4*)(ws + s.rec);
  __nv_bfloat16* e = (__nv_bfloat16*)(ws + s.rec + s.chunks);
  __nv_bfloat16* st[4];                // states, their gradients, low parts of both
  for (int i = 0; i < 4; ++i) st[i] = i < 2 || s.lo ? (__nv_bfloat16*)(ws + s.rec + s.chunks + s.e + i * s.states) : nullptr;
  cudaError_t err = gated_prep(a, ws, chunks, a.dS0 != nullptr);
  if (err != cudaSuccess) return err;
  err = gated_split_wanted(a, true) ? gated_split_backward(a, ws, e, st) : gated_chain_backward(a, ws, e, st);
  if (err != cudaSuccess) return err;
  GradArgs p{};
  p.q = (const __nv_bfloat16*)a.q; p.k = (const __nv_bfloat16*)a.k; p.dout = (const __nv_bfloat16*)a.dout; p.e = e;
  p.dr = (const __nv_bfloat16*)a.dv_; p.states = st[0]; p.dstates = st[1]; p.states_lo = st[2]; p.dstates_lo = st[3]; p.rec = ws; p.chunks = chunks;
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
