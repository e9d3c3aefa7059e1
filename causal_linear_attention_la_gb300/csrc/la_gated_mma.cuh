// Gated delta rule on the tensor cores: what its kernels share. Chunks of C
// tokens; in a chunk, with G the running sum of g, D_tj = exp(G_t - G_j) and
// T = (I + tril(D k.k, -1) diag(beta))^-1,
//   E = T (V - e^G K S_0),  U = beta E,
//   O = scale e^G Q S_0 + P U,  P_tj = scale D_tj q_t.k_j (j <= t),
//   S_C = e^{G_C} S_0 + K^T (e^{G_C - G} U)
// and back, from dO and the gradient dS_C behind the chunk,
//   dU = P^T dO + e^{G_C-G} K dS_C,  dR = T^T (beta dU) (= dV),
//   dS_0 = e^{G_C} dS_C + Q^T (scale e^G dO) - K^T (e^G dR).
// T and P depend on no state: a kernel over all chunks writes them once
// (la_gated_prep.cu), as the B fragments of mma.m16n8k16 that the chains take.
//
// mma.sync and not tcgen05.mma for the chains: the state is both the result of
// a chunk's last product and an operand of the next one's first. In registers
// the accumulator of m16n8k16 is laid out as its A operand, so that a warp keeps
// 16 columns of S through all chunks (every column evolves on its own) and goes
// from product to product without a barrier or a trip through tensor memory,
// whose five round trips a chunk (wait, load, split, store, issue; ~0.8 us each as
// measured in the 16-token decode) would be the chain. One warp per sub-core
// keeps its tensor pipe busy: 8 cycles an instruction (measured: 595 TFLOP/s
// on 152 SMs, the same with 1, 2 and 4 warps a sub-core).
//
// Precision: fp32 operands go in as bf16 high and low parts (lo lo is left out: a
// product is off by 2^-15 of itself at most, 2^-18 as a root mean square); q, k, v, dO
// are bf16 as they are; the state itself, its sums and decays are fp32. Rounding what only
// reaches rows of bf16 once would take 232 products of 16 x 8 x 16 a chunk and 16 columns (d = 128)
// in the place of 504, but R, the triangles and the sums over them cancel where keys are
// alike: with cosines of 0.9 between them outputs were off by up to 2e-2 of their two-norm (3.4e-3
// with independent keys), dv and dk by as much, dg by up to 1.5e-1.
#pragma once

#include "la_gated.cuh"
#include "la_tree_ops.cuh"

namespace la {
namespace gmma {

using treeops::ldmatrix4t;
using treeops::low_half;
using treeops::high_half;
using treeops::mma;
using treeops::pack2;
using treeops::split2;

constexpr int C = 64;                      // tokens per chunk
constexpr int NB = 10;                     // 16 x 16 blocks on and below the diagonal
constexpr int FRAG = NB * 512;             // bytes of a triangle's B fragments, bf16
constexpr int VEC = 3 * C * 4;             // e^G, e^{G_C - G}, beta
// A chunk's record: [T lo | T hi | vec | P hi | P lo], backward [T lo | T hi | vec | T^T hi |
// P^T hi | T^T lo | P^T lo | G / log 2 as two fp32].
constexpr int REC_FWD = 4 * FRAG + VEC;
constexpr int OFF_VEC = 2 * FRAG, OFF_REST = OFF_VEC + VEC, OFF_SUMS = OFF_REST + 4 * FRAG;
constexpr int REC_BWD = OFF_SUMS + 2 * C * 4;

__device__ __forceinline__ int block_of(int i, int j) { return i * (i + 1) / 2 + j; }   // row block i >= j

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stmatrix4t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes global -> shared, or zeros
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Byte offset of 16-byte piece c of row r in a tile of rows of CH pieces: the
// pieces of 8 rows that one ldmatrix reads lie in 8 different bank groups.
template <int CH>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  if constexpr (CH >= 8) return (uint32_t)(r * CH + (c ^ (r & 7))) * 16;
  else if constexpr (CH == 4) return (uint32_t)(r * 4 + (c ^ ((r >> 1) & 3))) * 16;
  else return (uint32_t)(r * 2 + (c ^ ((r >> 2) & 1))) * 16;
}

// rows of `CH` pieces, n of them there, the rest zeros
template <int CH, int NT>
__device__ __forceinline__ void load_tile(uint32_t dst, const __nv_bfloat16* src, long long stride, int n, int tid) {
#pragma unroll
  for (int i = 0; i < (C * CH + NT - 1) / NT; ++i) {
    const int j = tid + i * NT, r = j / CH, c = j % CH;
    if ((C * CH) % NT == 0 || j < C * CH)
      cp16(dst + tile_at<CH>(r, c), src + (r < n ? r : 0) * stride + c * 8, r < n);
  }
}

// whether any of an accumulator's values is not a finite number
template <int T>
__device__ __forceinline__ bool not_finite(const float (&x)[T][4]) {
  float bad[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < T; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) bad[e] = fmaf(0.f, x[j][e], bad[e]);
  return (bad[0] + bad[1]) + (bad[2] + bad[3]) != 0.f;
}

// A fragment `a` of tokens 16 jb .. with those behind token t made zero
__device__ __forceinline__ void rows_to(uint32_t (&m)[4], const uint32_t (&a)[4], int jb, int t, int tig) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int j = 16 * jb + 8 * (e >> 1) + 2 * tig;
    m[e] = a[e] & ((j <= t ? 0xffffu : 0u) | (j + 1 <= t ? 0xffff0000u : 0u));
  }
}

// As split2, the high parts as a rounding to bf16 has them (infinite beyond bf16's
// largest number): rows that the caller gets.
__device__ __forceinline__ void split2_out(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2(a, b);
  lo = pack2(a - low_half(hi), b - high_half(hi));
}

// TMA copies: every wait for one is bounded
constexpr uint64_t kWaitNs = 2000000000ull;

// Byte offset of 16-byte piece c of row r in boxes of 64 rows and 64 columns
__device__ __forceinline__ uint32_t box_at(int r, int c) {
  return (uint32_t)((c >> 3) * (C * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

template <int BYTES, int NT>
__device__ __forceinline__ void load_bytes(uint32_t dst, const uint8_t* src, int tid) {
  static_assert(BYTES % 16 == 0, "16-byte pieces");
#pragma unroll
  for (int i = 0; i < (BYTES / 16 + NT - 1) / NT; ++i) {
    const int j = tid + i * NT;
    if ((BYTES / 16) % NT == 0 || j < BYTES / 16) cp16(dst + j * 16, src + j * 16, true);
  }
}

}  // namespace gmma

// The records of every chunk slot and head (la_gated_prep.cu); chunks given: those of the
// backward, with the transposed triangles, and every slot's batch entry, first row and
// number of tokens.
cudaError_t gated_prep(const GatedArgs& a, uint8_t* records, int4* chunks);
// What the backward's chains leave for the gradients' products, as bf16 high and low parts:
// E and dR [B,H,N,dv] (the high part of dR is the gradient dv), the states before and
// their gradients behind each chunk [slot,H,dv,dk].
struct ChainOut {
  __nv_bfloat16 *e, *e_lo, *dr_lo;
  __nv_bfloat16 *states, *states_lo, *dstates, *dstates_lo;
};
// The chains over the records (la_gated_chain.cu).
cudaError_t gated_chain_forward(const GatedArgs& a, const uint8_t* records);
cudaError_t gated_chain_backward(const GatedArgs& a, const uint8_t* records, const ChainOut& o);
// The forward ones by two warps for 16 columns (la_gated_pair.cu), and whether they are taken.
cudaError_t gated_pair_forward(const GatedArgs& a, const uint8_t* records);
bool gated_pair_wanted(const GatedArgs& a);
// The same for few heads, eight warps on 16 columns (la_gated_split.cu).
cudaError_t gated_split_forward(const GatedArgs& a, const uint8_t* records);
cudaError_t gated_split_backward(const GatedArgs& a, const uint8_t* records, const ChainOut& o);
// Whether they are taken.
bool gated_split_wanted(const GatedArgs& a, bool backward);
// A tensor map of [heads][N][d] bf16 in boxes of `cols` columns (16: rows of 32 bytes,
// swizzled so; 64: of 128) and C rows; false where there is none.
bool gated_map(CUtensorMap* m, const void* ptr, long long heads, int N, int d, int cols);

}  // namespace la
