// Host side of the gated delta rule's entry points and of the norm with
// rotation: argument checks and kernel choice. Nothing here allocates device
// memory or synchronises the stream.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <atomic>

#include "la_gated.cuh"
#include "la_spec.cuh"

namespace la {
namespace {

la_status fail(la_status s, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return set_error(s, msg);
}

la_status cuda_fail(cudaError_t e, const char* where) {
  return fail(LA_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool head_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
// a null pointer passes: whether it may be null is checked by itself
bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

la_status check_sizes(const char* who, int B, int Hk, int H, int N, int dk, int dv, int nseq, float scale,
                      la_dtype dtype, bool packed, bool* empty) {
  if (B < 0 || Hk < 0 || H < 0 || N < 0 || nseq < 0)
    return fail(LA_ERR_INVALID_ARG, "%s: negative size B=%d Hk=%d H=%d N=%d nseq=%d", who, B, Hk, H, N, nseq);
  if (dtype != LA_F32 && dtype != LA_BF16) return fail(LA_ERR_UNSUPPORTED, "%s: dtype %d not supported", who, (int)dtype);
  if (!head_ok(dk) || !head_ok(dv))
    return fail(LA_ERR_UNSUPPORTED, "%s: head sizes dk=%d dv=%d not in {16,32,64,128}", who, dk, dv);
  if (!(scale > -INFINITY && scale < INFINITY)) return fail(LA_ERR_INVALID_ARG, "%s: scale must be finite", who);
  if (packed ? B != 1 : nseq != B)
    return fail(LA_ERR_INVALID_ARG, packed ? "%s: packed sequences need B = 1" : "%s: nseq must be B without offsets", who);
  if ((H > 0) != (Hk > 0) || (Hk > 0 && H % Hk != 0))
    return fail(LA_ERR_INVALID_ARG, "%s: H=%d must be a multiple of Hk=%d", who, H, Hk);
  // CTAs: 8 a head and sequence at most, one a chunk of 32 tokens and head
  const long long limit = 0x7fffffffLL;
  if ((long long)nseq * H > limit / 8 || (long long)B * N > limit ||
      (chunk_slots(B, N, nseq, packed, 32)) > limit / (H > 0 ? H : 1))
    return fail(LA_ERR_INVALID_ARG, "%s: problem too large", who);
  *empty = nseq == 0 || H == 0;
  return LA_OK;
}

la_status check_call(const char* who, const GatedArgs& a, bool backward, bool* empty) {
  la_status st = check_sizes(who, a.B, a.Hk, a.H, a.N, a.dk, a.dv, a.nseq, a.scale, a.dtype, a.offsets != nullptr, empty);
  if (st != LA_OK || *empty) return st;
  if (a.N > 0 && (!a.q || !a.k || !a.v || !a.g || !a.beta))
    return fail(LA_ERR_INVALID_ARG, "%s: q, k, v, g, beta must be non-NULL", who);
  if (a.N > 0 && !backward && !a.out) return fail(LA_ERR_INVALID_ARG, "%s: out must be non-NULL", who);
  if (a.N > 0 && backward && (!a.dout || !a.dq || !a.dk_ || !a.dv_ || !a.dg || !a.dbeta))
    return fail(LA_ERR_INVALID_ARG, "%s: dout, dq, dk_, dv_, dg, dbeta must be non-NULL", who);
  const void* p16[] = {a.q, a.k, a.v, a.S0, a.S_final, a.out, a.dout, a.dS, a.dS0, a.dq, a.dk_, a.dv_, a.workspace};
  for (const void* p : p16)
    if (!aligned(p, 16))
      return fail(LA_ERR_INVALID_ARG, "%s: rows, states and workspace must be 16-byte aligned", who);
  if (!aligned(a.g, 4) || !aligned(a.beta, 4) || !aligned(a.offsets, 4))
    return fail(LA_ERR_INVALID_ARG, "%s: g, beta, offsets must be 4-byte aligned", who);
  if (!aligned(a.dg, 4) || !aligned(a.dbeta, 4))
    return fail(LA_ERR_INVALID_ARG, "%s: dg, dbeta must be 4-byte aligned", who);
  return LA_OK;
}

// Whole sequences on the tensor cores; N <= kShortN tokens are read token by token. Forward:
// 16 heads of 8, 16, 32, 48 tokens 5, 7, 12, 15 us against 12 on the tensor cores, 256 heads
// 10, 17, 32, 56 against 23. Backward: 16 heads of 8, 32 tokens 41, 54 against 28, 256 heads
// 96, 155 against 61, 67; but of so few tokens without a state dg is mostly what cancels (a first
// token's all of it, to exactly zero in this path, to what rounding leaves of the terms in the other).
constexpr int kShortN = 32;
bool use_mma(int N, int dk, int dv, la_dtype dtype) {
  return N > kShortN && current_path() == LA_PATH_AUTO && gated_on_tensor_cores(dk, dv, dtype);
}

bool packed_size(int B, int nseq) { return B == 1 && nseq != 1; }

// Strides of rows [B][N][heads][d]; where they are written, no row may begin inside its
// neighbour.
la_status check_strides(const char* who, const char* name, const long long* s, int size, const int* written, int d) {
  if (s == nullptr) return fail(LA_ERR_INVALID_ARG, "%s: %s must be non-NULL", who, name);
  const int per = 16 / size;
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] % per != 0 || s[i] > (1LL << 40))
      return fail(LA_ERR_INVALID_ARG, "%s: %s must be non-negative multiples of 16 bytes", who, name);
  for (int i = 0; i < 3 && written != nullptr; ++i)
    if (written[i] > 1 && s[i] < d) return fail(LA_ERR_INVALID_ARG, "%s: %s of written rows must not be below d=%d", who, name, d);
  return LA_OK;
}

la_status norm_call(const char* who, NormArgs& a, int norm, const long long* const (&stride)[2],
                    const long long* const (&dstride)[2], size_t workspace_bytes, bool backward) {
  const int Hq = a.H[0], Hk = a.H[1];
  if (a.B < 0 || a.N < 0 || Hq < 0 || Hk < 0)
    return fail(LA_ERR_INVALID_ARG, "%s: negative size B=%d N=%d Hq=%d Hk=%d", who, a.B, a.N, Hq, Hk);
  if (a.dtype != LA_F32 && a.dtype != LA_BF16) return fail(LA_ERR_UNSUPPORTED, "%s: dtype %d not supported", who, (int)a.dtype);
  if (!head_ok(a.d)) return fail(LA_ERR_UNSUPPORTED, "%s: head size d=%d not in {16,32,64,128}", who, a.d);
  if (a.rot < 0 || a.rot > a.d || a.rot % 16 != 0)
    return fail(LA_ERR_UNSUPPORTED, "%s: rot=%d must be a multiple of 16 up to d", who, a.rot);
  if (norm != LA_NORM_RMS && norm != LA_NORM_L2) return fail(LA_ERR_INVALID_ARG, "%s: unknown norm %d", who, norm);
  if (!(a.eps >= 0.f) || isinf(a.eps)) return fail(LA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
  a.l2 = norm == LA_NORM_L2;
  if ((long long)a.B * a.N > 0x7fffffffLL || (long long)Hq + Hk > 1 << 20)
    return fail(LA_ERR_INVALID_ARG, "%s: problem too large", who);
  const bool empty = a.B == 0 || a.N == 0 || Hq + Hk == 0;
  const int size = a.dtype == LA_BF16 ? 2 : 4;
  if (a.rot > 0 && !a.freqs && !empty) return fail(LA_ERR_INVALID_ARG, "%s: freqs must be non-NULL", who);
  if (!aligned(a.positions, 4) || !aligned(a.freqs, 4))
    return fail(LA_ERR_INVALID_ARG, "%s: positions, freqs must be 4-byte aligned", who);
  for (int i = 0; i < 2; ++i) {
    if (!aligned(a.w[i], 4) || !aligned(a.dw[i], 4))
      return fail(LA_ERR_INVALID_ARG, "%s: weights must be 4-byte aligned", who);
    if (a.dw[i] && !a.w[i]) return fail(LA_ERR_INVALID_ARG, "%s: a weight's gradient without the weight", who);
    if (a.H[i] == 0 || empty) continue;
    if (!a.x[i] || (backward ? !a.dy[i] || !a.dx[i] : !a.y[i]))
      return fail(LA_ERR_INVALID_ARG, "%s: rows of %s must be non-NULL", who, i ? "k" : "q");
    if (!aligned(a.x[i], 16) || !aligned(a.y[i], 16) || !aligned(a.dy[i], 16) || !aligned(a.dx[i], 16))
      return fail(LA_ERR_INVALID_ARG, "%s: rows must be 16-byte aligned", who);
    const int extent[3] = {a.B, a.N, a.H[i]};
    la_status st = check_strides(who, i ? "k_stride" : "q_stride", stride[i], size, nullptr, a.d);
    if (st == LA_OK && backward) st = check_strides(who, i ? "dk_stride" : "dq_stride", dstride[i], size, extent, a.d);
    if (st != LA_OK) return st;
    for (int j = 0; j < 3; ++j) {
      a.stride[i][j] = stride[i][j];
      if (backward) a.dstride[i][j] = dstride[i][j];
    }
  }
  cudaError_t e = cudaSuccess;
  if (empty) {
    // no rows: the weights' gradients are sums of nothing
    for (int i = 0; i < 2 && e == cudaSuccess; ++i)
      if (a.dw[i]) e = cudaMemsetAsync(a.dw[i], 0, sizeof(float) * a.d, a.stream);
    return e == cudaSuccess ? LA_OK : cuda_fail(e, who);
  }
  if (backward && (a.dw[0] || a.dw[1])) {
    const size_t need = norm_rotate_backward_workspace(a.B, a.N, Hq, Hk, a.d, a.dtype);
    if (!a.workspace || workspace_bytes < need || !aligned(a.workspace, 16))
      return fail(LA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, 16-byte aligned, got %zu", who, need, workspace_bytes);
  }
  e = backward ? norm_rotate_backward(a) : norm_rotate(a);
  return e == cudaSuccess ? LA_OK : cuda_fail(e, who);
}

std::atomic<int> g_gated_timeout_test{0};

}  // namespace

bool take_gated_timeout_test(int kernel) {
  int want = 1 + kernel;
  return g_gated_timeout_test.load(std::memory_order_relaxed) == want && g_gated_timeout_test.compare_exchange_strong(want, 0);
}

}  // namespace la

using namespace la;

extern "C" {

int la_gated_delta_path(int dk, int dv, la_dtype dtype) {
  if (!head_ok(dk) || !head_ok(dv) || (dtype != LA_F32 && dtype != LA_BF16)) return -1;
  return current_path() == LA_PATH_AUTO && gated_on_tensor_cores(dk, dv, dtype) ? 1 : 0;
}

void la_test_timeout_next_gated(int gradients) { g_gated_timeout_test.store(gradients ? 2 : 1); }

size_t la_forward_gated_delta_workspace_size(int B, int Hk, int H, int N, int dk, int dv, int nseq, la_dtype dtype) {
  bool empty = false;
  if (check_sizes("", B, Hk, H, N, dk, dv, nseq, 1.f, dtype, packed_size(B, nseq), &empty) != LA_OK || empty) return 0;
  return use_mma(N, dk, dv, dtype) ? mma_gated_forward_workspace(B, H, N, dk, dv, nseq, B == 1) : 0;
}

la_status la_forward_gated_delta(const void* q, const void* k, const void* v, const float* g, const float* beta,
                                 const float* S0, const int* offsets, void* out, float* S_final, int B, int Hk, int H,
                                 int N, int dk, int dv, int nseq, float scale, la_dtype dtype, void* workspace,
                                 size_t workspace_bytes, la_stream_t stream) {
  const char* who = "la_forward_gated_delta";
  GatedArgs a{};
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S0 = S0; a.S_final = S_final; a.offsets = offsets; a.out = out;
  a.B = B; a.Hk = Hk; a.H = H; a.N = N; a.dk = dk; a.dv = dv; a.nseq = nseq; a.scale = scale; a.dtype = dtype;
  a.workspace = workspace; a.workspace_bytes = workspace_bytes; a.stream = (cudaStream_t)stream;
  bool empty = false;
  la_status st = check_call(who, a, false, &empty);
  if (st != LA_OK || empty) return st;
  if (N == 0 && S_final == nullptr) return LA_OK;
  const size_t need = la_forward_gated_delta_workspace_size(B, Hk, H, N, dk, dv, nseq, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(LA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, got %zu", who, need, workspace_bytes);
  const cudaError_t e = use_mma(N, dk, dv, dtype) ? mma_gated_forward(a) : simt_gated_forward(a);
  return e == cudaSuccess ? LA_OK : cuda_fail(e, who);
}

size_t la_backward_gated_delta_workspace_size(int B, int Hk, int H, int N, int dk, int dv, int nseq, la_dtype dtype) {
  bool empty = false;
  if (check_sizes("", B, Hk, H, N, dk, dv, nseq, 1.f, dtype, packed_size(B, nseq), &empty) != LA_OK || empty) return 0;
  return use_mma(N, dk, dv, dtype) ? mma_gated_backward_workspace(B, H, N, dk, dv, nseq, B == 1)
                                                  : simt_gated_backward_workspace(B, H, N, dk, dv, nseq, B == 1);
}

la_status la_backward_gated_delta(const void* q, const void* k, const void* v, const float* g, const float* beta,
                                  const float* S0, const int* offsets, const void* dout, const float* dS, void* dq,
                                  void* dk_, void* dv_, void* dg, void* dbeta, float* dS0, int B, int Hk, int H, int N,
                                  int dk, int dv, int nseq, float scale, la_dtype dtype, void* workspace,
                                  size_t workspace_bytes, la_stream_t stream) {
  const char* who = "la_backward_gated_delta";
  GatedArgs a{};
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S0 = S0; a.offsets = offsets; a.dout = dout; a.dS = dS;
  a.dq = dq; a.dk_ = dk_; a.dv_ = dv_; a.dg = dg; a.dbeta = dbeta; a.dS0 = dS0;
  a.B = B; a.Hk = Hk; a.H = H; a.N = N; a.dk = dk; a.dv = dv; a.nseq = nseq; a.scale = scale; a.dtype = dtype;
  a.workspace = workspace; a.workspace_bytes = workspace_bytes; a.stream = (cudaStream_t)stream;
  bool empty = false;
  la_status st = check_call(who, a, true, &empty);
  if (st != LA_OK || empty) return st;
  if (N == 0 && dS0 == nullptr) return LA_OK;
  const size_t need = la_backward_gated_delta_workspace_size(B, Hk, H, N, dk, dv, nseq, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(LA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, got %zu", who, need, workspace_bytes);
  const cudaError_t e = use_mma(N, dk, dv, dtype) ? mma_gated_backward(a) : simt_gated_backward(a);
  return e == cudaSuccess ? LA_OK : cuda_fail(e, who);
}

la_status la_decode_steps_gated_delta(const float* S, const void* q, const void* k, const void* v, const float* g,
                                      const float* beta, const int* count, void* out, float* S_out, int B, int Hk, int H,
                                      int T, int dk, int dv, float scale, la_dtype dtype, la_stream_t stream) {
  const char* who = "la_decode_steps_gated_delta";
  bool empty = false;
  la_status st = check_sizes(who, B, Hk, H, T, dk, dv, B, scale, dtype, false, &empty);
  if (st != LA_OK || empty) return st;
  if (!S || !S_out || (T > 0 && (!q || !k || !v || !g || !beta || !out)))
    return fail(LA_ERR_INVALID_ARG, "%s: S, S_out, q, k, v, g, beta, out must be non-NULL", who);
  const void* p16[] = {S, S_out, q, k, v, out};
  for (const void* p : p16)
    if (!aligned(p, 16)) return fail(LA_ERR_INVALID_ARG, "%s: S, S_out, q, k, v, out must be 16-byte aligned", who);
  if (!aligned(g, 4) || !aligned(beta, 4) || !aligned(count, 4))
    return fail(LA_ERR_INVALID_ARG, "%s: g, beta, count must be 4-byte aligned", who);
  if (T == 0 && S == S_out) return LA_OK;
  GatedStepArgs a{};
  a.S = S; a.S_out = S_out; a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.count = count; a.out = out;
  a.B = B; a.Hk = Hk; a.H = H; a.T = T; a.dk = dk; a.dv = dv; a.scale = scale; a.dtype = dtype;
  a.stream = (cudaStream_t)stream;
  const cudaError_t e = simt_gated_steps(a);
  return e == cudaSuccess ? LA_OK : cuda_fail(e, who);
}

la_status la_clear_outside(void* const* rows, const int* row_bytes, const int* heads, int count, const int* offsets, int N,
                           int nseq, la_stream_t stream) {
  const char* who = "la_clear_outside";
  if (count < 0 || N < 0 || nseq < 0) return fail(LA_ERR_INVALID_ARG, "%s: negative size count=%d N=%d nseq=%d", who, count, N, nseq);
  if (count > kClearMost) return fail(LA_ERR_UNSUPPORTED, "%s: %d arrays, at most %d", who, count, kClearMost);
  if (count > 0 && (!rows || !row_bytes || !heads || !offsets))
    return fail(LA_ERR_INVALID_ARG, "%s: rows, row_bytes, heads, offsets must be non-NULL", who);
  if (!aligned(offsets, 4)) return fail(LA_ERR_INVALID_ARG, "%s: offsets must be 4-byte aligned", who);
  for (int i = 0; i < count; ++i) {
    if (heads[i] < 0 || row_bytes[i] <= 0 || row_bytes[i] % 2 != 0 || row_bytes[i] > 1 << 16)
      return fail(LA_ERR_INVALID_ARG, "%s: array %d has %d heads and rows of %d bytes", who, i, heads[i], row_bytes[i]);
    if (!rows[i] && heads[i] > 0 && N > 0) return fail(LA_ERR_INVALID_ARG, "%s: rows must be non-NULL", who);
    if (!aligned(rows[i], row_bytes[i] % 16 == 0 ? 16 : 2)) return fail(LA_ERR_INVALID_ARG, "%s: rows must be 16-byte aligned", who);
  }
  if (count == 0 || N == 0) return LA_OK;
  const cudaError_t e = clear_outside(rows, row_bytes, heads, count, offsets, N, nseq, (cudaStream_t)stream);
  return e == cudaSuccess ? LA_OK : cuda_fail(e, who);
}

la_status la_qk_norm_rotate(const void* q, const void* k, const float* q_weight, const float* k_weight,
                            const int* positions, const float* freqs, void* q_out, void* k_out, int B, int N, int Hq,
                            int Hk, int d, int rot, const long long* q_stride, const long long* k_stride, int norm,
                            int interleaved, float eps, la_dtype dtype, la_stream_t stream) {
  NormArgs a{};
  a.x[0] = q; a.x[1] = k; a.y[0] = q_out; a.y[1] = k_out; a.w[0] = q_weight; a.w[1] = k_weight;
  a.positions = positions; a.freqs = freqs; a.B = B; a.N = N; a.H[0] = Hq; a.H[1] = Hk; a.d = d; a.rot = rot;
  a.interleaved = interleaved != 0; a.eps = eps; a.dtype = dtype; a.stream = (cudaStream_t)stream;
  const long long* none[2] = {nullptr, nullptr};
  const long long* strides[2] = {q_stride, k_stride};
  return norm_call("la_qk_norm_rotate", a, norm, strides, none, 0, false);
}

size_t la_qk_norm_rotate_backward_workspace_size(int B, int N, int Hq, int Hk, int d, la_dtype dtype) {
  if (B <= 0 || N <= 0 || Hq < 0 || Hk < 0 || Hq + Hk <= 0 || !head_ok(d) || (dtype != LA_F32 && dtype != LA_BF16) ||
      (long long)B * N > 0x7fffffffLL || (long long)Hq + Hk > 1 << 20)
    return 0;
  return norm_rotate_backward_workspace(B, N, Hq, Hk, d, dtype);
}

la_status la_qk_norm_rotate_backward(const void* q, const void* k, const float* q_weight, const float* k_weight,
                                     const int* positions, const float* freqs, const void* dq_out, const void* dk_out,
                                     void* dq, void* dk_, float* dq_weight, float* dk_weight, int B, int N, int Hq,
                                     int Hk, int d, int rot, const long long* q_stride, const long long* k_stride,
                                     const long long* dq_stride, const long long* dk_stride, int norm, int interleaved,
                                     float eps, la_dtype dtype, void* workspace, size_t workspace_bytes,
                                     la_stream_t stream) {
  NormArgs a{};
  a.x[0] = q; a.x[1] = k; a.w[0] = q_weight; a.w[1] = k_weight; a.dy[0] = dq_out; a.dy[1] = dk_out; a.dx[0] = dq;
  a.dx[1] = dk_; a.dw[0] = dq_weight; a.dw[1] = dk_weight;
  a.positions = positions; a.freqs = freqs; a.B = B; a.N = N; a.H[0] = Hq; a.H[1] = Hk; a.d = d; a.rot = rot;
  a.interleaved = interleaved != 0; a.eps = eps; a.dtype = dtype; a.workspace = (float*)workspace;
  a.stream = (cudaStream_t)stream;
  const long long* strides[2] = {q_stride, k_stride};
  const long long* dstrides[2] = {dq_stride, dk_stride};
  return norm_call("la_qk_norm_rotate_backward", a, norm, strides, dstrides, workspace_bytes, true);
}

}  // extern "C"
