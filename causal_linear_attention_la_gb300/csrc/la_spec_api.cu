// Host side of the speculative-decoding entry points of include/la.h:
// argument checks and kernel choice. Nothing here allocates device memory or
// synchronises the stream.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <atomic>

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

// Sizes of B*H states; *empty when there is none.
la_status check_states(const char* who, int B, int H, int T, int dk, int dv, la_dtype dtype, bool* empty) {
  if (B < 0 || H < 0 || T < 0) return fail(LA_ERR_INVALID_ARG, "%s: negative size B=%d H=%d T=%d", who, B, H, T);
  if (dtype != LA_F32 && dtype != LA_BF16) return fail(LA_ERR_UNSUPPORTED, "%s: dtype %d not supported", who, (int)dtype);
  if (!head_ok(dk) || !head_ok(dv))
    return fail(LA_ERR_UNSUPPORTED, "%s: head sizes dk=%d dv=%d not in {16,32,64,128}", who, dk, dv);
  const long long BH = (long long)B * H;
  if (BH > 0x7fffffffLL) return fail(LA_ERR_INVALID_ARG, "%s: B*H too large", who);
  *empty = BH == 0;
  return LA_OK;
}

la_status tree_call(const char* who, const TreeArgs& a, int B, bool delta) {
  bool empty = false;
  la_status st = check_states(who, B, a.H, a.T, a.dk, a.dv, a.dtype, &empty);
  if (st != LA_OK) return st;
  if (a.T > kTreeMax) return fail(LA_ERR_UNSUPPORTED, "%s: T=%d nodes, at most %d", who, a.T, kTreeMax);
  if (!(a.eps >= 0.f) || isinf(a.eps)) return fail(LA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
  if (empty || a.T == 0) return LA_OK;
  if (!a.S || (!delta && !a.z) || !a.q || !a.k || !a.v || !a.parent || !a.out)
    return fail(LA_ERR_INVALID_ARG, "%s: S, %sq, k, v, parent, out must be non-NULL", who, delta ? "" : "z, ");
  if (!aligned(a.S, 16) || !aligned(a.z, 16) || !aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) ||
      !aligned(a.out, 16))
    return fail(LA_ERR_INVALID_ARG, "%s: S, z, q, k, v, out must be 16-byte aligned", who);
  if (!aligned(a.parent, 4) || !aligned(a.count, 4) || !aligned(a.alpha, 4))
    return fail(LA_ERR_INVALID_ARG, "%s: parent, count, alpha must be 4-byte aligned", who);
  TreeArgs t = a;
  t.BH = B * a.H;
  cudaError_t e;
  if (current_path() != LA_PATH_AUTO || !tree_on_tensor_cores(t.dk, t.dv, t.dtype))
    e = simt_tree(t);
  else if (t.dk == 64)
    e = t.dv == 64 ? tree_mma_64_64(t) : tree_mma_64_128(t);
  else
    e = t.dv == 64 ? tree_mma_128_64(t) : tree_mma_128_128(t);
  return e == cudaSuccess ? LA_OK : cuda_fail(e, who);
}

la_status advance_call(const char* who, const AdvanceArgs& a, int B, bool delta) {
  bool empty = false;
  la_status st = check_states(who, B, a.H, a.T, a.dk, a.dv, a.dtype, &empty);
  if (st != LA_OK) return st;
  if (empty) return LA_OK;
  if (!a.S || !a.S_out || (!delta && (!a.z || !a.z_out)))
    return fail(LA_ERR_INVALID_ARG, "%s: S, S_out%s must be non-NULL", who, delta ? "" : ", z, z_out");
  if (a.T > 0 && (!a.k || !a.v)) return fail(LA_ERR_INVALID_ARG, "%s: k, v must be non-NULL", who);
  if (!delta && (a.S == a.S_out) != (a.z == a.z_out))
    return fail(LA_ERR_INVALID_ARG, "%s: S and z must be both in place or both not", who);
  if (!aligned(a.S, 16) || !aligned(a.z, 16) || !aligned(a.S_out, 16) || !aligned(a.z_out, 16) || !aligned(a.k, 16) ||
      !aligned(a.v, 16))
    return fail(LA_ERR_INVALID_ARG, "%s: S, z, S_out, z_out, k, v must be 16-byte aligned", who);
  if (!aligned(a.path, 4) || !aligned(a.accepted, 4) || !aligned(a.alpha, 4))
    return fail(LA_ERR_INVALID_ARG, "%s: path, accepted, alpha must be 4-byte aligned", who);
  if (a.T == 0 && a.S == a.S_out) return LA_OK;
  AdvanceArgs t = a;
  t.BH = B * a.H;
  const cudaError_t e = state_advance(t);
  return e == cudaSuccess ? LA_OK : cuda_fail(e, who);
}

la_status check_verify(const char* who, int B, int T, int V, la_dtype dtype) {
  if (B < 0 || T < 0) return fail(LA_ERR_INVALID_ARG, "%s: negative size B=%d T=%d", who, B, T);
  if (dtype != LA_F32 && dtype != LA_BF16) return fail(LA_ERR_UNSUPPORTED, "%s: dtype %d not supported", who, (int)dtype);
  if (T > kTreeMax) return fail(LA_ERR_UNSUPPORTED, "%s: T=%d tokens, at most %d", who, T, kTreeMax);
  if (V < 1 || V > (1 << 30)) return fail(LA_ERR_INVALID_ARG, "%s: V=%d not in 1 .. 2^30", who, V);
  if (B > (1 << 27)) return fail(LA_ERR_INVALID_ARG, "%s: B too large", who);
  return LA_OK;
}

la_status pack_call(const char* who, const PackArgs& a, bool pack) {
  bool empty = false;
  la_status st = check_states(who, a.B, a.H, 0, a.dk, a.dv, LA_F32, &empty);
  if (st != LA_OK) return st;
  if (a.slots < 0) return fail(LA_ERR_INVALID_ARG, "%s: negative number of slots", who);
  // every CTA looks through the later sequences' slots: B^2 reads in all, which
  // take minutes from 2^24 sequences on
  if (pack && a.B > (1 << 20)) return fail(LA_ERR_UNSUPPORTED, "%s: B=%d sequences, at most %d", who, a.B, 1 << 20);
  if ((a.z == nullptr) != (a.z_pool == nullptr))
    return fail(LA_ERR_INVALID_ARG, "%s: z and z_pool must be both given or both NULL", who);
  // one sequence's states are indexed with 32 bits, one CTA takes 4096 values
  const long long words = (long long)a.H * a.dk * a.dv;
  if (words > (1LL << 30) || (words / 4096 + 1) * a.B > 0x7fffffffLL)
    return fail(LA_ERR_INVALID_ARG, "%s: problem too large", who);
  if (empty || a.slots == 0) return LA_OK;
  if (!a.S || !a.codes || !a.scales || !a.slot)
    return fail(LA_ERR_INVALID_ARG, "%s: S, codes, scales, slot must be non-NULL", who);
  if (!aligned(a.S, 16) || !aligned(a.z, 16) || !aligned(a.codes, 16) || !aligned(a.z_pool, 16))
    return fail(LA_ERR_INVALID_ARG, "%s: S, z, codes, z_pool must be 16-byte aligned", who);
  if (!aligned(a.slot, 4)) return fail(LA_ERR_INVALID_ARG, "%s: slot must be 4-byte aligned", who);
  const cudaError_t e = pack ? state_pack(a) : state_unpack(a);
  return e == cudaSuccess ? LA_OK : cuda_fail(e, who);
}

std::atomic<int> g_tree_timeout_test{0};

}  // namespace

bool take_tree_timeout_test() {
  return g_tree_timeout_test.load(std::memory_order_relaxed) != 0 && g_tree_timeout_test.exchange(0) != 0;
}

}  // namespace la

using namespace la;

extern "C" {

int la_tree_path(int dk, int dv, la_dtype dtype) {
  if (!head_ok(dk) || !head_ok(dv) || (dtype != LA_F32 && dtype != LA_BF16)) return -1;
  return current_path() == LA_PATH_AUTO && tree_on_tensor_cores(dk, dv, dtype) ? 1 : 0;
}

void la_test_timeout_next_tree(void) { la::g_tree_timeout_test.store(1); }

la_status la_decode_tree(const float* S, const float* z, const void* q, const void* k, const void* v,
                         const int* parent, const int* count, void* out, int B, int H, int T, int dk, int dv,
                         const float* alpha, float eps, la_dtype dtype, la_stream_t stream) {
  TreeArgs a{};
  a.S = S; a.z = z; a.q = q; a.k = k; a.v = v; a.parent = parent; a.count = count; a.out = out;
  a.H = H; a.T = T; a.dk = dk; a.dv = dv; a.alpha = alpha; a.eps = eps; a.dtype = dtype;
  a.stream = (cudaStream_t)stream;
  return tree_call("la_decode_tree", a, B, false);
}

la_status la_decode_tree_delta(const float* S, const void* q, const void* k, const void* v, const int* parent,
                               const int* count, void* out, int B, int H, int T, int dk, int dv, la_dtype dtype,
                               la_stream_t stream) {
  TreeArgs a{};
  a.S = S; a.q = q; a.k = k; a.v = v; a.parent = parent; a.count = count; a.out = out;
  a.H = H; a.T = T; a.dk = dk; a.dv = dv; a.dtype = dtype;
  a.stream = (cudaStream_t)stream;
  return tree_call("la_decode_tree_delta", a, B, true);
}

la_status la_verify_chain(const void* target, const void* draft, const int* tokens, const int* count,
                          const float* uniform, int* accepted, int* next, int B, int T, int V, la_dtype dtype,
                          la_stream_t stream) {
  const char* who = "la_verify_chain";
  la_status st = check_verify(who, B, T, V, dtype);
  if (st != LA_OK) return st;
  if (B == 0) return LA_OK;
  if (!target || !uniform || !accepted || !next || (T > 0 && (!draft || !tokens)))
    return fail(LA_ERR_INVALID_ARG, "%s: target, draft, tokens, uniform, accepted, next must be non-NULL", who);
  if (!aligned(target, 16) || !aligned(draft, 16))
    return fail(LA_ERR_INVALID_ARG, "%s: target, draft must be 16-byte aligned", who);
  if (!aligned(tokens, 4) || !aligned(count, 4) || !aligned(uniform, 4) || !aligned(accepted, 4) || !aligned(next, 4))
    return fail(LA_ERR_INVALID_ARG, "%s: tokens, count, uniform, accepted, next must be 4-byte aligned", who);
  VerifyArgs a{};
  a.target = target; a.draft = draft; a.tokens = tokens; a.count = count; a.uniform = uniform;
  a.accepted = accepted; a.next = next; a.B = B; a.T = T; a.V = V; a.dtype = dtype;
  a.stream = (cudaStream_t)stream;
  const cudaError_t e = verify(a);
  return e == cudaSuccess ? LA_OK : cuda_fail(e, who);
}

la_status la_verify_tree(const void* target, const int* tokens, const int* parent, const int* count,
                         const float* uniform, int* path, int* accepted, int* next, int B, int T, int V,
                         la_dtype dtype, la_stream_t stream) {
  const char* who = "la_verify_tree";
  la_status st = check_verify(who, B, T, V, dtype);
  if (st != LA_OK) return st;
  if (B == 0) return LA_OK;
  if (!target || !uniform || !accepted || !next || (T > 0 && (!tokens || !parent || !path)))
    return fail(LA_ERR_INVALID_ARG, "%s: target, tokens, parent, uniform, path, accepted, next must be non-NULL", who);
  if (!aligned(target, 16)) return fail(LA_ERR_INVALID_ARG, "%s: target must be 16-byte aligned", who);
  if (!aligned(tokens, 4) || !aligned(parent, 4) || !aligned(count, 4) || !aligned(uniform, 4) || !aligned(path, 4) ||
      !aligned(accepted, 4) || !aligned(next, 4))
    return fail(LA_ERR_INVALID_ARG, "%s: tokens, parent, count, uniform, path, accepted, next must be 4-byte aligned", who);
  VerifyArgs a{};
  a.target = target; a.tokens = tokens; a.parent = parent; a.count = count; a.uniform = uniform;
  a.path = path; a.accepted = accepted; a.next = next; a.B = B; a.T = T; a.V = V; a.dtype = dtype;
  a.stream = (cudaStream_t)stream;
  const cudaError_t e = verify(a);
  return e == cudaSuccess ? LA_OK : cuda_fail(e, who);
}

la_status la_state_advance(const float* S, const float* z, const void* k, const void* v, const int* path,
                           const int* accepted, float* S_out, float* z_out, int B, int H, int T, int dk, int dv,
                           const float* alpha, la_dtype dtype, la_stream_t stream) {
  AdvanceArgs a{};
  a.S = S; a.z = z; a.k = k; a.v = v; a.path = path; a.accepted = accepted; a.S_out = S_out; a.z_out = z_out;
  a.H = H; a.T = T; a.dk = dk; a.dv = dv; a.alpha = alpha; a.dtype = dtype;
  a.stream = (cudaStream_t)stream;
  return advance_call("la_state_advance", a, B, false);
}

la_status la_state_advance_delta(const float* S, const void* k, const void* v, const int* path, const int* accepted,
                                 float* S_out, int B, int H, int T, int dk, int dv, la_dtype dtype,
                                 la_stream_t stream) {
  AdvanceArgs a{};
  a.S = S; a.k = k; a.v = v; a.path = path; a.accepted = accepted; a.S_out = S_out;
  a.H = H; a.T = T; a.dk = dk; a.dv = dv; a.dtype = dtype;
  a.stream = (cudaStream_t)stream;
  return advance_call("la_state_advance_delta", a, B, true);
}

la_status la_state_pack(const float* S, const float* z, unsigned char* codes, unsigned char* scales, float* z_pool,
                        const int* slot, int B, int H, int dk, int dv, int slots, la_stream_t stream) {
  PackArgs a{};
  a.S = const_cast<float*>(S); a.z = const_cast<float*>(z); a.codes = codes; a.scales = scales; a.z_pool = z_pool;
  a.slot = slot; a.B = B; a.H = H; a.dk = dk; a.dv = dv; a.slots = slots; a.stream = (cudaStream_t)stream;
  return pack_call("la_state_pack", a, true);
}

la_status la_state_unpack(const unsigned char* codes, const unsigned char* scales, const float* z_pool,
                          const int* slot, float* S, float* z, int B, int H, int dk, int dv, int slots,
                          la_stream_t stream) {
  PackArgs a{};
  a.S = S; a.z = z; a.codes = const_cast<unsigned char*>(codes); a.scales = const_cast<unsigned char*>(scales);
  a.z_pool = const_cast<float*>(z_pool);
  a.slot = slot; a.B = B; a.H = H; a.dk = dk; a.dv = dv; a.slots = slots; a.stream = (cudaStream_t)stream;
  return pack_call("la_state_unpack", a, false);
}

}  // extern "C"
