// Packed state pool: states leave for, and come back from, slots of 8-bit
// codes with a power-of-two scale for each block of min(32, dv) consecutive
// values of a state row (about a quarter of the fp32 bytes); z stays fp32.
//
//   scale = the smallest 2^e, e >= -127, with max|x| <= 448 * 2^e over the
//           block's finite values (448: the largest e4m3 number), stored as e + 127
//   code  = e4m3(x / 2^e), to nearest, ties to even
// Dividing by a power of two is exact, so the only rounding is the one to the
// code's four significant bits, a relative 2^-4 at most of a normal code; the
// way back, code * 2^e, is exact. A NaN is kept; an infinite value takes the
// largest code (the format has no infinity).
//
// Memory-bound: 4 bytes in and 1.03 out a value, or the reverse - if there are
// few instructions a value: packing with one 16-byte piece a lane and the
// finite magnitudes picked out value by value took 22 and 29 us for 2048 d =
// 128 states, three quarters of the issue slots. Packing, a lane takes eight
// consecutive values, so that four lanes (two for dv = 16) share a block and
// two shuffles join its maximum; infinities are looked for only where the
// maximum is one: 26.7 us, 0.94 of the floor. Unpacking, a lane takes four
// values, so that a warp's stores are whole lines (30 us for 2048 states, four
// bytes written for each one read). Four loads of a lane are in flight.
#include <cuda_fp8.h>

#include "la_spec.cuh"

namespace la {

namespace {

constexpr int PT = 256;     // threads
constexpr int PU = 4;       // 16-byte pieces of state per thread (two and two together where they are packed)
constexpr int PTILE = PT * PU * 4;   // values per CTA

// The exponent e of the block's scale from its largest finite magnitude: with
// m = 1.f * 2^x (f the mantissa bits), m <= 448 * 2^e = 1.75 * 2^(8 + e).
__device__ __forceinline__ int block_exponent(float m) {
  if (m == 0.f) return -127;
  const uint32_t bits = __float_as_uint(m);
  const int x = (int)(bits >> 23);
  if (x == 0) return -127;                          // a subnormal: far below 448 * 2^-127
  const int e = x - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -127);
}

// 2^n for -149 <= n <= 127
__device__ __forceinline__ float pow2(int n) {
  return n >= -126 ? __uint_as_float((uint32_t)(n + 127) << 23) : __uint_as_float(1u << (n + 149));
}

// Blocks with the largest scale, 2^120, reach fp32's range: 248 and above would
// round to 256 * 2^120, which is infinite, so they stop at 240 (still within
// 2^-4 of the value).
constexpr int kTopExponent = 120;
__device__ __forceinline__ float below_top(float y) { return fabsf(y) > 240.f ? copysignf(240.f, y) : y; }

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < __uint_as_float(0x7f800000u) ? a : 0.f;
}

// Does a later sequence store into the same slot? Then it has the last word,
// as if the sequences were stored one after the other.
__device__ __forceinline__ bool overwritten(const int* slot, int b, int B) {
  const int mine = slot[b];
  int later = 0;
  for (int i = b + 1 + threadIdx.x; i < B; i += PT) later |= slot[i] == mine;
  return __syncthreads_or(later) != 0;
}

// Eight scaled values as codes.
__device__ __forceinline__ uint2 to_codes(const float (&y)[8]) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i], y[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <int DV>
__global__ void __launch_bounds__(PT)
pack_kernel(const float* __restrict__ S, const float* __restrict__ z, unsigned char* __restrict__ codes,
            unsigned char* __restrict__ scales, float* __restrict__ z_pool, const int* __restrict__ slot, int B,
            int words, int zwords, int slots, int tiles) {
  constexpr int W = DV < 32 ? DV : 32;              // values per block
  constexpr int LW = W / 8;                          // lanes per block
  constexpr int U = PU / 2;
  const int b = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int to = slot[b];
  if (to < 0 || to >= slots) return;
  const float* src = S + (long long)b * words;
  unsigned char* dc = codes + (long long)to * words;
  unsigned char* ds = scales + (long long)to * (words / W);
  const int base = tile * PTILE + threadIdx.x * 8;
  float x[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = base + u * PT * 8;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), c = a;
    if (at < words) {
      a = *reinterpret_cast<const float4*>(src + at);
      c = *reinterpret_cast<const float4*>(src + at + 4);
    }
    x[u][0] = a.x; x[u][1] = a.y; x[u][2] = a.z; x[u][3] = a.w;
    x[u][4] = c.x; x[u][5] = c.y; x[u][6] = c.z; x[u][7] = c.w;
  }
  if (overwritten(slot, b, B)) return;            // (with the loads on their way)
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = base + u * PT * 8;
    float m = 0.f;                                 // (the larger of a number and a NaN is the number)
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[u][i]));
    if (m == __uint_as_float(0x7f800000u)) {
      m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(x[u][i]));
    }
    __syncwarp();
#pragma unroll
    for (int o = 1; o < LW; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int e = block_exponent(m);
    const float r = pow2(-e);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[u][i] * r;
    if (e == kTopExponent) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = below_top(y[i]);
    }
    if (at < words) {
      *reinterpret_cast<uint2*>(dc + at) = to_codes(y);
      if ((threadIdx.x & (LW - 1)) == 0) ds[at / W] = (unsigned char)(e + 127);
    }
  }
  if (tile == 0 && z != nullptr)
    for (int i = threadIdx.x; i < zwords; i += PT) z_pool[(long long)to * zwords + i] = z[(long long)b * zwords + i];
}

template <int DV>
__global__ void __launch_bounds__(PT)
unpack_kernel(float* __restrict__ S, float* __restrict__ z, const unsigned char* __restrict__ codes,
              const unsigned char* __restrict__ scales, const float* __restrict__ z_pool,
              const int* __restrict__ slot, int words, int zwords, int slots, int tiles) {
  constexpr int W = DV < 32 ? DV : 32;
  const int b = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int from = slot[b];
  if (from < 0 || from >= slots) return;
  float* dst = S + (long long)b * words;
  const unsigned char* sc = codes + (long long)from * words;
  const unsigned char* ss = scales + (long long)from * (words / W);
  const int base = tile * PTILE + threadIdx.x * 4;
  uint32_t c[PU];
  unsigned char e[PU];
#pragma unroll
  for (int u = 0; u < PU; ++u) {
    const int at = base + u * PT * 4;
    c[u] = at < words ? *reinterpret_cast<const uint32_t*>(sc + at) : 0u;
    e[u] = at < words ? ss[at / W] : 0;
  }
#pragma unroll
  for (int u = 0; u < PU; ++u) {
    const int at = base + u * PT * 4;
    __nv_fp8x4_e4m3 q;
    q.__x = c[u];
    float4 x = static_cast<float4>(q);
    const float r = pow2((int)e[u] - 127);
    if (at < words) __stcs(reinterpret_cast<float4*>(dst + at), make_float4(x.x * r, x.y * r, x.z * r, x.w * r));
  }
  if (tile == 0 && z != nullptr)
    for (int i = threadIdx.x; i < zwords; i += PT) z[(long long)b * zwords + i] = z_pool[(long long)from * zwords + i];
}

template <int DV>
cudaError_t launch(const PackArgs& a, bool pack) {
  const int words = a.H * a.dk * a.dv, zwords = a.H * a.dk;
  const int tiles = (words + PTILE - 1) / PTILE;
  const long long ctas = (long long)a.B * tiles;
  if (pack)
    pack_kernel<DV><<<(unsigned)ctas, PT, 0, a.stream>>>(a.S, a.z, a.codes, a.scales, a.z_pool, a.slot, a.B, words,
                                                         zwords, a.slots, tiles);
  else
    unpack_kernel<DV><<<(unsigned)ctas, PT, 0, a.stream>>>(a.S, a.z, a.codes, a.scales, a.z_pool, a.slot, words,
                                                           zwords, a.slots, tiles);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t dispatch(const PackArgs& a, bool pack) {
  switch (a.dv) {
    case 16: return launch<16>(a, pack);
    case 32: return launch<32>(a, pack);
    case 64: return launch<64>(a, pack);
    case 128: return launch<128>(a, pack);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t state_pack(const PackArgs& a) { return dispatch(a, true); }
cudaError_t state_unpack(const PackArgs& a) { return dispatch(a, false); }

}  // namespace la
