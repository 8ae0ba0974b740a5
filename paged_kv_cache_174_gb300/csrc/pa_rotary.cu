// pa_rotary.cu -- rotary positions with several axes on a step's queries and
// keys, and the slot scatter of its keys and values, in one pass.
//
// Pair i of a head (i < rot / 2) is turned by the angle
// theta_i = pos[axis_i] * inv_freq_i, where pos[a] is the token's position on
// axis a (time, height, width, ...):
//   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin),
// with (x1, x2) = (x[i], x[i + rot/2]), or (x[2i], x[2i + 1]) interleaved; the
// elements from rot on are passed through.  q is written to q_out; k and v go
// to the token's slot in the cache, as pa_reshape_and_cache writes them.
//
// Angles: a rotation only needs theta modulo one turn, so the frequency is
// taken in turns as a 64-bit fraction, F = frac(f / 2 pi) 2^64, and pos * F in
// 64-bit arithmetic wraps by itself.  The product's error is |pos| 2^-64 turns
// or so, where an fp32 product is off by a radian at positions near 10^7.  Its
// top 32 bits, as a signed fraction of a half turn, feed sincospif, which
// reduces nothing further.
//
// Bytes: q, k and v are read once and written once (HBM-bound); a lane holds
// the same 16 elements of every head it handles, so it needs the same eight
// (cos, sin) pairs for all of them.
#include <cstdint>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kRotThreads = 128;

// frac(f / 2 pi) * 2^64 of a finite f with |f| < 2^31: the 53-bit mantissa times
// 2^66 / (2 pi), shifted by the exponent; below 2^-64 of a turn exact.
__device__ __forceinline__ unsigned long long turn_fraction(double f, bool& bad) {
  constexpr unsigned long long kInvTwoPi66 = 0xA2F9836E4E441529ull;  // floor(2^66 / (2 pi))
  const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
  const int e = (int)((bits >> 52) & 0x7ff) - 1023;
  if (e >= 31) {  // also infinities and NaN
    bad = true;
    return 0;
  }
  const unsigned long long m = (bits & 0xfffffffffffffull) | (e > -1023 ? 1ull << 52 : 0);
  const unsigned long long hi = __umul64hi(m, kInvTwoPi66), lo = m * kInvTwoPi66;
  const int shift = 54 - (e > -1023 ? e : -1022);  // >= 24
  unsigned long long t;
  if (shift < 64)
    t = (hi << (64 - shift)) | (lo >> shift);
  else if (shift < 128)
    t = hi >> (shift - 64);
  else
    t = 0;
  return (bits >> 63) ? 0ull - t : t;
}

// Cosine and sine of pair i's angle for a token.
__device__ __forceinline__ float2 pair_cos_sin(const RotaryArgs& p, int64_t t, int i, bool& bad) {
  int axis = p.axes ? p.axes[i] : 0;
  if (axis < 0 || axis >= p.num_axes) bad = true, axis = 0;
  const long long pos = p.positions[axis * p.positions_stride + t];
  const unsigned long long turns = (unsigned long long)pos * turn_fraction(p.inv_freq[i], bad);
  const float half_turns = (float)(int)(turns >> 32) * 4.656612873077393e-10f;  // 2^-31
  float2 cs;
  sincospif(half_turns, &cs.y, &cs.x);
  return cs;
}

// 16 elements of a head (two 8-element chunks) in fp32.
struct Piece {
  float a[8], b[8];
};

__device__ __forceinline__ void widen(const uint4& w, float (&x)[8]) {
  const float2 p0 = bf16x2_to_float2(w.x), p1 = bf16x2_to_float2(w.y);
  const float2 p2 = bf16x2_to_float2(w.z), p3 = bf16x2_to_float2(w.w);
  x[0] = p0.x, x[1] = p0.y, x[2] = p1.x, x[3] = p1.y;
  x[4] = p2.x, x[5] = p2.y, x[6] = p3.x, x[7] = p3.y;
}

__device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Turn the lane's eight pairs: chunk a with chunk b, or neighbours inside each.
__device__ __forceinline__ void turn(Piece& x, const float2 (&cs)[8], bool interleaved) {
  if (!interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = x.a[e], w = x.b[e];
      x.a[e] = u * cs[e].x - w * cs[e].y;
      x.b[e] = w * cs[e].x + u * cs[e].y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float u = x.a[2 * e], w = x.a[2 * e + 1];
      x.a[2 * e] = u * cs[e].x - w * cs[e].y;
      x.a[2 * e + 1] = w * cs[e].x + u * cs[e].y;
      const float y = x.b[2 * e], z = x.b[2 * e + 1];
      x.b[2 * e] = y * cs[4 + e].x - z * cs[4 + e].y;
      x.b[2 * e + 1] = z * cs[4 + e].x + y * cs[4 + e].y;
    }
  }
}

// Store a row's piece to the 8-bit cache: scale = row max / 448 (1 for an
// all-zero row) over the row's LPR lanes, codes e4m3(x / scale), as
// pa_reshape_and_cache_fp8 defines them, from the fp32 values (a rotated key
// is rounded once, to its code).
template <int D>
__device__ __forceinline__ void store_fp8(unsigned char* cache, int64_t slot, int n_kv, int h,
                                          int ca, int cb, int l, const Piece& x, bool on) {
  constexpr int LPR = D / 16;
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(x.a[e]), fabsf(x.b[e])));
#pragma unroll
  for (int m = LPR / 2; m >= 1; m >>= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  if (!on) return;
  const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
  unsigned char* page = cache + (slot / kFp8PageTokens) * fp8_page_bytes(n_kv, D);
  const int64_t row = (slot % kFp8PageTokens) * n_kv + h;
  auto codes = [&](const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = e4m3x2_from_floats(__fdiv_rn(v[2 * e], sc), __fdiv_rn(v[2 * e + 1], sc));
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  };
  *reinterpret_cast<uint2*>(page + row * D + ca * 8) = codes(x.a);
  *reinterpret_cast<uint2*>(page + row * D + cb * 8) = codes(x.b);
  if (l == 0) *reinterpret_cast<float*>(page + fp8_scales_offset(n_kv, D) + row * 4) = sc;
}

template <int D, bool F8>
__global__ void __launch_bounds__(kRotThreads) rotary_cache_kernel(const RotaryArgs p) {
  constexpr int LPR = D / 16;  // lanes of a head: 16 elements each
  __shared__ float2 cs_s[D / 2];
  const int64_t t = blockIdx.x;
  const int half = p.rotary_dim / 2;
  bool bad = false;
  for (int i = threadIdx.x; i < half; i += kRotThreads) cs_s[i] = pair_cos_sin(p, t, i, bad);
  __syncthreads();
  int64_t slot = p.slot_mapping[t];
  if (slot >= p.num_slots) bad = true, slot = -1;
  const int l = threadIdx.x % LPR;
  const bool rot = l < p.rotary_dim / 16;
  // this lane's two chunks of 8 elements
  int ca = 2 * l, cb = 2 * l + 1;
  float2 cs[8];
  if (rot) {
    if (!p.interleaved) ca = l, cb = l + p.rotary_dim / 16;
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = cs_s[8 * l + e];
  }
  const int rows = p.n_q + 2 * p.n_kv;
  for (int r0 = 0; r0 < rows; r0 += kRotThreads / LPR) {
    const int r = r0 + threadIdx.x / LPR;
    const bool on = r < rows;
    const uint16_t* src = p.q + t * p.q_stride + (int64_t)r * D;
    int h = r;
    if (r >= p.n_q) h = r - p.n_q, src = p.k + t * p.k_stride + (int64_t)h * D;
    const bool is_v = r >= p.n_q + p.n_kv;
    if (is_v) h -= p.n_kv, src = p.v + t * p.v_stride + (int64_t)h * D;
    const bool needed = on && (r < p.n_q || slot >= 0);
    uint4 wa = make_uint4(0u, 0u, 0u, 0u), wb = wa;
    if (needed) {
      wa = *reinterpret_cast<const uint4*>(src + ca * 8);
      wb = *reinterpret_cast<const uint4*>(src + cb * 8);
    }
    Piece x;
    widen(wa, x.a);
    widen(wb, x.b);
    if (rot && !is_v) turn(x, cs, p.interleaved);
    if (F8) {
      // every lane takes part in the row maximum's shuffles
      store_fp8<D>(is_v ? static_cast<unsigned char*>(p.v_cache)
                        : static_cast<unsigned char*>(p.k_cache),
                   slot, p.n_kv, h, ca, cb, l, x, needed && r >= p.n_q);
    }
    if (!needed || (F8 && r >= p.n_q)) continue;
    uint16_t* dst = r < p.n_q ? p.q_out + (t * p.n_q + r) * D
                              : static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) +
                                    (slot * p.n_kv + h) * D;
    *reinterpret_cast<uint4*>(dst + ca * 8) = narrow(x.a);
    *reinterpret_cast<uint4*>(dst + cb * 8) = narrow(x.b);
  }
  if (bad) flag_error(p.err, DEVERR_BOUNDS);
}

}  // namespace

cudaError_t launch_rotary_cache(const RotaryArgs& p, cudaStream_t stream) {
  if (p.head_dim == 128 && !p.fp8)
    rotary_cache_kernel<128, false><<<p.num_tokens, kRotThreads, 0, stream>>>(p);
  else if (p.head_dim == 64 && !p.fp8)
    rotary_cache_kernel<64, false><<<p.num_tokens, kRotThreads, 0, stream>>>(p);
  else if (p.head_dim == 128)
    rotary_cache_kernel<128, true><<<p.num_tokens, kRotThreads, 0, stream>>>(p);
  else if (p.head_dim == 64)
    rotary_cache_kernel<64, true><<<p.num_tokens, kRotThreads, 0, stream>>>(p);
  else
    return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace pa
