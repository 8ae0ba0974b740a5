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
// Bytes: q, k and v are read once and written once (HBM-bound).  A warp works
// on one token by itself: its lanes compute the token's cosines and sines, two
// each, into shared memory while the first heads' loads are in flight, and a
// lane then holds the same 16 elements of every head it handles, so it keeps
// the same eight (cos, sin) pairs in registers for all of them.
#include <cstdint>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kRotThreads = 128;
constexpr int kRotWarps = kRotThreads / 32;
// Warps that share a token's heads: more of them wait less for the heads, but
// each computes the token's angles.  A token of at least kRotLong passes (a pass
// is 32 lanes' heads) is shared by two warps, by four in a call of at most
// kRotFew tokens; a shorter one by two in such a call.  32 + 8 heads of 128 (12
// passes), 1 / 2 / 4 warps: 128 tokens 5.1 / 3.6 / 3.1 us, 2048 tokens 11.6 /
// 10.7 / 12.2 us, 8192 tokens 33.6 / 33.2 / 37.7 us; 16 + 4 heads of 64 (4
// passes): 2.7 / 2.4 / 2.4, 3.5 / 4.4 / 6.2 and 11.3 / 14.6 / 21.9 us.
constexpr int kRotLong = 8, kRotFew = 512;

// frac(f / 2 pi) * 2^64 of a finite f with |f| < 2^31, to within one: the 53-bit
// mantissa times 128 bits of 1 / (2 pi), of which those that whole turns take are
// shifted out (M. Payne and R. Hanek, "Radian reduction for trigonometric
// functions", 1983).  64 bits of 1 / (2 pi) would leave an error of |f| 2^-66 turns,
// times the position.
__device__ __forceinline__ unsigned long long turn_fraction(double f, bool& bad) {
  // floor(2^130 / (2 pi)), from Machin's formula for pi in integers
  constexpr unsigned long long kInvHi = 0xA2F9836E4E441529ull, kInvLo = 0xFC2757D1F534DDC0ull;
  const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
  const int e = (int)((bits >> 52) & 0x7ff) - 1023;
  if (e >= 31) {  // also infinities and NaN
    bad = true;
    return 0;
  }
  const unsigned long long m = (bits & 0xfffffffffffffull) | (e > -1023 ? 1ull << 52 : 0);
  // the product's upper 128 of 192 bits (the shift drops 64 and more)
  unsigned long long hi = __umul64hi(m, kInvHi), lo = m * kInvHi;
  const unsigned long long below = __umul64hi(m, kInvLo);
  lo += below;
  hi += lo < below ? 1 : 0;
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

// 16 elements of a head (two 8-element chunks) in fp32, as neighbouring pairs.
struct Piece {
  float2 a[4], b[4];
};

__device__ __forceinline__ void widen(const uint4& w, float2 (&x)[4]) {
  x[0] = bf16x2_to_float2(w.x), x[1] = bf16x2_to_float2(w.y);
  x[2] = bf16x2_to_float2(w.z), x[3] = bf16x2_to_float2(w.w);
}

__device__ __forceinline__ uint4 narrow(const float2 (&x)[4]) {
  return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                    pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
}

// Cosines and sines of a lane's eight pairs.
struct Angles {
  float2 c[4], s[4];
};

// Turn the lane's eight pairs: chunk a with chunk b, or neighbours inside each.
template <bool INTER>
__device__ __forceinline__ void turn(Piece& x, const Angles& t) {
  if constexpr (!INTER) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = x.a[e], b = x.b[e];
      x.a[e] = __ffma2_rn(b, make_float2(-t.s[e].x, -t.s[e].y), __fmul2_rn(a, t.c[e]));
      x.b[e] = __ffma2_rn(a, t.s[e], __fmul2_rn(b, t.c[e]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = x.a[e], b = x.b[e];
      const float ca = e & 1 ? t.c[e >> 1].y : t.c[e >> 1].x;
      const float sa = e & 1 ? t.s[e >> 1].y : t.s[e >> 1].x;
      const float cb = e & 1 ? t.c[2 + (e >> 1)].y : t.c[2 + (e >> 1)].x;
      const float sb = e & 1 ? t.s[2 + (e >> 1)].y : t.s[2 + (e >> 1)].x;
      x.a[e] = make_float2(a.x * ca - a.y * sa, a.y * ca + a.x * sa);
      x.b[e] = make_float2(b.x * cb - b.y * sb, b.y * cb + b.x * sb);
    }
  }
}

// x / d rounded to nearest, given r = 1 / d rounded to nearest: the residual of
// x * r is exact in one FMA, and adding it times r gives the correctly rounded
// quotient (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990), as long as no product leaves the normal range.
// The residual is rounded down, which being exact it only notices as the sign of a
// zero: -0 leaves the zero it is added to as it is, where +0 would turn -0 to +0.
__device__ __forceinline__ float2 quotient(float2 x, float2 minus_d, float2 r) {
  const float2 y = __fmul2_rn(x, r);
  return __ffma2_rn(__ffma2_rd(y, minus_d, x), r, y);
}

// Store a row's piece to the 8-bit cache: scale = row max / 448 (1 for an
// all-zero row) over the row's LPR lanes, codes e4m3(x / scale), as
// pa_reshape_and_cache_fp8 defines them, from the fp32 values (a rotated key
// is rounded once, to its code).  codes_at, scale_at: the row's.
template <int D>
__device__ __forceinline__ void store_fp8(unsigned char* codes_at, float* scale_at, int ca, int cb,
                                          int l, const Piece& x, bool on) {
  constexpr int LPR = D / 16;
  float m4[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    m4[e] = fmaxf(fmaxf(fabsf(x.a[e].x), fabsf(x.a[e].y)), fmaxf(fabsf(x.b[e].x), fabsf(x.b[e].y)));
  float amax = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
#pragma unroll
  for (int m = LPR / 2; m >= 1; m >>= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  if (!on) return;
  const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
  const float inv = __frcp_rn(sc);
  const float2 d2 = make_float2(-sc, -sc), r2 = make_float2(inv, inv);
  float2 y[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] = quotient(x.a[e], d2, r2);
    y[4 + e] = quotient(x.b[e], d2, r2);
  }
  // a divider near the ends of fp32's range takes the plain division; elements
  // so small that their residual underflows have the code 0 either way
  if (!(amax >= 1e-18f && amax <= 1e18f)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[e] = make_float2(__fdiv_rn(x.a[e].x, sc), __fdiv_rn(x.a[e].y, sc));
      y[4 + e] = make_float2(__fdiv_rn(x.b[e].x, sc), __fdiv_rn(x.b[e].y, sc));
    }
  }
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = e4m3x2_from_floats(y[e].x, y[e].y);
  *reinterpret_cast<uint2*>(codes_at + ca * 8) =
      make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  *reinterpret_cast<uint2*>(codes_at + cb * 8) =
      make_uint2(w[4] | (w[5] << 16), w[6] | (w[7] << 16));
  if (l == 0) *scale_at = sc;
}

// 2^split_log2 warps share a token's heads.  DEPTH passes of a warp have their
// loads in flight together: three with the bf16 cache (4099 tokens of 16 + 4
// heads of 64, half rotated: 5.9 us, 4.3 TB/s; two: 6.2), two with the 8-bit
// cache, whose codes cost more instructions, at eight CTAs an SM (8191 tokens of
// 32 + 8 heads of 128: 35.0 us, 5.3 TB/s; three: 36.6, before the angles took 128
// bits of 1 / (2 pi)).  Eight leave 64 registers a thread, and those instances
// spill: 20 bytes stored and 68 loaded with halves paired, 4 and 20 interleaved.
template <int D, bool F8, bool INTER>
__global__ void __launch_bounds__(kRotThreads, F8 ? 8 : 6)
    rotary_cache_kernel(const RotaryArgs p, int split_log2) {
  constexpr int DEPTH = F8 ? 2 : 3;
  constexpr int LPR = D / 16;      // lanes of a head: 16 elements each
  constexpr int HEADS = 32 / LPR;  // heads of a pass of the warp
  __shared__ float2 cs_s[kRotWarps][D / 2];
  // (read from lane 0, so that what follows from it is known to be the warp's)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kRotWarps + warp;
  const int64_t t = unit >> split_log2;
  const int split = 1 << split_log2;
  after_prior_kernels();
  if (t >= p.num_tokens) return;
  const int step = HEADS * split;
  const int l = lane % LPR;
  const int h_lane = (int)(unit & (split - 1)) * HEADS + lane / LPR;  // head of the first pass
  const bool rot = l < p.rotary_dim / 16;
  // this lane's two chunks of 8 elements
  int ca = 2 * l, cb = 2 * l + 1;
  if (rot && !INTER) ca = l, cb = l + p.rotary_dim / 16;
  // the passes over the token's heads: queries, then keys, then values
  const int nq = (p.n_q + step - 1) / step, nk = (p.n_kv + step - 1) / step;
  const int passes = nq + 2 * nk;
  const uint16_t* q = p.q + t * p.q_stride;
  const uint16_t* k = p.k + t * p.k_stride;
  const uint16_t* v = p.v + t * p.v_stride;
  uint4 wa[DEPTH], wb[DEPTH];
  auto load = [&](int i, int pass) {
    const bool is_q = pass < nq, is_v = pass >= nq + nk;
    const int h = h_lane + (is_q ? pass : is_v ? pass - nq - nk : pass - nq) * step;
    wa[i] = wb[i] = make_uint4(0u, 0u, 0u, 0u);
    if (pass < passes && h < (is_q ? p.n_q : p.n_kv)) {
      const uint16_t* src = (is_q ? q : is_v ? v : k) + h * D;
      wa[i] = *reinterpret_cast<const uint4*>(src + ca * 8);
      wb[i] = *reinterpret_cast<const uint4*>(src + cb * 8);
    }
  };
  // the first passes' loads; their wait covers the angles' arithmetic
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) load(i, i);
  int64_t slot = p.slot_mapping[t];
  bool bad = false;
  for (int i = lane; i < p.rotary_dim / 2; i += 32) cs_s[warp][i] = pair_cos_sin(p, t, i, bad);
  __syncwarp();
  if (slot >= p.num_slots) bad = true, slot = -1;
  Angles cs;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 u = rot ? cs_s[warp][8 * l + 2 * e] : make_float2(1.f, 0.f);
    const float2 w = rot ? cs_s[warp][8 * l + 2 * e + 1] : make_float2(1.f, 0.f);
    cs.c[e] = make_float2(u.x, w.x), cs.s[e] = make_float2(u.y, w.y);
  }
  uint16_t* q_out = p.q_out + t * p.n_q * D;
  // the token's row in the caches: of values, or (8-bit) of codes and scales
  int64_t row = slot * p.n_kv * (int64_t)(2 * D), scales = 0;
  if (F8) {
    row = (slot / kFp8PageTokens) * fp8_page_bytes(p.n_kv, D);
    const int r = (int)(slot % kFp8PageTokens) * p.n_kv;
    scales = row + fp8_scales_offset(p.n_kv, D) + r * 4;
    row += r * D;
  }
  for (int p0 = 0; p0 < passes; p0 += DEPTH) {
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
      const int pass = p0 + i;
      if (pass >= passes) break;
      const bool is_q = pass < nq, is_v = pass >= nq + nk;
      const int h = h_lane + (is_q ? pass : is_v ? pass - nq - nk : pass - nq) * step;
      unsigned char* cache = static_cast<unsigned char*>(is_v ? p.v_cache : p.k_cache);
      if (F8 && !is_q) {
        // from fp32 (a turned key is rounded once, to its code); every lane of
        // the warp takes part in the row maximum's shuffles
        Piece x;
        widen(wa[i], x.a);
        widen(wb[i], x.b);
        if (rot && !is_v) turn<INTER>(x, cs);
        store_fp8<D>(cache + row + h * D, reinterpret_cast<float*>(cache + scales) + h, ca, cb, l,
                     x, slot >= 0 && h < p.n_kv);
      } else if (is_q ? h < p.n_q : slot >= 0 && h < p.n_kv) {
        if (rot && !is_v) {
          Piece x;
          widen(wa[i], x.a);
          widen(wb[i], x.b);
          turn<INTER>(x, cs);
          wa[i] = narrow(x.a);
          wb[i] = narrow(x.b);
        }
        uint16_t* dst = is_q ? q_out + h * D : reinterpret_cast<uint16_t*>(cache + row) + h * D;
        *reinterpret_cast<uint4*>(dst + ca * 8) = wa[i];
        *reinterpret_cast<uint4*>(dst + cb * 8) = wb[i];
      }
      load(i, pass + DEPTH);
    }
  }
  if (bad) flag_error(p.err, DEVERR_BOUNDS);
}

}  // namespace

template <int D, bool F8>
static cudaError_t launch_rotary_t(const RotaryArgs& p, cudaStream_t stream) {
  constexpr int HEADS = 32 / (D / 16);
  const int passes = (p.n_q + HEADS - 1) / HEADS + 2 * ((p.n_kv + HEADS - 1) / HEADS);
  const int split = (passes >= kRotLong ? 1 : 0) + (p.num_tokens <= kRotFew ? 1 : 0);
  const int64_t warps = (int64_t)p.num_tokens << split;
  const unsigned grid = (unsigned)((warps + kRotWarps - 1) / kRotWarps);
  return launch_early(p.interleaved ? rotary_cache_kernel<D, F8, true>
                                    : rotary_cache_kernel<D, F8, false>,
                      dim3(grid), dim3(kRotThreads), 0, stream, 1, p, split);
}

cudaError_t launch_rotary_cache(const RotaryArgs& p, cudaStream_t stream) {
  if (p.head_dim == 128)
    return p.fp8 ? launch_rotary_t<128, true>(p, stream) : launch_rotary_t<128, false>(p, stream);
  if (p.head_dim == 64)
    return p.fp8 ? launch_rotary_t<64, true>(p, stream) : launch_rotary_t<64, false>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
