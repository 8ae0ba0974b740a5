// pa_blocks.cu -- which blocks of the cache a query attends to: bounds of each
// block's keys, and the choice of blocks by a score from the bounds.
//
// Bounds.  For a block and a kv head, the largest and the smallest value of each
// channel over the block's keys, as 8-bit codes with one power-of-two scale for the
// 2 d of them: p the least power of two with top <= 127 p, codes ceil(max / p) and
// floor(min / p).
//
// Score.  With q's codes rint(q / p_q), p_q by the same rule for each head,
//   score(head, block) = p_q p sum_c x_c (x_c > 0 ? max_c : min_c),  x q's codes,
// bounds the product of q and any key of the block (up to the rounding of q), and a
// kv head's score is the largest of its group's.  The term of a channel is
// x+ max + x- min, so the sum is an integer product of [q+, q-] with [max, min] of
// length 2 d: below 2^21 in size, exact for any order of the sums.  Scores compare by
// that integer and the two exponents (the product of the three leaves fp32's range for
// large or small q and keys), so ties are real ties (the lowest index wins).
#include <cstdint>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_select.cuh"

namespace pa {
namespace {

// The exponent of the least power of two p with top <= 127 p, for finite top >= 0
// (at least -126; top = 0: p = 1).
__device__ __forceinline__ int code_exponent(float top) {
  const uint32_t b = __float_as_uint(top);
  const int e = (int)(b >> 23) - 126 - 7 + ((b & 0x7fffffu) > 63u << 17 ? 1 : 0);
  return b == 0 ? 0 : max(e, -126);
}
__device__ __forceinline__ float power_of_two(int e) {  // -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// NaN as 0, infinities as the largest finite value.
__device__ __forceinline__ float finite(float x) {
  return x != x ? 0.f : fminf(fmaxf(x, -3.402823466e38f), 3.402823466e38f);
}

// ------------------------------------------------------------------- bounds
// A warp for a block and `heads` of its kv heads in turn.  A lane holds 16 bytes of a row
// (8 channels, or 16 codes), a few lanes a row, so a page of 16 rows is two to eight
// loads in flight.  Largest and smallest are kept in pairs of bf16 (exact), or of fp32
// products of code and scale; values that are not finite are found by their bits and
// send the warp through a slower loop.  Whole caches are bound by memory (16 requests of
// 1K to 8K tokens, 8 heads of 128, bf16: 30.7 us, 77% of the copy rate) or, of 8-bit ones,
// by the conversion of the codes (30.3 us); a step by the chain of three loads (3.2 us).
constexpr int kBoundWarps = 8;

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float y;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// The codes of N channels in a row from the largest and smallest values; writes 2^e of the
// block.  Every lane of the warp; those with `store` write at channel c.
template <int D, int N>
__device__ __forceinline__ void store_bounds(const float (&hi)[N], const float (&lo)[N],
                                             int8_t* to, float* scale, int c, bool store) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) top = fmax3(top, fabsf(hi[j]), fabsf(lo[j]));
  // (positive floats order as their bits)
  const int e = code_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top))));
  const float inv = power_of_two(-e);
  constexpr int W = (N + 3) / 4;
  uint32_t up[W], down[W];
#pragma unroll
  for (int w = 0; w < W; ++w) up[w] = down[w] = 0u;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    up[j / 4] |= ((uint32_t)(int)ceilf(hi[j] * inv) & 255u) << (8 * (j % 4));
    down[j / 4] |= ((uint32_t)(int)floorf(lo[j] * inv) & 255u) << (8 * (j % 4));
  }
  if (store) {
    if constexpr (N == 2) {
      *reinterpret_cast<uint16_t*>(to + c) = (uint16_t)up[0];
      *reinterpret_cast<uint16_t*>(to + D + c) = (uint16_t)down[0];
    } else if constexpr (N == 4) {
      *reinterpret_cast<uint32_t*>(to + c) = up[0];
      *reinterpret_cast<uint32_t*>(to + D + c) = down[0];
    } else {
      *reinterpret_cast<uint2*>(to + c) = make_uint2(up[0], up[1]);
      *reinterpret_cast<uint2*>(to + D + c) = make_uint2(down[0], down[1]);
    }
  }
  if ((threadIdx.x & 31) == 0) *scale = power_of_two(e);
}

// Any values: NaN counts as 0, an infinity as the largest finite value.  Four channels
// a lane, row by row.
template <int D, bool F8>
__device__ __noinline__ void slow_bounds(const BoundsArgs& p, int id, int h, int rows) {
  const int lane = threadIdx.x & 31, c = (lane * 4) % D;
  float hi[4], lo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) hi[j] = -INFINITY, lo[j] = INFINITY;
#pragma unroll 1
  for (int r = 0; r < rows; ++r) {
    float x[4];
    if constexpr (F8) {
      const int64_t page = ((int64_t)id << (p.block_log2 - 4)) + (r >> 4);
      const uint8_t* at = static_cast<const uint8_t*>(p.k_cache) + page * fp8_page_bytes(p.n_kv, D);
      const float sc = reinterpret_cast<const float*>(
          at + fp8_scales_offset(p.n_kv, D))[(r & 15) * p.n_kv + h];
      uint32_t a, b;
      f16x2x2_from_e4m3x4(
          *reinterpret_cast<const uint32_t*>(at + ((int64_t)(r & 15) * p.n_kv + h) * D + c), a, b);
      const float2 f = half2_bits_to_float2(a), g = half2_bits_to_float2(b);
      x[0] = f.x * sc, x[1] = f.y * sc, x[2] = g.x * sc, x[3] = g.y * sc;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(
          static_cast<const uint16_t*>(p.k_cache) +
          ((((int64_t)id << p.block_log2) + r) * p.n_kv + h) * D + c);
      const float2 f = bf16x2_to_float2(w.x), g = bf16x2_to_float2(w.y);
      x[0] = f.x, x[1] = f.y, x[2] = g.x, x[3] = g.y;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = finite(x[j]);
      hi[j] = fmaxf(hi[j], v);
      lo[j] = fminf(lo[j], v);
    }
  }
  store_bounds<D, 4>(hi, lo, p.bounds + ((int64_t)id * p.n_kv + h) * (2 * D),
                     p.scales + (int64_t)id * p.n_kv + h, c, lane * 4 < D);
}

// The heads h0 .. h0 + p.heads - 1 of block id, whose first `rows` rows are live; the next
// page's (or head's) loads are in flight while a page is worked on.
template <int D>
__device__ __forceinline__ void bf16_bounds(const BoundsArgs& p, int id, int h0, int rows) {
  constexpr int LPR = D / 8, RPL = 32 / LPR, LOADS = 16 / RPL;
  const int lane = threadIdx.x & 31, sub = lane / LPR, c = (lane % LPR) * 8;
  const int64_t row = (int64_t)p.n_kv * D;
  const uint16_t* at = static_cast<const uint16_t*>(p.k_cache) +
                       (((int64_t)id << p.block_log2) * p.n_kv + h0) * D + c;
  uint32_t hi[4], lo[4], odd = 0u;
  uint4 w[LOADS], next[LOADS];
  const auto load = [&](int h, int r0, uint4 (&to)[LOADS]) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int r = r0 + i * RPL + sub;
      if (r < rows) to[i] = *reinterpret_cast<const uint4*>(at + h * D + r * row);
    }
  };
  load(0, 0, w);
  int h = 0, r0 = 0;
  while (h < p.heads) {
    const bool last = r0 + 16 >= rows;  // page of this head
    const int h1 = last ? h + 1 : h, r1 = last ? 0 : r0 + 16;
    if (h1 < p.heads) load(h1, r1, next);
    if (r0 == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) hi[j] = 0xff80ff80u, lo[j] = 0x7f807f80u;
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      if (r0 + i * RPL + sub >= rows) continue;
      const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        hi[j] = max_bf16x2(hi[j], x[j]);
        lo[j] = min_bf16x2(lo[j], x[j]);
        odd |= (x[j] & 0x7f807f80u) + 0x00800080u;  // (a half's top bit: not finite)
      }
    }
    if (last) {
      if (__any_sync(0xffffffffu, odd & 0x80008000u)) {
        slow_bounds<D, false>(p, id, h0 + h, rows);
        odd = 0u;
      } else {
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            hi[j] = max_bf16x2(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], o));
            lo[j] = min_bf16x2(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], o));
          }
        }
        float up[8], down[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = bf16x2_to_float2(hi[j]), g = bf16x2_to_float2(lo[j]);
          up[2 * j] = f.x, up[2 * j + 1] = f.y, down[2 * j] = g.x, down[2 * j + 1] = g.y;
        }
        const int64_t to = (int64_t)id * p.n_kv + h0 + h;
        store_bounds<D, 8>(up, down, p.bounds + to * (2 * D), p.scales + to, c, sub == 0);
      }
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) w[i] = next[i];
    h = h1, r0 = r1;
  }
}

template <int D>
__device__ __forceinline__ void fp8_bounds(const BoundsArgs& p, int id, int h0, int rows) {
  constexpr int LPR = D / 16, RPL = 32 / LPR, LOADS = 16 / RPL, N = 16 / RPL;
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const int64_t page_bytes = fp8_page_bytes(p.n_kv, D);
  const uint8_t* at = static_cast<const uint8_t*>(p.k_cache) +
                      ((int64_t)id << (p.block_log2 - 4)) * page_bytes;
  float hi[16], lo[16];
  bool odd = false;
  uint4 w[LOADS], next[LOADS];
  float sc[LOADS], next_sc[LOADS];
  const auto load = [&](int h, int r0, uint4 (&to)[LOADS], float (&scale)[LOADS]) {
    const uint8_t* page = at + (r0 >> 4) * page_bytes;
    const float* scales = reinterpret_cast<const float*>(page + fp8_scales_offset(p.n_kv, D));
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      // (a row past the live ones: the page's first one again)
      const int r = r0 + i * RPL + sub < rows ? i * RPL + sub : 0;
      to[i] = *reinterpret_cast<const uint4*>(page + ((int64_t)r * p.n_kv + h) * D + l * 16);
      scale[i] = scales[r * p.n_kv + h];
    }
  };
  load(h0, 0, w, sc);
  int h = 0, r0 = 0;
  while (h < p.heads) {
    const bool last = r0 + 16 >= rows;  // page of this head
    const int h1 = last ? h + 1 : h, r1 = last ? 0 : r0 + 16;
    if (h1 < p.heads) load(h0 + h1, r1, next, next_sc);
    if (r0 == 0) {
#pragma unroll
      for (int j = 0; j < 16; ++j) hi[j] = -INFINITY, lo[j] = INFINITY;
    }
#pragma unroll
    for (int i = 0; i < LOADS; i += 2) {
      const uint32_t x[2][4] = {{w[i].x, w[i].y, w[i].z, w[i].w},
                                {w[i + 1].x, w[i + 1].y, w[i + 1].z, w[i + 1].w}};
      // (448 times the scale has to be finite)
      odd |= !(fabsf(sc[i]) < 7e35f) || !(fabsf(sc[i + 1]) < 7e35f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          odd |= (((x[k][j] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u;  // a NaN code
          uint32_t a, b;
          f16x2x2_from_e4m3x4(x[k][j], a, b);
          const float2 f = half2_bits_to_float2(a), g = half2_bits_to_float2(b);
          v[k][0] = f.x * sc[i + k], v[k][1] = f.y * sc[i + k];
          v[k][2] = g.x * sc[i + k], v[k][3] = g.y * sc[i + k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          hi[4 * j + k] = fmax3(hi[4 * j + k], v[0][k], v[1][k]);
          lo[4 * j + k] = fmin3(lo[4 * j + k], v[0][k], v[1][k]);
        }
      }
    }
    if (last) {
      if (__any_sync(0xffffffffu, odd)) {
        slow_bounds<D, true>(p, id, h0 + h, rows);
        odd = false;
      } else {
        // over the lanes that hold other rows of the same channels, by halves: a lane ends
        // up with N channels
        int c = l * 16;
#pragma unroll
        for (int o = 16, n = 8; o >= LPR; o >>= 1, n >>= 1) {
          const bool up = lane & o;
#pragma unroll
          for (int j = 0; j < n; ++j) {
            const float give_hi = up ? hi[j] : hi[j + n], keep_hi = up ? hi[j + n] : hi[j];
            const float give_lo = up ? lo[j] : lo[j + n], keep_lo = up ? lo[j + n] : lo[j];
            hi[j] = fmaxf(keep_hi, __shfl_xor_sync(0xffffffffu, give_hi, o));
            lo[j] = fminf(keep_lo, __shfl_xor_sync(0xffffffffu, give_lo, o));
          }
          if (up) c += n;
        }
        float up[N], down[N];
#pragma unroll
        for (int j = 0; j < N; ++j) up[j] = hi[j], down[j] = lo[j];
        const int64_t to = (int64_t)id * p.n_kv + h0 + h;
        store_bounds<D, N>(up, down, p.bounds + to * (2 * D), p.scales + to, c, true);
      }
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) w[i] = next[i], sc[i] = next_sc[i];
    h = h1, r0 = r1;
  }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kBoundWarps * 32) bounds_kernel(const __grid_constant__ BoundsArgs p) {
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kBoundWarps + (threadIdx.x >> 5);
  const int parts = p.n_kv / p.heads;
  const int h0 = (int)(unit % parts) * p.heads;
  const long long slot = unit / parts;
  after_prior_kernels();
  if (slot >= p.slots) return;
  int s, col, L;
  if (p.query_start_loc) {
    // Request s has the places from starts[s] / block_size + 2 s on, as many as its
    // new tokens can touch blocks; the request of a place is the last one that
    // begins at or before it.
    int begun = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
      const int i = s0 + lane;
      const bool b = i < p.num_seqs &&
                     (long long)(p.query_start_loc[i] >> p.block_log2) + 2ll * i <= slot;
      const unsigned ball = __ballot_sync(0xffffffffu, b);
      begun += __popc(ball);
      if (ball != 0xffffffffu) break;
    }
    if (begun == 0) return;
    s = begun - 1;
    const int a = p.query_start_loc[s], b = p.query_start_loc[s + 1];
    L = p.seq_lens[s];
    const int ql = b - a;
    if (ql == 0) return;
    const long long nth = slot - ((long long)(a >> p.block_log2) + 2ll * s);
    if (ql < 0 || a < 0 || b > p.num_tokens || L < ql ||
        L > (long long)p.max_blocks << p.block_log2) {
      if (nth == 0 && lane == 0) flag_error(p.err, DEVERR_BOUNDS);
      return;
    }
    const long long c = ((L - ql) >> p.block_log2) + nth;
    if (c > (L - 1) >> p.block_log2) return;
    col = (int)c;
  } else {
    s = (int)(slot / p.max_blocks);
    col = (int)(slot % p.max_blocks);
    L = p.seq_lens[s];
    if (L < 0 || L > (long long)p.max_blocks << p.block_log2) {
      if (col == 0 && lane == 0) flag_error(p.err, DEVERR_BOUNDS);
      return;
    }
    if (((long long)col << p.block_log2) >= L) return;
  }
  const int rows = min(L - (col << p.block_log2), 1 << p.block_log2);
  const int id = p.block_tables[(int64_t)s * p.max_blocks + col];
  if (id < 0 || id >= p.num_blocks) {
    if (lane == 0) flag_error(p.err, DEVERR_BOUNDS);
    return;
  }
  if constexpr (F8)
    fp8_bounds<D>(p, id, h0, rows);
  else
    bf16_bounds<D>(p, id, h0, rows);
}

// ------------------------------------------------------------------- choice
// Threads of a CTA: eight warps where requests have at most kInWarp blocks, else sixteen,
// for the choice by digits.
constexpr int kFewThreads = 256, kManyThreads = 512;
constexpr int kMaxGroup = 8;

// A cluster of CTAs for each (token, kv head), each CTA scoring its share of the
// blocks; the first gets all keys and chooses.  A warp scores 16 blocks at a time on the
// integer tensor cores: blocks are the rows of A, 32 of a block's 2 d codes a product, and
// the group's heads the columns of B (the codes of a product's k may be any as long as
// both sides agree, so a lane's operands of two products are 16 bytes of a block as they
// lie).  Up to kInWarp blocks are chosen from by one warp over its registers, with no
// barriers.
constexpr int kInWarp = 1024;

__device__ __forceinline__ void mma_s8_16832(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A head's sum is held as c 2^(e - 16), e its power of two's exponent: |c| < 2^21 and e
// between -126 and 122 make it at most 2^127 and, where it is no normal number, a multiple of
// 2^-142, so exact.
constexpr float kHeadUnit = 1.f / 65536.f;

// v u as an unsigned number in the order of the scores: v a head's sum, u >= 0 a power of two
// or 0 (of another number the first 22 bits of the product count).  Zero is 2^31, and the rest
// lie above and below it by 10 bits of exponent and 21 of fraction, which hold all of c's.
// (The exponent's field is between 146 and 670, so neither 0 nor kAlways is a score's.)
__device__ __forceinline__ uint32_t score_key(float v, float u) {
  const uint32_t b = __float_as_uint(u);
  const bool low = fabsf(v) < 0x1p-64f;  // (to a normal number, whatever the fraction below)
  const float m =
      v * (low ? 0x1p64f : 1.f) * __uint_as_float((b & 0x7fffffu) | 127u << 23);
  const uint32_t size = ((__float_as_uint(m) & 0x7fffffffu) >> 2) +
                        ((b >> 23) + (low ? 160u - 64u : 160u) << 21);
  if (v == 0.f || b >> 23 == 0) return 0x80000000u;
  return v > 0.f ? 0x80000000u + size : 0x80000000u - size;
}

template <int NJ>
__device__ __forceinline__ void choose_in_warp(const uint32_t* keys, int n, int K, int32_t* out) {
  const int lane = threadIdx.x & 31;
  uint32_t k[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) k[j] = 32 * j + lane < n ? keys[32 * j + lane] : 0u;
  const uint32_t chosen = select_in_warp<NJ>(k, n, K);
  int at = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool mine = chosen >> j & 1u;
    const uint32_t ball = __ballot_sync(0xffffffffu, mine);
    if (mine) out[at + __popc(ball & ((1u << lane) - 1u))] = 32 * j + lane;
    at += __popc(ball);
  }
}

template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    select_kernel(const SelectArgs p) {
  constexpr int J = D / 32;  // 16-byte pieces of a block's codes for a lane
  constexpr int kWarps = THREADS / 32;
  extern __shared__ uint32_t keys[];  // of all blocks; [one CTA] table entries before
  __shared__ SelectShared B;
  __shared__ __align__(16) int8_t codes[kMaxGroup][2 * D];
  __shared__ float unit_q[kMaxGroup];
  __shared__ int4 found;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ctas = cluster_size(), rank = cluster_rank();
  const long long unit = blockIdx.x / ctas;
  const int h = (int)(unit % p.n_kv);
  const int t = (int)(unit / p.n_kv);
  if (tid == 0) found.x = -1;
  __syncthreads();
  if (ctas > 1) cluster_arrive();
  after_prior_kernels();
  // the token's request: every thread looks at some, in one round of loads
  for (int i = tid; i < p.num_seqs; i += THREADS) {
    const int a = p.query_start_loc[i], b = p.query_start_loc[i + 1], len = p.seq_lens[i];
    if (a <= t && t < b) found = make_int4(i, a, b, len);
  }
  // the query's codes: a warp for each head of the group (zeros for heads past it), four
  // channels a lane
  for (int i = warp; i < kMaxGroup; i += kWarps) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (lane < D / 4 && i < p.group) {
      const uint2 w = *reinterpret_cast<const uint2*>(
          p.q + (((int64_t)t * p.n_kv + h) * p.group + i) * D + lane * 4);
      const float2 f = bf16x2_to_float2(w.x), v = bf16x2_to_float2(w.y);
      x[0] = finite(f.x), x[1] = finite(f.y), x[2] = finite(v.x), x[3] = finite(v.y);
    }
    const float most = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    const int e = code_exponent(
        __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most))));
    const float inv = power_of_two(-e);
    uint32_t up = 0, down = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = (int)rintf(x[j] * inv);
      up |= ((uint32_t)max(c, 0) & 255u) << (8 * j);
      down |= ((uint32_t)min(c, 0) & 255u) << (8 * j);
    }
    if (lane < D / 4) {
      *reinterpret_cast<uint32_t*>(&codes[i][lane * 4]) = up;
      *reinterpret_cast<uint32_t*>(&codes[i][D + lane * 4]) = down;
    }
    if (lane == 0) unit_q[i] = power_of_two(e) * kHeadUnit;
  }
  __syncthreads();
  const int4 f = found;
  if (ctas > 1) cluster_wait();  // (the first CTA runs: it may be written to)
  if (f.x < 0) return;  // behind the last sequence
  const int s = f.x, b = f.z, L = f.w;
  if (f.y < 0 || b > p.num_tokens || L < b - f.y || L > p.max_seq_len ||
      L > (long long)p.max_blocks << p.block_log2) {
    if (tid == 0) flag_error(p.err, DEVERR_BOUNDS);
    return;
  }
  const int pos = L - (b - t);
  const int visible = (pos >> p.block_log2) + 1;
  int32_t* out = p.selected + ((int64_t)t * p.n_kv + h) * p.num_selected;
  if (visible <= p.num_selected) {  // all of them
    for (int i = rank * THREADS + tid; i < p.num_selected; i += ctas * THREADS)
      out[i] = i < visible ? i : -1;
    return;
  }
  const int per = (visible + (int)ctas - 1) / (int)ctas;
  const int first = min((int)rank * per, visible), n = min(per, visible - first);
  const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks + first;
  uint32_t* ids = ctas > 1 ? keys + p.max_keys : keys;
  for (int i = tid; i < n; i += THREADS) ids[i] = (uint32_t)table[i];
  __syncthreads();
  const int g = lane >> 2, l = lane & 3;
  // this lane's sums are of heads 2 l and 2 l + 1
  const float uq0 = unit_q[2 * l], uq1 = unit_q[2 * l + 1];
  for (int i0 = warp * 16; i0 < n; i0 += kWarps * 16) {
    uint4 w[2][J];
    float ub[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = i0 + g + 8 * r;
      const uint32_t id = i < n ? ids[i] : ~0u;
      ub[r] = -1.f;  // no such block
      if (id < (uint32_t)p.num_blocks) {
        const int64_t at = (int64_t)id * p.n_kv + h;
        ub[r] = __ldg(p.scales + at);
#pragma unroll
        for (int j = 0; j < J; ++j)
          w[r][j] = __ldg(reinterpret_cast<const uint4*>(p.bounds + at * (2 * D)) + 4 * j + l);
      } else {
#pragma unroll
        for (int j = 0; j < J; ++j) w[r][j] = make_uint4(0u, 0u, 0u, 0u);
        if (i < n && l == 0) flag_error(p.err, DEVERR_BOUNDS);
      }
    }
    int c[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint4 q = *reinterpret_cast<const uint4*>(&codes[g][(4 * j + l) * 16]);
      mma_s8_16832(c, w[0][j].x, w[1][j].x, w[0][j].y, w[1][j].y, q.x, q.y);
      mma_s8_16832(c, w[0][j].z, w[1][j].z, w[0][j].w, w[1][j].w, q.z, q.w);
    }
    __syncwarp();  // (one CTA: the keys take the place of the table entries)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float most = -INFINITY;
      if (2 * l < p.group) most = (float)c[2 * r] * uq0;
      if (2 * l + 1 < p.group) most = fmaxf(most, (float)c[2 * r + 1] * uq1);
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const int mine = i0 + g + 8 * r;
      if (mine < n && l == 0) {
        const int col = first + mine;
        const bool forced = col < p.num_sinks || col >= visible - p.num_recent;
        // (a scale below 0 is that of a table entry that names no block: chosen last)
        const uint32_t key = forced ? kAlways : ub[r] >= 0.f ? score_key(most, ub[r]) : 0u;
        if (ctas > 1)
          st_cluster_u32(cluster_addr(smem_addr(keys + col), 0), key);
        else
          keys[mine] = key;
      }
    }
  }
  group_sync(ctas);
  if (rank > 0) return;
  if (visible <= kInWarp) {
    if (warp == 0) {
      if (visible <= 256)
        choose_in_warp<8>(keys, visible, p.num_selected, out);
      else
        choose_in_warp<kInWarp / 32>(keys, visible, p.num_selected, out);
    }
    return;
  }
  if constexpr (THREADS == kFewThreads) return;  // (no request has more)
  __shared__ uint32_t hist[THREADS == kFewThreads ? 1 : kSelectBins];
  KeyBits seen;
  for (int i = tid; i < visible; i += THREADS) seen.see(keys[i]);
  const Threshold th = select_threshold(B, hist, visible, (uint32_t)p.num_selected,
                                        [&](int i) { return keys[i]; }, seen);
  // each thread a run of blocks, of odd length (no bank conflicts)
  const int run = (visible + THREADS - 1) / THREADS | 1;
  const int lo = min(tid * run, visible), hi = min(lo + run, visible);
  uint32_t above = 0, equal = 0;
  for (int i = lo; i < hi; ++i) {
    above += keys[i] > th.key;
    equal += keys[i] == th.key;
  }
  uint32_t pre_above, pre_equal, all_above, all_equal;
  block_scan2(B, above, equal, pre_above, pre_equal, all_above, all_equal);
  for (int i = lo; i < hi; ++i) {
    const uint32_t k = keys[i];
    if (k > th.key || (k == th.key && pre_equal < th.equal))
      out[pre_above + min(pre_equal, th.equal)] = i;
    pre_above += k > th.key;
    pre_equal += k == th.key;
  }
}

template <int D, int THREADS>
cudaError_t launch_select_t(const SelectArgs& p, int ctas, size_t smem, cudaStream_t stream) {
  auto kern = select_kernel<D, THREADS>;
  if (smem > 32 * 1024) {
    // (always the most any call takes, so that calls on other threads agree)
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectSmem);
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = (unsigned)((long long)p.num_tokens * p.n_kv * ctas);
  return launch_early(kern, dim3(grid), dim3(THREADS), smem, stream, ctas, p);
}

template <int D>
cudaError_t launch_select_d(const SelectArgs& p, int ctas, size_t smem, cudaStream_t stream) {
  return p.max_keys <= kInWarp ? launch_select_t<D, kFewThreads>(p, ctas, smem, stream)
                               : launch_select_t<D, kManyThreads>(p, ctas, smem, stream);
}

}  // namespace

cudaError_t launch_bounds(BoundsArgs p, int sm_count, cudaStream_t stream) {
  p.slots = p.query_start_loc ? (long long)(p.num_tokens >> p.block_log2) + 2ll * p.num_seqs
                              : (long long)p.num_seqs * p.max_blocks;
  // A warp takes several heads in turn, so that it looks its block up once and has the next
  // head's rows in flight, as long as that leaves seven warps an SM.  One, two, four and
  // eight heads a warp: 64 decode rows (1056 pairs) 3.2* 3.7 5.7 9.3 us; four prompts of 4096
  // rows (8256) 12.5 10.6 9.1* 11.2; 16 whole requests of 1K to 8K tokens (65536) 53.3 39.0
  // 33.0 30.7*, 8-bit 54.1 39.4 32.6 30.3*.
  p.heads = 1;
  while (p.heads < p.n_kv && p.slots * p.n_kv >= 2ll * p.heads * 7 * sm_count) p.heads *= 2;
  const long long ctas = (p.slots * (p.n_kv / p.heads) + kBoundWarps - 1) / kBoundWarps;
  if (ctas <= 0) return cudaSuccess;
  const dim3 grid((unsigned)ctas), block(kBoundWarps * 32);
  if (p.head_dim == 128)
    return p.fp8 ? launch_early(bounds_kernel<128, true>, grid, block, 0, stream, 1, p)
                 : launch_early(bounds_kernel<128, false>, grid, block, 0, stream, 1, p);
  return p.fp8 ? launch_early(bounds_kernel<64, true>, grid, block, 0, stream, 1, p)
               : launch_early(bounds_kernel<64, false>, grid, block, 0, stream, 1, p);
}

cudaError_t launch_select(SelectArgs p, int sm_count, cudaStream_t stream) {
  const long long blocks = ((long long)p.max_seq_len + (1 << p.block_log2) - 1) >> p.block_log2;
  const long long units = (long long)p.num_tokens * p.n_kv;
  // CTAs of a cluster: until there are 1.6 an SM, for requests of more than 256 blocks each.
  // One, two, four and eight: 512 pairs of 8 to 256 blocks 10.4* 12.3 19.2 32.7 us; 64 pairs
  // of 6144 to 8192 blocks 70.9 44.2 37.4* 43.1; 8 pairs of 8192 44.2 27.9 18.8 14.2*.  (With
  // scores compared in fp32; by their integers and exponents 10.7, 37.9 and 14.6.)
  int ctas = 1;
  while (ctas < 8 && blocks > 256ll * ctas &&
         (5 * units * ctas < 8ll * sm_count || blocks > 4096ll * ctas))
    ctas *= 2;
  p.max_keys = (int)blocks;
  const size_t smem = (size_t)(ctas > 1 ? blocks + (blocks + ctas - 1) / ctas : blocks) * 4;
  return p.head_dim == 128 ? launch_select_d<128>(p, ctas, smem, stream)
                           : launch_select_d<64>(p, ctas, smem, stream);
}

}  // namespace pa
