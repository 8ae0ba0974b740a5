// pa_rows.cuh -- attention of one token's query heads of one kv head over 16-token
// pages of the cache, by a warp: what the attention over chosen blocks (pa_sparse.cu)
// and the weighing decode (pa_weights.cu) share.
//
// A page is 16 keys of one kv head.  Both products are m16n8k16 on the tensor cores
// with the query heads as rows 0..7 of A: S = Q K^T takes K rows as they lie in memory
// as its B operand (the channels of a k step may be any as long as q's agree, so a lane
// loads 16 contiguous bytes of a key and has the operands of two or four steps), and
// S's accumulator layout is the A layout of O += P V.  V's operand pairs two keys of a
// channel: two rows' words are interleaved in registers.  Nothing goes through shared
// memory, so the loads of several pages per SM are in flight with no ring to manage;
// the products are a few percent of the time.
//
// P is split into two bf16, p = hi + lo: lo takes the otherwise idle rows 8..15, so O
// has the weights to 2^-17 and the row sums are of the fp32 values.
// 8-bit cache: K codes become f16 (exact) against q as f16 (divided by a power of two
// near its largest element, so that what q's rounding loses is below 2^-24 of that);
// V codes become bf16 (exact) and their scales multiply p before it is split.
#pragma once

#include <cstdint>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_select.cuh"

namespace pa {

__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A page's rows are read once by an SM: past L1.
__device__ __forceinline__ uint4 ld_page16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_page8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}

// The request of token t (all threads of the block; uniform), or false: a row behind
// the last sequence, or lengths out of range (flagged by one thread).
struct TokenRequest {
  int s, pos, len, rows;
};
__device__ __forceinline__ bool find_request(const int32_t* qsl, const int32_t* seq_lens,
                                             int num_seqs, int num_tokens, long long most, int t,
                                             unsigned* err, bool report, TokenRequest& R) {
  int begun = 0;
  for (int s0 = 0; s0 < num_seqs; s0 += blockDim.x) {
    const int n = __syncthreads_count(s0 + (int)threadIdx.x < num_seqs &&
                                      qsl[s0 + threadIdx.x] <= t);
    begun += n;
    if (n < (int)blockDim.x) break;
  }
  if (begun == 0) return false;
  R.s = begun - 1;
  const int a = qsl[R.s], b = qsl[R.s + 1];
  R.len = seq_lens[R.s];
  R.rows = b - a;
  if (t >= b) return false;
  if (a < 0 || b > num_tokens || R.len < R.rows || R.len > most) {
    if (report) flag_error(err, DEVERR_BOUNDS);
    return false;
  }
  R.pos = R.len - (b - t);
  return true;
}

template <int D, int G, bool F8>
struct WarpRows {
  static constexpr int STEPS = D / 16;            // k steps of S
  static constexpr int KC = F8 ? D / 64 : D / 32; // 16-byte chunks of a key for a lane
  static constexpr int VW = F8 ? D / 32 : D / 16; // words of a V row for a lane
  static constexpr int TILES = D / 8;             // 8-channel tiles of O
  uint32_t q0[STEPS], q2[STEPS];
  float o[TILES][4];
  float m, l;      // of head lane / 4: reference max (log2 units), this lane's share of the sum
  float mul;       // score to log2 units (8-bit cache: to be multiplied by the key's scale)
  uint4 k[2][KC];  // keys lane / 4 and lane / 4 + 8
  float ks;        // 8-bit cache: K scale of key lane % 16 (lanes 0-15), V scale (16-31)

  // q: the token's G heads of this kv head
  __device__ __forceinline__ void begin(const uint16_t* q, float scale_log2) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    m = -INFINITY;
    l = 0.f;
    mul = scale_log2;
#pragma unroll
    for (int n = 0; n < TILES; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    if constexpr (!F8) {
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (g < G) w = __ldg(reinterpret_cast<const uint4*>(q + g * D + (4 * j + t) * 8));
        q0[2 * j] = w.x, q2[2 * j] = w.y, q0[2 * j + 1] = w.z, q2[2 * j + 1] = w.w;
      }
    } else {
      uint32_t w[KC][8];
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
        if (g < G) {
          const uint4* at = reinterpret_cast<const uint4*>(q + g * D + (4 * j + t) * 16);
          a = __ldg(at), b = __ldg(at + 1);
        }
        w[j][0] = a.x, w[j][1] = a.y, w[j][2] = a.z, w[j][3] = a.w;
        w[j][4] = b.x, w[j][5] = b.y, w[j][6] = b.z, w[j][7] = b.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = bf16x2_to_float2(w[j][i]);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the power of two below the largest element (its reciprocal is normal too)
      const int e = min(max((int)(__float_as_uint(top) >> 23), 1), 253);
      const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
      mul *= __uint_as_float((uint32_t)e << 23);
#pragma unroll
      for (int j = 0; j < KC; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = bf16x2_to_float2(w[j][2 * i]), h = bf16x2_to_float2(w[j][2 * i + 1]);
          q0[4 * j + i] = f16x2_from_floats(f.x * inv, f.y * inv);
          q2[4 * j + i] = f16x2_from_floats(h.x * inv, h.y * inv);
        }
      }
    }
  }

  // Row r of a page: its first byte for kv head h.
  static __device__ __forceinline__ const uint8_t* row(const uint8_t* page, int r, int n_kv,
                                                       int h) {
    return page + ((int64_t)r * n_kv + h) * (F8 ? D : 2 * D);
  }
  static __device__ __forceinline__ int64_t page_bytes(int n_kv) {
    return F8 ? fp8_page_bytes(n_kv, D) : (int64_t)16 * n_kv * D * 2;
  }

  __device__ __forceinline__ void load_k(const uint8_t* k_page, const uint8_t* v_page, int n_kv,
                                         int h) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint8_t* at = row(k_page, g + 8 * n, n_kv, h) + t * 16;
#pragma unroll
      for (int j = 0; j < KC; ++j) k[n][j] = ld_page16(at + j * 64);
    }
    if constexpr (F8) {
      const uint8_t* page = lane < 16 ? k_page : v_page;
      ks = __ldg(reinterpret_cast<const float*>(page + fp8_scales_offset(n_kv, D)) +
                 (lane & 15) * n_kv + h);
    }
  }
  // The rows 2t, 2t + 1, 2t + 8, 2t + 9 of a V page, this lane's channels.
  __device__ __forceinline__ void load_v(const uint8_t* v_page, int n_kv, int h,
                                         uint32_t (&v)[4][VW]) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* at = row(v_page, 2 * t + (i & 1) + (i >> 1) * 8, n_kv, h);
      if constexpr (F8 && D == 64) {
        const uint2 w = ld_page8(at + g * 8);
        v[i][0] = w.x, v[i][1] = w.y;
      } else {
#pragma unroll
        for (int c = 0; c < VW / 4; ++c) {
          const uint4 w = ld_page16(at + c * 128 + g * 16);
          v[i][4 * c] = w.x, v[i][4 * c + 1] = w.y, v[i][4 * c + 2] = w.z, v[i][4 * c + 3] = w.w;
        }
      }
    }
  }

  // x: scores of head lane / 4 with keys 2t, 2t + 1, 2t + 8, 2t + 9 in log2 units; vs:
  // the V scales of those keys.
  __device__ __forceinline__ void scores(float (&x)[4], float (&vs)[4]) const {
    const int t = threadIdx.x & 3;
    float c[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const uint32_t w[4] = {k[n][j].x, k[n][j].y, k[n][j].z, k[n][j].w};
        if constexpr (F8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            f16x2x2_from_e4m3x4(w[i], b0, b1);
            mma_f16_16816(c[n], q0[4 * j + i], 0u, q2[4 * j + i], 0u, b0, b1);
          }
        } else {
          mma_bf16_16816(c[n], q0[2 * j], 0u, q2[2 * j], 0u, w[0], w[1]);
          mma_bf16_16816(c[n], q0[2 * j + 1], 0u, q2[2 * j + 1], 0u, w[2], w[3]);
        }
      }
    }
    x[0] = c[0][0] * mul, x[1] = c[0][1] * mul, x[2] = c[1][0] * mul, x[3] = c[1][1] * mul;
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 2 * t + (i & 1) + (i >> 1) * 8;
        x[i] *= __shfl_sync(0xffffffffu, ks, r);
        vs[i] = __shfl_sync(0xffffffffu, ks, 16 + r);
      }
    }
  }

  // Keys at and past `live` of the page are not seen: their scores and what is
  // added of their V rows, which may hold anything, count nothing.
  __device__ __forceinline__ void hide(int live, float (&x)[4], float (&vs)[4],
                                       uint32_t (&v)[4][VW]) const {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * t + (i & 1) + (i >> 1) * 8 < live) continue;
      x[i] = -INFINITY;
      vs[i] = 0.f;
#pragma unroll
      for (int j = 0; j < VW; ++j) v[i][j] = 0u;
    }
  }

  // The running softmax and O += P V.  O is rescaled only when a row's max has grown
  // by more than 2^8: the same reference scales numerator and sum.
  __device__ __forceinline__ void add(const float (&x)[4], const float (&vs)[4],
                                      const uint32_t (&v)[4][VW]) {
    float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    if (__any_sync(0xffffffffu, mx > m + 8.f)) {
      const float to = fmaxf(m, mx);
      const float alpha = to == -INFINITY ? 1.f : fast_exp2(m - to);
      l *= alpha;
      m = to;
#pragma unroll
      for (int n = 0; n < TILES; ++n) {
        o[n][0] *= alpha, o[n][1] *= alpha, o[n][2] *= alpha, o[n][3] *= alpha;
      }
    }
    const float ref = m == -INFINITY ? 0.f : m;
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = fast_exp2(x[i] - ref);
    l += (p[0] + p[1]) + (p[2] + p[3]);
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] *= vs[i];
    }
    const uint32_t hi0 = pack_bf16x2(p[0], p[1]), hi1 = pack_bf16x2(p[2], p[3]);
    const float2 f0 = bf16x2_to_float2(hi0), f1 = bf16x2_to_float2(hi1);
    const uint32_t lo0 = pack_bf16x2(p[0] - f0.x, p[1] - f0.y);
    const uint32_t lo1 = pack_bf16x2(p[2] - f1.x, p[3] - f1.y);
    if constexpr (F8) {
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        float f[4][4];  // [row][channel]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a, b;
          f16x2x2_from_e4m3x4(v[i][w], a, b);
          const float2 fa = half2_bits_to_float2(a), fb = half2_bits_to_float2(b);
          f[i][0] = fa.x, f[i][1] = fa.y, f[i][2] = fb.x, f[i][3] = fb.y;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_bf16_16816(o[4 * w + j], hi0, lo0, hi1, lo1, pack_bf16x2(f[0][j], f[1][j]),
                         pack_bf16x2(f[2][j], f[3][j]));
      }
    } else {
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        mma_bf16_16816(o[2 * w], hi0, lo0, hi1, lo1, __byte_perm(v[0][w], v[1][w], 0x5410),
                       __byte_perm(v[2][w], v[3][w], 0x5410));
        mma_bf16_16816(o[2 * w + 1], hi0, lo0, hi1, lo1, __byte_perm(v[0][w], v[1][w], 0x7632),
                       __byte_perm(v[2][w], v[3][w], 0x7632));
      }
    }
  }

  // The channel of column c (0 or 1) of O's tile n.
  __device__ __forceinline__ int channel(int n, int c) const {
    const int t = threadIdx.x & 3;
    return F8 ? (2 * t + c) * (D / 8) + n : (n >> 3) * 64 + (2 * t + c) * 8 + (n & 7);
  }
};

// A warp's piece of the result in shared memory, and the CTA's.
template <int D, int G, int W>
struct RowsShared {
  float o[W][G][D];
  float m[W][G], l[W][G];
  float cta_m[G], cta_l[G];  // o[0] is the CTA's once cta_m is
};

// Joins the warps' pieces, then the cluster's; writes G rows of out.  M, L: the rows'
// reference max and sum over the whole cluster (for each head g, in shared memory of
// every CTA afterwards: cta_m, cta_l).  Every thread of the cluster calls it.
template <int D, int G, bool F8, int W>
__device__ __forceinline__ void join_rows(RowsShared<D, G, W>& B, WarpRows<D, G, F8>& R,
                                          uint32_t ctas, uint32_t rank, uint16_t* out) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2;
  R.l += __shfl_xor_sync(0xffffffffu, R.l, 1);
  R.l += __shfl_xor_sync(0xffffffffu, R.l, 2);
  if (g < G) {
#pragma unroll
    for (int n = 0; n < WarpRows<D, G, F8>::TILES; ++n) {
      B.o[warp][g][R.channel(n, 0)] = R.o[n][0] + R.o[n][2];
      B.o[warp][g][R.channel(n, 1)] = R.o[n][1] + R.o[n][3];
    }
    if ((lane & 3) == 0) B.m[warp][g] = R.m, B.l[warp][g] = R.l;
  }
  __syncthreads();
  for (int i = tid; i < G * D; i += W * 32) {
    const int h = i / D, c = i % D;
    float top = B.m[0][h];
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, B.m[w][h]);
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = B.m[w][h] == -INFINITY ? 0.f : fast_exp2(B.m[w][h] - top);
      // (a piece that saw nothing has sum 0, and a sum that is NaN stays so)
      sum += f * B.l[w][h];
      acc += f * B.o[w][h][c];
    }
    B.o[0][h][c] = acc;  // (only this thread reads this element of any warp's)
    if (c == 0) B.cta_m[h] = top, B.cta_l[h] = sum;
    if (ctas == 1) out[i] = float_to_bf16_rn(sum == 0.f ? 0.f : acc / sum);
  }
  if (ctas == 1) {
    __syncthreads();
    return;
  }
  cluster_sync();
  const int per = G * D / (int)ctas;
  float top_all[G], sum_all[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    top_all[h] = -INFINITY;
    sum_all[h] = 0.f;
    for (uint32_t r = 0; r < ctas; ++r)
      top_all[h] = fmaxf(top_all[h], ld_cluster_f32(cluster_addr(smem_addr(&B.cta_m[h]), r)));
    for (uint32_t r = 0; r < ctas; ++r) {
      const float m = ld_cluster_f32(cluster_addr(smem_addr(&B.cta_m[h]), r));
      sum_all[h] += (m == -INFINITY ? 0.f : fast_exp2(m - top_all[h])) *
                    ld_cluster_f32(cluster_addr(smem_addr(&B.cta_l[h]), r));
    }
  }
  for (int i = (int)rank * per + tid; i < (int)(rank + 1) * per; i += W * 32) {
    const int h = i / D;
    float top = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
    for (int j = 0; j < G; ++j)
      if (j == h) top = top_all[j], sum = sum_all[j];
    for (uint32_t r = 0; r < ctas; ++r) {
      const float m = ld_cluster_f32(cluster_addr(smem_addr(&B.cta_m[h]), r));
      acc += (m == -INFINITY ? 0.f : fast_exp2(m - top)) *
             ld_cluster_f32(cluster_addr(smem_addr(&B.o[0][0][0] + i), r));
    }
    out[i] = float_to_bf16_rn(sum == 0.f ? 0.f : acc / sum);
  }
  cluster_sync();  // no CTA leaves, or changes its numbers, while they are read
  if (tid == 0) {
#pragma unroll
    for (int h = 0; h < G; ++h) B.cta_m[h] = top_all[h], B.cta_l[h] = sum_all[h];
  }
  __syncthreads();
}

}  // namespace pa
