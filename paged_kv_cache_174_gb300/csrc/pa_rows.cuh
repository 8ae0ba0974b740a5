// pa_rows.cuh -- attention of one token's query heads of one kv head over 16-token
// pages of the cache, by a warp: what the attention over chosen blocks (pa_sparse.cu)
// and the weighing decode (pa_weights.cu) share.
//
// A page is 16 keys of one kv head.  Each warp streams pages through a ring of its own
// in shared memory: one TMA box for a page's K and one for its V (the rows of a head lie
// n_kv rows apart), completion on the stage's mbarrier, and no synchronisation with
// other warps, so that what is in flight is the ring's bytes whatever the warp does.
// Both products are m16n8k16 on the tensor cores, transposed, with the query heads as the
// eight columns, so that no row of a product is idle and O takes 4 d / 16 registers:
// S^T = K Q^T has the page's keys as its 16 rows, O^T += V^T P^T 16 channels.  K's operand
// comes by ldmatrix, V's by ldmatrix.trans, P^T's by transposing S^T's accumulators
// (movmatrix).
//
// P is split into two bf16, p = hi + lo, a product each, so O has the weights to 2^-16
// and the row sums are of the fp32 values.
// 8-bit cache: ldmatrix moves pairs of codes.  K codes become f16 (exact) against q as
// f16 (divided by a power of two near its largest element, so that what q's rounding
// loses is below 2^-24 of that); V codes become bf16 (exact) and their scales multiply
// p before it is split.
#pragma once

#include <cstdint>
#include <cuda.h>

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
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// An 8 x 8 block of 16-bit values (row lane / 4, columns 2 (lane % 4) and the next) transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, int h, int z,
                                              int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(h), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// The request of token t, or false: a row behind the last sequence, or lengths out of
// range (flagged by one thread).  All threads of the block; found: shared memory that one
// of them set to -1 (its x) before a barrier.
struct TokenRequest {
  int s, pos;
};
__device__ __forceinline__ bool find_request(const int32_t* qsl, const int32_t* seq_lens,
                                             int num_seqs, int num_tokens, long long most, int t,
                                             unsigned* err, bool report, int4* found,
                                             TokenRequest& R) {
  // one round of independent loads: every thread looks at requests of its own
  for (int i = threadIdx.x; i < num_seqs; i += blockDim.x) {
    const int a = qsl[i], b = qsl[i + 1], len = seq_lens[i];
    if (a <= t && t < b) *found = make_int4(i, a, b, len);
  }
  __syncthreads();
  const int4 f = *found;
  if (f.x < 0) return false;
  const int rows = f.z - f.y;
  if (f.y < 0 || f.z > num_tokens || f.w < rows || f.w > most) {
    if (report) flag_error(err, DEVERR_BOUNDS);
    return false;
  }
  R.s = f.x;
  R.pos = f.w - (f.z - t);
  return true;
}

constexpr int kRowsWarps = 4;  // of a CTA

// A warp's ring in shared memory, of at most ROOM bytes.
template <int D, bool F8, int ROOM>
struct RowsRing {
  static constexpr int ROW = F8 ? D : 128;              // bytes of a row as it lies there
  static constexpr int PAGE = 16 * (F8 ? D : 2 * D);    // bytes of a K or V page
  static constexpr int STAGE = 2 * PAGE;
  static constexpr int STAGES = ROOM / STAGE < 8 ? ROOM / STAGE : 8;
  static_assert(STAGES >= 2, "");
  static constexpr int BYTES = STAGES * STAGE;          // of a warp
  uint64_t full[kRowsWarps][STAGES];
  int live[kRowsWarps][STAGES];                         // keys of the page that count
  alignas(16) float scales[kRowsWarps][STAGES][32];     // 8-bit cache: 16 of K, 16 of V
  int abort_flag;
  int late;                                             // a wait of settle() was given up too
};

template <int D, int G, bool F8>
struct WarpRows {
  static constexpr int ROW = F8 ? D : 128;  // bytes of a row in a ring
  static constexpr int STEPS = D / 16;      // k steps of S^T, and 16-channel tiles of O^T
  uint32_t q0[STEPS], q2[STEPS];
  float o[STEPS][4];  // channels lane / 4 and 8 on, heads 2 (lane % 4) and the next
  float m[2], l[2];   // of those heads: reference max (log2 units), this lane's share of the sum
  float mul;          // score to log2 units (8-bit cache: to be multiplied by the key's scale)

  // q: the token's G heads of this kv head (its loads come back while the first pages do)
  __device__ __forceinline__ void begin(const uint16_t* q, float scale_log2) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    mul = scale_log2;
#pragma unroll
    for (int n = 0; n < STEPS; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    if constexpr (!F8) {
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        q0[j] = q2[j] = 0u;
        if (g < G) {
          const uint32_t* at = reinterpret_cast<const uint32_t*>(q + g * D + j * 16 + 2 * t);
          q0[j] = __ldg(at), q2[j] = __ldg(at + 4);
        }
      }
    } else {
      // (a product's k step of 16 codes has codes 4t, 4t + 1 where k is 2t, 2t + 1, and the
      // next two where k is 2t + 8, 2t + 9: as a lane gets four codes in a register)
      uint2 w[STEPS];
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        w[j] = make_uint2(0u, 0u);
        if (g < G) w[j] = __ldg(reinterpret_cast<const uint2*>(q + g * D + j * 16 + 4 * t));
        const float2 f = bf16x2_to_float2(w[j].x), v = bf16x2_to_float2(w[j].y);
        top = fmaxf(fmax3(top, fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(v.x), fabsf(v.y)));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the power of two below the head's largest element (its reciprocal is normal too)
      const int e = min(max((int)(__float_as_uint(top) >> 23), 1), 253);
      const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        const float2 f = bf16x2_to_float2(w[j].x), v = bf16x2_to_float2(w[j].y);
        q0[j] = f16x2_from_floats(f.x * inv, f.y * inv);
        q2[j] = f16x2_from_floats(v.x * inv, v.y * inv);
      }
      // the scores' heads are 2t and 2t + 1, not lane / 4: their factors by lane
      const float own = __uint_as_float((uint32_t)e << 23);
      head_mul[0] = __shfl_sync(0xffffffffu, own, 8 * t);
      head_mul[1] = __shfl_sync(0xffffffffu, own, 8 * t + 4);
    }
  }
  float head_mul[2];  // (8-bit cache)

  // This lane's row of the four 8 x 8 blocks of an ldmatrix over a page: the one of matrices
  // 0-3 is (key half, chunk) = (0, 0) (1, 0) (0, 1) (1, 1); chunk c's is an xor with 16 c away.
  static __device__ __forceinline__ uint32_t k_lane(uint32_t page) {
    const int lane = threadIdx.x & 31, r = (lane & 7) + 8 * ((lane >> 3) & 1), c = lane >> 4;
    return row_at(page, r) ^ (c << 4);
  }
  // The same with (0, 0) (0, 1) (1, 0) (1, 1) for V in 16 bits; V's codes go as K's.
  static __device__ __forceinline__ uint32_t v_lane(uint32_t page) {
    const int lane = threadIdx.x & 31, r = (lane & 7) + 8 * (lane >> 4), c = (lane >> 3) & 1;
    return F8 ? k_lane(page) : row_at(page, r) ^ (c << 4);
  }
  static __device__ __forceinline__ uint32_t row_at(uint32_t page, int r) {
    return ROW == 128 ? page + r * 128 + ((r & 7) << 4) : page + r * 64 + (((r >> 1) & 3) << 4);
  }

  // x: scores of keys lane / 4 (x[0], x[1]) and 8 on with heads 2t and 2t + 1, in log2 units,
  // of the page at k (shared memory); scales: the stage's (8-bit cache).
  __device__ __forceinline__ void scores(uint32_t k, const float* scales, float (&x)[4]) const {
    const uint32_t at = k_lane(k);
    float c[2][4];  // (two chains of products)
#pragma unroll
    for (int n = 0; n < 2; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
    if constexpr (F8) {
#pragma unroll
      for (int j = 0; j < STEPS; j += 2) {  // 16 codes a chunk, two chunks
        uint32_t w[4];
        ldmatrix4(at ^ (j << 4), w);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t a0, a1, a2, a3;
          f16x2x2_from_e4m3x4(w[2 * i], a0, a2);
          f16x2x2_from_e4m3x4(w[2 * i + 1], a1, a3);
          mma_f16_16816(c[i], a0, a1, a2, a3, q0[j + i], q2[j + i]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {  // 8 values a chunk, two chunks
        uint32_t w[4];
        ldmatrix4((at ^ ((2 * j & 7) << 4)) + (j >> 2) * 2048, w);
        mma_bf16_16816(c[j & 1], w[0], w[1], w[2], w[3], q0[j], q2[j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (c[0][i] + c[1][i]) * mul;
    if constexpr (F8) {
      const int g = (threadIdx.x & 31) >> 2;
      const float a = scales[g], b = scales[g + 8];
      x[0] *= a * head_mul[0], x[1] *= a * head_mul[1];
      x[2] *= b * head_mul[0], x[3] *= b * head_mul[1];
    }
  }

  // Keys at and past `live` of the page are not seen.
  __device__ __forceinline__ void hide(int live, float (&x)[4]) const {
    const int g = (threadIdx.x & 31) >> 2;
    if (g >= live) x[0] = x[1] = -INFINITY;
    if (g + 8 >= live) x[2] = x[3] = -INFINITY;
  }

  // The running softmax and O^T += V^T P^T with the V page at v (its rows past the live ones
  // are zeros).  The reference max follows only when a score is more than 2^8 above it: the
  // same reference scales numerator and sum.
  __device__ __forceinline__ void add(const float (&x)[4], uint32_t v, const float* scales) {
    const int g = (threadIdx.x & 31) >> 2;
    const float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
    if (__any_sync(0xffffffffu, mx0 > m[0] + 8.f || mx1 > m[1] + 8.f)) {
      float to[2] = {mx0, mx1};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o_ = 4; o_ < 32; o_ <<= 1)
          to[i] = fmaxf(to[i], __shfl_xor_sync(0xffffffffu, to[i], o_));
        to[i] = fmaxf(to[i], m[i]);
        const float alpha = to[i] == -INFINITY ? 1.f : fast_exp2(m[i] - to[i]);
        l[i] *= alpha;
        m[i] = to[i];
#pragma unroll
        for (int n = 0; n < STEPS; ++n) o[n][i] *= alpha, o[n][i + 2] *= alpha;
      }
    }
    const float r0 = m[0] == -INFINITY ? 0.f : m[0], r1 = m[1] == -INFINITY ? 0.f : m[1];
    float p[4] = {fast_exp2(x[0] - r0), fast_exp2(x[1] - r1), fast_exp2(x[2] - r0),
                  fast_exp2(x[3] - r1)};
    l[0] += p[0] + p[2];
    l[1] += p[1] + p[3];
    if constexpr (F8) {
      const float a = scales[16 + g], b = scales[24 + g];
      p[0] *= a, p[1] *= a, p[2] *= b, p[3] *= b;
    }
    const uint32_t hi0 = pack_bf16x2(p[0], p[1]), hi1 = pack_bf16x2(p[2], p[3]);
    const float2 f0 = bf16x2_to_float2(hi0), f1 = bf16x2_to_float2(hi1);
    const uint32_t bh0 = movmatrix_trans(hi0), bh1 = movmatrix_trans(hi1);
    const uint32_t bl0 = movmatrix_trans(pack_bf16x2(p[0] - f0.x, p[1] - f0.y));
    const uint32_t bl1 = movmatrix_trans(pack_bf16x2(p[2] - f1.x, p[3] - f1.y));
    const uint32_t at = v_lane(v);
    if constexpr (F8) {
      // a register: keys 2t and 2t + 1 (low and high half), codes 2g and 2g + 1 of a chunk;
      // the even codes are the tile's rows 0-7, the odd ones rows 8-15
#pragma unroll
      for (int c = 0; c < STEPS; c += 2) {
        uint32_t w[4];
        ldmatrix4_trans(at ^ (c << 4), w);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t a, b, a8, b8;
          f16x2x2_from_e4m3x4(w[2 * i], a, b);
          f16x2x2_from_e4m3x4(w[2 * i + 1], a8, b8);
          const float2 fa = half2_bits_to_float2(a), fb = half2_bits_to_float2(b);
          const float2 ga = half2_bits_to_float2(a8), gb = half2_bits_to_float2(b8);
          const uint32_t a0 = pack_bf16x2(fa.x, fb.x), a1 = pack_bf16x2(fa.y, fb.y);
          const uint32_t a2 = pack_bf16x2(ga.x, gb.x), a3 = pack_bf16x2(ga.y, gb.y);
          mma_bf16_16816(o[c + i], a0, a1, a2, a3, bh0, bh1);
          mma_bf16_16816(o[c + i], a0, a1, a2, a3, bl0, bl1);
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < STEPS; ++n) {
        uint32_t w[4];
        ldmatrix4_trans((at ^ ((2 * n & 7) << 4)) + (n >> 2) * 2048, w);
        mma_bf16_16816(o[n], w[0], w[1], w[2], w[3], bh0, bh1);
        mma_bf16_16816(o[n], w[0], w[1], w[2], w[3], bl0, bl1);
      }
    }
  }

  // The channel of the first or second row (0 or 1) of this lane in O^T's tile n.
  __device__ __forceinline__ int channel(int n, int second) const {
    const int g = (threadIdx.x & 31) >> 2;
    return n * 16 + (F8 ? 2 * g + second : g + 8 * second);
  }
};

// The stages of a warp's ring, in the order of its pages: stage c % STAGES, use c / STAGES.
template <int D, bool F8, int ROOM>
struct RowsStream {
  using Ring = RowsRing<D, F8, ROOM>;
  Ring& B;
  unsigned char* smem;  // this warp's stages
  const uint8_t* kc;
  const uint8_t* vc;
  const CUtensorMap* kmap;
  const CUtensorMap* vmap;
  unsigned* err;
  int n_kv, h, warp, lane;
  uint32_t issued = 0;

  // The copies of a page (of which the first `live` keys count) into the next stage,
  // whose last page this warp has finished with.
  __device__ __forceinline__ void issue(int page, int live, bool with_v) {
    const uint32_t st = issued % Ring::STAGES;
    const uint32_t bar = smem_addr(&B.full[warp][st]);
    const uint32_t to = smem_addr(smem + st * Ring::STAGE);
    if (lane == 0) {
      B.live[warp][st] = live;
      mbar_arrive_expect_tx(bar, with_v ? Ring::STAGE : Ring::PAGE);
      const int z = F8 ? 0 : page * 16, w = F8 ? page : 0;
      tma_load_page(to, kmap, h, z, w, bar);
      if (with_v) tma_load_page(to + Ring::PAGE, vmap, h, z, w, bar);
    }
    if constexpr (F8) {
      const uint8_t* at = (lane < 16 ? kc : vc) + page * fp8_page_bytes(n_kv, D) +
                          fp8_scales_offset(n_kv, D) + ((lane & 15) * n_kv + h) * 4;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                       smem_addr(&B.scales[warp][st][lane])),
                   "l"(at)
                   : "memory");
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
    }
    ++issued;
  }
  // Page c (all lanes): its stage's bytes and how many of its keys count.  The stage's
  // next use is issued by this warp after it is done with this one, so the phase waited
  // for is the current one or the one just completed.  here: it came; where it did not for
  // a lane, the warp issues nothing more.
  __device__ __forceinline__ uint32_t wait(uint32_t c, int& live, bool& here) {
    const uint32_t st = c % Ring::STAGES;
    here = mbar_wait(smem_addr(&B.full[warp][st]), (c / Ring::STAGES) & 1, err, &B.abort_flag);
    live = B.live[warp][st];
    return smem_addr(smem + st * Ring::STAGE);
  }
  // Behind the last page: where a wait was given up, the copies that may still be in flight
  // are waited for (again with a limit), as others will write in their place.
  __device__ __forceinline__ void settle() {
    if (!*static_cast<volatile int*>(&B.abort_flag)) return;
    for (uint32_t c = issued > Ring::STAGES ? issued - Ring::STAGES : 0; c < issued; ++c)
      mbar_wait_landed(smem_addr(&B.full[warp][c % Ring::STAGES]), (c / Ring::STAGES) & 1, err,
                       &B.late);
    __syncwarp();
  }
  __device__ __forceinline__ float* scales(uint32_t c) { return B.scales[warp][c % Ring::STAGES]; }
  // Rows at and past `live` of the V page of page c hold anything: zeros from here on.
  __device__ __forceinline__ void clear_v(uint32_t c, int live) {
    unsigned char* v = smem + (c % Ring::STAGES) * Ring::STAGE + Ring::PAGE;
    constexpr int HALVES = Ring::PAGE / (16 * Ring::ROW), CHUNKS = Ring::ROW / 16;
    for (int i = lane; i < (16 - live) * CHUNKS * HALVES; i += 32) {
      const int hf = i / ((16 - live) * CHUNKS), e = i % ((16 - live) * CHUNKS);
      *reinterpret_cast<uint4*>(v + hf * 16 * Ring::ROW + (live + e / CHUNKS) * Ring::ROW +
                                (e % CHUNKS) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    if (F8 && lane >= 16 + live) scales(c)[lane] = 0.f;
    // (the stage's next copy comes behind these writes)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
  }
};

// What a CTA holds for the join of its warps' results (a warp's O lies where its ring
// was) and of the cluster's: each CTA gets a slice of every CTA's O, and all maxima and
// sums, written by their owners, so that one barrier of the cluster is all they wait for.
constexpr int kRowsMaxCtas = 16;
template <int D, int G>
struct RowsShared {
  float m[kRowsWarps][G], l[kRowsWarps][G];
  float all_m[kRowsMaxCtas][G], all_l[kRowsMaxCtas][G];
  float slice[G * D];    // [CTA][elements of this CTA]
  float top[G], sum[G];  // the rows' reference max and sum over the cluster
  int4 found;
};

// Joins the warps' pieces, then the cluster's; writes G rows of out; B.top and B.sum are
// the rows' afterwards.  Every thread of the cluster calls it, each warp with nothing in
// flight, after a cluster_arrive() of its own (more than one CTA).  smem: the warps' rings,
// STRIDE bytes each.
template <int STRIDE, int D, int G, bool F8>
__device__ __forceinline__ void join_rows(RowsShared<D, G>& B, WarpRows<D, G, F8>& R,
                                          unsigned char* smem, uint32_t ctas, uint32_t rank,
                                          uint16_t* out) {
  constexpr int W = kRowsWarps;
  static_assert(STRIDE >= G * D * 4, "a warp's O in the place of its ring");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, t = lane & 3;
  const auto o_of = [&](int w) { return reinterpret_cast<float*>(smem + w * STRIDE); };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) R.l[i] += __shfl_xor_sync(0xffffffffu, R.l[i], o);
    const int h = 2 * t + i;
    if (h < G) {
      float* o = o_of(warp) + h * D;
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        o[R.channel(n, 0)] = R.o[n][i];
        o[R.channel(n, 1)] = R.o[n][i + 2];
      }
      if (lane < 4) B.m[warp][h] = R.m[i], B.l[warp][h] = R.l[i];
    }
  }
  if (ctas > 1) cluster_wait();  // (every CTA of the cluster runs: it may be written to)
  __syncthreads();
  const int per = G * D / (int)ctas;  // elements of a CTA's slice
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
      acc += f * o_of(w)[i];
    }
    if (ctas == 1) {
      if (c == 0) B.top[h] = top, B.sum[h] = sum;
      out[i] = float_to_bf16_rn(sum == 0.f ? 0.f : acc / sum);
    } else {
      st_cluster_f32(cluster_addr(smem_addr(&B.slice[(int)rank * per + i % per]), i / per), acc);
      // (the threads of a head's first channels tell one CTA each its max and sum)
      if (c < (int)ctas) {
        st_cluster_f32(cluster_addr(smem_addr(&B.all_m[rank][h]), c), top);
        st_cluster_f32(cluster_addr(smem_addr(&B.all_l[rank][h]), c), sum);
      }
    }
  }
  if (ctas == 1) {
    __syncthreads();
    return;
  }
  cluster_sync();
  for (int e = tid; e < per; e += W * 32) {
    const int i = (int)rank * per + e, h = i / D;
    float top = -INFINITY;
    for (uint32_t r = 0; r < ctas; ++r) top = fmaxf(top, B.all_m[r][h]);
    float sum = 0.f, acc = 0.f;
    for (uint32_t r = 0; r < ctas; ++r) {
      const float m = B.all_m[r][h], f = m == -INFINITY ? 0.f : fast_exp2(m - top);
      sum += f * B.all_l[r][h];
      acc += f * B.slice[r * per + e];
    }
    out[i] = float_to_bf16_rn(sum == 0.f ? 0.f : acc / sum);
  }
  if (tid < G) {
    float top = -INFINITY, sum = 0.f;
    for (uint32_t r = 0; r < ctas; ++r) top = fmaxf(top, B.all_m[r][tid]);
    for (uint32_t r = 0; r < ctas; ++r) {
      const float m = B.all_m[r][tid];
      sum += (m == -INFINITY ? 0.f : fast_exp2(m - top)) * B.all_l[r][tid];
    }
    B.top[tid] = top, B.sum[tid] = sum;
  }
  __syncthreads();
}

// Barriers of the CTA's rings (every thread; before any other use), and the tensor maps on
// their way ahead of the first copy.
template <int D, bool F8, int ROOM>
__device__ __forceinline__ void init_rings(RowsRing<D, F8, ROOM>& B, int4* found,
                                           const CUtensorMap* kmap, const CUtensorMap* vmap) {
  using Ring = RowsRing<D, F8, ROOM>;
  if (threadIdx.x == 0) {
    found->x = -1;
    for (int w = 0; w < kRowsWarps; ++w)
      for (int i = 0; i < Ring::STAGES; ++i) mbar_init(smem_addr(&B.full[w][i]), F8 ? 33 : 1);
    B.abort_flag = B.late = 0;
    fence_mbar_init();
  } else if (threadIdx.x == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(vmap)) : "memory");
  }
  __syncthreads();
}

}  // namespace pa
