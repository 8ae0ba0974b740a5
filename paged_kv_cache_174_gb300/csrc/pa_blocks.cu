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
// length 2 d: at most 2^22 in size, exact in fp32 together with the powers of two.
// So the choice is the same for any order of the sums, and ties are real ties (the
// lowest index wins).
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
// A warp for each (block, kv head): a lane holds four channels and reads every
// row's four, 16 rows' loads in flight.  Memory is the bound for whole caches, one
// round trip of loads for a decode step.
constexpr int kBoundWarps = 8;

template <int D, bool F8>
__global__ void __launch_bounds__(kBoundWarps * 32) bounds_kernel(const BoundsArgs p) {
  constexpr int LPR = D / 4;          // lanes of a row
  constexpr int RPL = 32 / LPR;       // rows of a load
  constexpr int LOADS = 16 / RPL;     // loads of 16 rows
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kBoundWarps + (threadIdx.x >> 5);
  const int h = (int)(unit % p.n_kv);
  const long long slot = unit / p.n_kv;
  after_prior_kernels();
  if (slot >= p.slots) return;
  int s, col;
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
    const int a = p.query_start_loc[s], b = p.query_start_loc[s + 1], L = p.seq_lens[s];
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
    const int L = p.seq_lens[s];
    if (L < 0 || L > (long long)p.max_blocks << p.block_log2) {
      if (col == 0 && lane == 0) flag_error(p.err, DEVERR_BOUNDS);
      return;
    }
    if (((long long)col << p.block_log2) >= L) return;
  }
  const int rows = min(p.seq_lens[s] - (col << p.block_log2), 1 << p.block_log2);
  const int id = p.block_tables[(int64_t)s * p.max_blocks + col];
  if (id < 0 || id >= p.num_blocks) {
    if (lane == 0) flag_error(p.err, DEVERR_BOUNDS);
    return;
  }
  float hi[4], lo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) hi[j] = -INFINITY, lo[j] = INFINITY;
  const int sub = lane / LPR, c4 = lane % LPR;
  for (int r0 = 0; r0 < rows; r0 += 16) {
    float x[LOADS][4];
    if constexpr (F8) {
      const int64_t page = ((int64_t)id << (p.block_log2 - 4)) + (r0 >> 4);
      const uint8_t* at = static_cast<const uint8_t*>(p.k_cache) + page * fp8_page_bytes(p.n_kv, D);
      const float* scales = reinterpret_cast<const float*>(at + fp8_scales_offset(p.n_kv, D));
      uint32_t w[LOADS];
      float sc[LOADS];
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int r = i * RPL + sub;
        w[i] = 0, sc[i] = 0.f;
        if (r0 + r < rows) {
          w[i] = *reinterpret_cast<const uint32_t*>(at + ((int64_t)r * p.n_kv + h) * D + c4 * 4);
          sc[i] = scales[r * p.n_kv + h];
        }
      }
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        uint32_t a, b;
        f16x2x2_from_e4m3x4(w[i], a, b);
        const float2 f = half2_bits_to_float2(a), g = half2_bits_to_float2(b);
        x[i][0] = f.x * sc[i], x[i][1] = f.y * sc[i], x[i][2] = g.x * sc[i], x[i][3] = g.y * sc[i];
      }
    } else {
      const uint16_t* at = static_cast<const uint16_t*>(p.k_cache) +
                           ((((int64_t)id << p.block_log2) + r0) * p.n_kv + h) * D + c4 * 4;
      uint2 w[LOADS];
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int r = i * RPL + sub;
        w[i] = make_uint2(0u, 0u);
        if (r0 + r < rows) w[i] = *reinterpret_cast<const uint2*>(at + (int64_t)r * p.n_kv * D);
      }
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const float2 f = bf16x2_to_float2(w[i].x), g = bf16x2_to_float2(w[i].y);
        x[i][0] = f.x, x[i][1] = f.y, x[i][2] = g.x, x[i][3] = g.y;
      }
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      if (r0 + i * RPL + sub >= rows) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = finite(x[i][j]);
        hi[j] = fmaxf(hi[j], v);
        lo[j] = fminf(lo[j], v);
      }
    }
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = fmaxf(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], o));
      lo[j] = fminf(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], o));
    }
  }
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(fabsf(hi[j]), fabsf(lo[j])));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int e = code_exponent(top);
  const float inv = power_of_two(-e);
  uint32_t up = 0, down = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    up |= ((uint32_t)(int)ceilf(hi[j] * inv) & 255u) << (8 * j);
    down |= ((uint32_t)(int)floorf(lo[j] * inv) & 255u) << (8 * j);
  }
  int8_t* to = p.bounds + ((int64_t)id * p.n_kv + h) * (2 * D) + c4 * 4;
  if (sub == 0) {
    *reinterpret_cast<uint32_t*>(to) = up;
    *reinterpret_cast<uint32_t*>(to + D) = down;
  }
  if (lane == 0) p.scales[(int64_t)id * p.n_kv + h] = power_of_two(e);
}

// ------------------------------------------------------------------- choice
constexpr int kSelectThreads = 256;
constexpr uint32_t kForced = 0xffffffffu;

// A cluster of CTAs for each (token, kv head), each CTA scoring its share of the
// blocks into its shared memory.  A block's 2 d codes lie over d / 8 lanes, 16 bytes
// each, beside the query codes of the same channels in registers; the G sums of
// several blocks are added up over those lanes by halving (each exchange halves what
// a lane still holds), one shuffle for each sum.
template <int D, int G>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectArgs p) {
  constexpr int LPB = D / 8;               // lanes of a block's codes
  constexpr int BPL = 32 / LPB;            // blocks of a load
  constexpr int U = LPB > G ? LPB / G : 1; // loads of a round: U G sums over LPB lanes
  static_assert(U * G == LPB, "");
  constexpr int kWarps = kSelectThreads / 32;
  extern __shared__ uint32_t keys[];  // table entries first, then the blocks' keys
  __shared__ SelectShared B;
  __shared__ __align__(16) int8_t codes[G][2 * D];
  __shared__ float unit_q[G];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ctas = cluster_size(), rank = cluster_rank();
  const long long unit = blockIdx.x / ctas;
  const int h = (int)(unit % p.n_kv);
  const int t = (int)(unit / p.n_kv);
  after_prior_kernels();
  // the token's request: the last that starts at or before it
  int begun = 0;
  for (int s0 = 0; s0 < p.num_seqs; s0 += kSelectThreads) {
    const int n = __syncthreads_count(s0 + tid < p.num_seqs &&
                                      p.query_start_loc[s0 + tid] <= t);
    begun += n;
    if (n < kSelectThreads) break;
  }
  if (begun == 0) return;
  const int s = begun - 1;
  const int a = p.query_start_loc[s], b = p.query_start_loc[s + 1], L = p.seq_lens[s];
  if (t >= b) return;  // behind the last sequence
  if (a < 0 || b > p.num_tokens || L < b - a || L > p.max_seq_len ||
      L > (long long)p.max_blocks << p.block_log2) {
    if (tid == 0) flag_error(p.err, DEVERR_BOUNDS);
    return;
  }
  const int pos = L - (b - t);
  const int visible = (pos >> p.block_log2) + 1;
  int32_t* out = p.selected + ((int64_t)t * p.n_kv + h) * p.num_selected;
  if (visible <= p.num_selected) {  // all of them
    for (int i = rank * kSelectThreads + tid; i < p.num_selected; i += ctas * kSelectThreads)
      out[i] = i < visible ? i : -1;
    return;
  }
  const int per = (visible + (int)ctas - 1) / (int)ctas;
  const int first = min((int)rank * per, visible), n = min(per, visible - first);
  const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks + first;
  for (int i = tid; i < n; i += kSelectThreads) keys[i] = (uint32_t)table[i];
  // the query's codes: a warp for each head of the group, four channels a lane
  for (int g = warp; g < G; g += kWarps) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (lane < D / 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(
          p.q + ((int64_t)t * p.n_kv * G + h * G + g) * D + lane * 4);
      const float2 f = bf16x2_to_float2(w.x), v = bf16x2_to_float2(w.y);
      x[0] = finite(f.x), x[1] = finite(f.y), x[2] = finite(v.x), x[3] = finite(v.y);
    }
    float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = code_exponent(top);
    const float inv = power_of_two(-e);
    uint32_t up = 0, down = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = (int)rintf(x[j] * inv);
      up |= ((uint32_t)max(c, 0) & 255u) << (8 * j);
      down |= ((uint32_t)min(c, 0) & 255u) << (8 * j);
    }
    if (lane < D / 4) {
      *reinterpret_cast<uint32_t*>(&codes[g][lane * 4]) = up;
      *reinterpret_cast<uint32_t*>(&codes[g][D + lane * 4]) = down;
    }
    if (lane == 0) unit_q[g] = power_of_two(e);
  }
  __syncthreads();
  const int l = lane % LPB, sub = lane / LPB;
  uint4 q[G];
#pragma unroll
  for (int g = 0; g < G; ++g) q[g] = *reinterpret_cast<const uint4*>(&codes[g][l * 16]);
  const float mine_q = unit_q[l % G];  // of the sum that this lane is left with
  constexpr int STEP = BPL * U;        // blocks of a warp's round
  for (int i0 = warp * STEP; i0 < n; i0 += kWarps * STEP) {
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * BPL + sub;
      const uint32_t id = i < n ? keys[i] : ~0u;
      w[u] = make_uint4(0u, 0u, 0u, 0u);
      if (id < (uint32_t)p.num_blocks)
        w[u] = __ldg(reinterpret_cast<const uint4*>(p.bounds + ((int64_t)id * p.n_kv + h) *
                                                                   (2 * D) + l * 16));
    }
    const int mine = i0 + (l / G) * BPL + sub;  // the block of the sum left to this lane
    const uint32_t id = mine < n ? keys[mine] : ~0u;
    const bool known = id < (uint32_t)p.num_blocks;
    const float unit = known ? __ldg(p.scales + (int64_t)id * p.n_kv + h) : 0.f;
    if (mine < n && !known && l % G == 0) flag_error(p.err, DEVERR_BOUNDS);
    int v[LPB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        int x = __dp4a((int)w[u].x, (int)q[g].x, 0);
        x = __dp4a((int)w[u].y, (int)q[g].y, x);
        x = __dp4a((int)w[u].z, (int)q[g].z, x);
        v[u * G + g] = __dp4a((int)w[u].w, (int)q[g].w, x);
      }
    }
#pragma unroll
    for (int o = LPB / 2; o > 0; o >>= 1) {
      const bool up = l & o;
#pragma unroll
      for (int j = 0; j < o; ++j) {
        const int give = up ? v[j] : v[j + o];
        const int keep = up ? v[j + o] : v[j];
        v[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
    float score = (float)v[0] * mine_q * unit;
#pragma unroll
    for (int o = 1; o < G; o <<= 1)
      score = fmaxf(score, __shfl_xor_sync(0xffffffffu, score, o));
    __syncwarp();  // the round's table entries have been read
    if (mine < n && l % G == 0) {
      const int c = first + mine;
      const bool forced = c < p.num_sinks || c >= visible - p.num_recent;
      keys[mine] = forced ? kForced : known ? ordered_key(score) : 0u;
    }
  }
  __syncthreads();
  const Threshold th = select_threshold(B, n, (uint32_t)p.num_selected, ctas,
                                        [&](int i) { return keys[i]; });
  // each thread a run of blocks, of odd length (no bank conflicts)
  const int run = (n + kSelectThreads - 1) / kSelectThreads | 1;
  const int lo = min(tid * run, n), hi = min(lo + run, n);
  uint32_t above = 0, equal = 0;
  for (int i = lo; i < hi; ++i) {
    above += keys[i] > th.key;
    equal += keys[i] == th.key;
  }
  uint32_t pre_above, pre_equal, all_above, all_equal;
  block_scan2(B, above, equal, pre_above, pre_equal, all_above, all_equal);
  if (ctas > 1) {
    if (tid == 0) B.mine[0] = all_above, B.mine[1] = all_equal;
    cluster_sync();
    for (uint32_t r = 0; r < rank; ++r) {
      pre_above += ld_cluster_u32(cluster_addr(smem_addr(&B.mine[0]), r));
      pre_equal += ld_cluster_u32(cluster_addr(smem_addr(&B.mine[1]), r));
    }
    cluster_sync();  // no CTA leaves while its counts are read
  }
  for (int i = lo; i < hi; ++i) {
    const uint32_t k = keys[i];
    if (k > th.key || (k == th.key && pre_equal < th.equal))
      out[pre_above + min(pre_equal, th.equal)] = first + i;
    pre_above += k > th.key;
    pre_equal += k == th.key;
  }
}

template <int D, int G>
cudaError_t launch_select_t(const SelectArgs& p, int ctas, size_t smem, cudaStream_t stream) {
  auto kern = select_kernel<D, G>;
  if (smem > 32 * 1024) {
    // (always the most any call takes, so that calls on other threads agree)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSelectMaxShare * 4);
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = (unsigned)((long long)p.num_tokens * p.n_kv * ctas);
  return launch_early(kern, dim3(grid), dim3(kSelectThreads), smem, stream, ctas, p);
}

template <int D>
cudaError_t launch_select_d(const SelectArgs& p, int ctas, size_t smem, cudaStream_t stream) {
  switch (p.group) {
    case 1: return launch_select_t<D, 1>(p, ctas, smem, stream);
    case 2: return launch_select_t<D, 2>(p, ctas, smem, stream);
    case 4: return launch_select_t<D, 4>(p, ctas, smem, stream);
    default: return launch_select_t<D, 8>(p, ctas, smem, stream);
  }
}

}  // namespace

cudaError_t launch_bounds(BoundsArgs p, cudaStream_t stream) {
  p.slots = p.query_start_loc ? (long long)(p.num_tokens >> p.block_log2) + 2ll * p.num_seqs
                              : (long long)p.num_seqs * p.max_blocks;
  const long long ctas = (p.slots * p.n_kv + kBoundWarps - 1) / kBoundWarps;
  if (ctas <= 0) return cudaSuccess;
  const dim3 grid((unsigned)ctas), block(kBoundWarps * 32);
  if (p.head_dim == 128)
    return p.fp8 ? launch_early(bounds_kernel<128, true>, grid, block, 0, stream, 1, p)
                 : launch_early(bounds_kernel<128, false>, grid, block, 0, stream, 1, p);
  return p.fp8 ? launch_early(bounds_kernel<64, true>, grid, block, 0, stream, 1, p)
               : launch_early(bounds_kernel<64, false>, grid, block, 0, stream, 1, p);
}

cudaError_t launch_select(const SelectArgs& p, int sm_count, cudaStream_t stream) {
  const long long blocks = ((long long)p.max_seq_len + (1 << p.block_log2) - 1) >> p.block_log2;
  const long long units = (long long)p.num_tokens * p.n_kv;
  int ctas = 1;
  while (ctas < 8 && ((blocks + ctas - 1) / ctas > kSelectMaxShare ||
                      (units * ctas < 2ll * sm_count && blocks > 256ll * ctas)))
    ctas *= 2;
  const size_t smem = (size_t)((blocks + ctas - 1) / ctas) * 4;
  return p.head_dim == 128 ? launch_select_d<128>(p, ctas, smem, stream)
                           : launch_select_d<64>(p, ctas, smem, stream);
}

}  // namespace pa
