// pa_weights.cu -- decode attention that adds up the attention weight of each cached
// token: the requests with one query row of pa_paged_attention_weights.
//
//   out = sum_j w_j v_j,   w_j = exp(scale q k_j) / sum_i exp(scale q k_i),
//   weights[s, h, j] += sum of w_j over the q heads of kv head h
//
// (the new token's entry starts at this call's).  A weight needs its row's sum, known
// after the last key; the scores stay in shared memory until then (4 G bytes a key
// against 4 d of K and V), and those of a cache too long for it are computed again
// from K.  One pass over K and V, so their bytes are the bound.  A cluster takes a
// (request, kv head), each CTA a run of its keys.
// 64 requests of 128 to 4096 tokens, 32 q / 8 kv heads of 128: 101 us, 82% of the copy rate;
// 8-bit 84 us, 52% (each warp's chain of conversions and products, 2.6 warps a scheduler and 46%
// issue, and the last CTAs of a grid of 2.2 for each place); 8 requests of 16384 to 32767 tokens,
// 8-bit, 122 us, 52%.
#include <cstdint>

#include "pa_rows.cuh"
#include "pa_tma_host.h"

namespace pa {
namespace {

// CTAs of an SM (with short contexts; the scores of long ones take the room of some),
// and the bytes of a warp's ring: two pages in flight a warp.  512 pairs with rings of 16 and
// 24 KB 101* 126 us, 8-bit with 8 and 12 KB 84* 90: the longer ones leave room for fewer CTAs.
// Heads of 64 with 8, 12, 16 and 24 KB (5, 4, 3 and 2 CTAs) 65.3* 70.6 69.9 110, 8-bit 64.0* 76.3
// 76.7 76.7.
template <int D, bool F8>
constexpr int kCtas = D == 128 && !F8 ? 3 : 5;
template <int D, bool F8>
constexpr int kRing = (D == 128 && !F8 ? 16 : 8) * 1024;

template <int D, int G, bool F8>
__global__ void __launch_bounds__(kRowsWarps * 32, kCtas<D, F8>)
    weigh_kernel(const WeighArgs p, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  using Ring = RowsRing<D, F8, kRing<D, F8>>;
  constexpr int W = kRowsWarps;
  extern __shared__ __align__(1024) unsigned char rings[];
  float* scores_s = reinterpret_cast<float*>(rings + W * Ring::BYTES);  // [key of the CTA][G]
  __shared__ Ring B;
  __shared__ RowsShared<D, G> J;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
  const uint32_t ctas = cluster_size(), rank = cluster_rank();
  const long long unit = blockIdx.x / ctas;
  const int h = (int)(unit % p.n_kv), s = (int)(unit / p.n_kv);
  init_rings(B, &J.found, &kmap, &vmap);
  after_prior_kernels();
  const int token = p.query_start_loc[s], rows = p.query_start_loc[s + 1] - token;
  const int L = p.seq_lens[s];
  if (rows == 0) return;
  const bool report = threadIdx.x == 0 && rank == 0 && h == 0;
  if (rows < 0 || (rows > 1 && !p.chunks)) {
    if (report) flag_error(p.err, DEVERR_BOUNDS);
    return;
  }
  if (rows > 1) return;  // a chunk: pa_weights_chunk.cu
  if (token < 0 || token >= p.num_tokens || L < 1 || L > p.max_seq_len ||
      L > ((long long)p.max_blocks << p.block_shift) * 16) {
    if (report) flag_error(p.err, DEVERR_BOUNDS);
    return;
  }
  if (ctas > 1) cluster_arrive();
  const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
  const int half = (1 << p.block_shift) - 1;
  const int all = (L + 15) >> 4;
  const int per = (all + (int)ctas - 1) / (int)ctas;
  const int first = min((int)rank * per, all), pages = min(per, all - first);
  RowsStream<D, F8, kRing<D, F8>> S{
      B,     rings + warp * Ring::BYTES, static_cast<const uint8_t*>(p.k_cache),
      static_cast<const uint8_t*>(p.v_cache), &kmap, &vmap, p.err, p.n_kv, h, warp, lane};
  // The warp's pages of this CTA: base, base + W, ...  Those that the table has no block
  // for weigh nothing.
  int base = warp, page = -1, next = 0;
  unsigned todo = 0;
  const auto issue_next = [&](bool with_v) {
    while (!todo) {
      if (base >= pages) return;
      const int i = base + lane * W;
      next = base;
      base += 32 * W;
      page = -1;
      if (i < pages) {
        const int b = table[(first + i) >> p.block_shift];
        if (b >= 0 && b < p.num_blocks) {
          page = (b << p.block_shift) + ((first + i) & half);
        } else if (with_v) {
          flag_error(p.err, DEVERR_BOUNDS);
          if (i < p.kept_pages)
            for (int e = 0; e < 16 * G; ++e) scores_s[i * 16 * G + e] = -INFINITY;
        }
      }
      todo = __ballot_sync(0xffffffffu, page >= 0);
    }
    const int at = __ffs(todo) - 1;
    todo &= todo - 1;
    // (`live` here is the page's place among the CTA's)
    const int pg = __shfl_sync(0xffffffffu, page, at);
    S.issue(pg, next + at * W, with_v);
  };
#pragma unroll 1
  for (int i = 0; i < Ring::STAGES; ++i) issue_next(true);
  WarpRows<D, G, F8> R;
  R.begin(p.q + ((int64_t)token * p.n_kv + h) * G * D, p.scale_log2);
  uint32_t c = 0;
  for (; c < S.issued; ++c) {
    int mine;
    bool here;
    const uint32_t at = S.wait(c, mine, here);
    float x[4];
    R.scores(at, S.scales(c), x);
    const int n = L - ((first + mine) << 4);
    if (n < 16) {
      R.hide(n, x);
      S.clear_v(c, n);
    }
    if (mine < p.kept_pages && 2 * t < G) {
      float* to = scores_s + (mine * 16 + g) * G + 2 * t;
      to[0] = x[0], to[8 * G] = x[2];
      if (G > 1) to[1] = x[1], to[8 * G + 1] = x[3];
    }
    R.add(x, at + Ring::PAGE, S.scales(c));
    if (!__all_sync(0xffffffffu, here)) break;  // (and the stage has been read)
    issue_next(true);
  }
  S.settle();
  join_rows<Ring::BYTES, D, G, F8>(J, R, rings, ctas, rank,
                                   p.out + ((int64_t)token * p.n_kv + h) * G * D);

  // the weights of this CTA's keys
  float* w = p.weights + ((int64_t)s * p.n_kv + h) * p.weights_stride + (first << 4);
  const int keys = min(pages << 4, L - (first << 4));
  const int fresh = L - 1 - (first << 4);  // the new token
  {
    float m[G], inv[G];
#pragma unroll
    for (int i = 0; i < G; ++i) m[i] = J.top[i], inv[i] = 1.f / J.sum[i];
    const int kept = min(keys, p.kept_pages << 4);
    for (int j = threadIdx.x; j < kept; j += W * 32) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const float x = scores_s[j * G + i];
        sum += x == -INFINITY ? 0.f : fast_exp2(x - m[i]) * inv[i];
      }
      w[j] = (j == fresh ? 0.f : w[j]) + sum;
    }
  }
  if (pages <= p.kept_pages || B.abort_flag) return;  // (the flag: of waits before the join)
  float m[2], inv[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m[i] = 2 * t + i < G ? J.top[2 * t + i] : 0.f;
    inv[i] = 2 * t + i < G ? 1.f / J.sum[2 * t + i] : 0.f;
  }
  // (the rings' places held the warps' results: copies come behind those)
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  base = p.kept_pages + warp;
  todo = 0;
#pragma unroll 1
  for (int i = 0; i < Ring::STAGES; ++i) issue_next(false);
  for (; c < S.issued; ++c) {
    int mine;
    bool here;
    const uint32_t at = S.wait(c, mine, here);
    float x[4];
    R.scores(at, S.scales(c), x);
    // (a head of no query has scores 0 and no part in the sums)
    float sum[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (2 * t + k < G && x[2 * i + k] != -INFINITY)
          sum[i] += fast_exp2(x[2 * i + k] - m[k]) * inv[k];
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    }
    if (t < 2) {
      const int j = mine * 16 + g + 8 * t;
      const float add = t ? sum[1] : sum[0];
      if (j < keys) w[j] = (j == fresh ? 0.f : w[j]) + add;
    }
    if (!__all_sync(0xffffffffu, here)) break;
    issue_next(false);
  }
  S.settle();
}

// Shared memory for scores beside the rings, at most.
constexpr size_t kScoreBytes = 44 * 1024;

template <int D, int G, bool F8>
cudaError_t launch_t(WeighArgs p, int ctas, cudaStream_t stream) {
  CUtensorMap km, vm;
  const int64_t all = (int64_t)p.num_blocks << p.block_shift;
  cudaError_t e = encode_page_map(&km, p.k_cache, F8, all, p.n_kv, D);
  if (e == cudaSuccess) e = encode_page_map(&vm, p.v_cache, F8, all, p.n_kv, D);
  if (e != cudaSuccess) return e;
  const int pages = (p.max_seq_len + 15) / 16;
  const int share = (pages + ctas - 1) / ctas;
  const int most = (int)(kScoreBytes / (16 * G * sizeof(float)));
  p.kept_pages = share < most ? share : most;
  constexpr size_t ring = kRowsWarps * RowsRing<D, F8, kRing<D, F8>>::BYTES;
  const size_t smem = ring + (size_t)p.kept_pages * 16 * G * sizeof(float);
  auto kern = weigh_kernel<D, G, F8>;
  if (ctas > 8) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  // (always the most any call takes, so that calls on other threads agree)
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)(ring + kScoreBytes));
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((long long)p.num_seqs * p.n_kv * ctas));
  return launch_early(kern, grid, dim3(kRowsWarps * 32), smem, stream, ctas, p, km, vm);
}
template <int D, int G>
cudaError_t launch_f(const WeighArgs& p, int ctas, cudaStream_t stream) {
  return p.fp8 ? launch_t<D, G, true>(p, ctas, stream) : launch_t<D, G, false>(p, ctas, stream);
}
template <int D>
cudaError_t launch_d(const WeighArgs& p, int ctas, cudaStream_t stream) {
  switch (p.group) {
    case 1: return launch_f<D, 1>(p, ctas, stream);
    case 2: return launch_f<D, 2>(p, ctas, stream);
    case 4: return launch_f<D, 4>(p, ctas, stream);
    default: return launch_f<D, 8>(p, ctas, stream);
  }
}

}  // namespace

cudaError_t launch_weigh(const WeighArgs& p, int sm_count, cudaStream_t stream) {
  const long long units = (long long)p.num_seqs * p.n_kv;
  const long long pages = ((long long)p.max_seq_len + 15) / 16;
  // CTAs of a cluster: until there are two an SM, and so many that a CTA's scores of up to 192
  // pages stay in shared memory.  One, two, four, eight and 16: 512 pairs of 128 to 4096
  // tokens 118 101* 112 155 212 us, 8-bit 116 84* 82 93 147; of 8192 to 16384 818 681 542 526*
  // 680, 8-bit 739 592 465 374* 400; 2048 pairs of 200 to 2000 185* 218 294 349 699, of 4096
  // to 8191 1268 1042 1003* 1150 1780; 128 pairs of 4096 to 8191 159 91.5 76.5* 82 122; 64
  // pairs of 16384 to 32767, 8-bit, 788 383 202 146 122*.  Many pairs get no more than eight
  // or four for scores that do not stay: max_seq_len may be no more than a bound, and what is
  // computed again is half a page's bytes at most.
  const int most = units >= 8ll * sm_count ? 4 : units >= 2ll * sm_count ? 8 : kRowsMaxCtas;
  int ctas = 1;
  while (ctas < most && pages > 2ll * ctas * kRowsWarps &&
         (units * ctas < 2ll * sm_count || pages > 192ll * ctas))
    ctas *= 2;
  return p.head_dim == 128 ? launch_d<128>(p, ctas, stream) : launch_d<64>(p, ctas, stream);
}

}  // namespace pa
