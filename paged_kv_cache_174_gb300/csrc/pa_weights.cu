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
#include <cstdint>

#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;

template <int D, int G, bool F8>
__global__ void __launch_bounds__(kWarps * 32) weigh_kernel(const WeighArgs p) {
  using Rows = WarpRows<D, G, F8>;
  extern __shared__ __align__(16) float scores_s[];  // [key of the CTA's first pages][G]
  __shared__ RowsShared<D, G, kWarps> B;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
  const uint32_t ctas = cluster_size(), rank = cluster_rank();
  const long long unit = blockIdx.x / ctas;
  const int h = (int)(unit % p.n_kv), s = (int)(unit / p.n_kv);
  after_prior_kernels();
  const int token = p.query_start_loc[s], rows = p.query_start_loc[s + 1] - token;
  if (rows == 0) return;
  const int L = p.seq_lens[s];
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
  const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
  const int half = (1 << p.block_shift) - 1;
  const uint8_t* kc = static_cast<const uint8_t*>(p.k_cache);
  const uint8_t* vc = static_cast<const uint8_t*>(p.v_cache);
  const int64_t page_bytes = Rows::page_bytes(p.n_kv);
  const int all = (L + 15) >> 4;
  const int per = (all + (int)ctas - 1) / (int)ctas;
  const int first = min((int)rank * per, all), pages = min(per, all - first);
  // The pool's page of this CTA's page i, or -1.
  const auto look_up = [&](int i, bool report_it) {
    const int lp = first + i;
    const int b = table[lp >> p.block_shift];
    if (b >= 0 && b < p.num_blocks) return (b << p.block_shift) + (lp & half);
    if (report_it) flag_error(p.err, DEVERR_BOUNDS);
    return -1;
  };
  const auto live_of = [&](int i) { return L - ((first + i) << 4); };

  Rows R;
  R.begin(p.q + ((int64_t)token * p.n_kv + h) * G * D, p.scale_log2);
  for (int base = warp; base < pages; base += 32 * kWarps) {
    const int i = base + lane * kWarps;
    const int page = i < pages ? look_up(i, true) : -1;
    unsigned todo = __ballot_sync(0xffffffffu, page >= 0);
    // (pages that are not there weigh nothing)
    if (page < 0 && i < min(pages, p.kept_pages))
      for (int e = 0; e < 16 * G; ++e) scores_s[i * 16 * G + e] = -INFINITY;
    if (!todo) continue;
    int at = __ffs(todo) - 1;
    int64_t off = __shfl_sync(0xffffffffu, page, at) * page_bytes;
    R.load_k(kc + off, vc + off, p.n_kv, h);
    while (todo) {
      todo &= todo - 1;
      const int mine = base + at * kWarps;
      uint32_t v[4][Rows::VW];
      R.load_v(vc + off, p.n_kv, h, v);
      float x[4], vs[4] = {0.f, 0.f, 0.f, 0.f};
      R.scores(x, vs);
      if (todo) {
        at = __ffs(todo) - 1;
        off = __shfl_sync(0xffffffffu, page, at) * page_bytes;
        R.load_k(kc + off, vc + off, p.n_kv, h);
      }
      const int n = live_of(mine);
      if (n < 16) R.hide(n, x, vs, v);
      if (mine < p.kept_pages && g < G) {
        float* to = scores_s + mine * 16 * G + g;
        to[(2 * t) * G] = x[0], to[(2 * t + 1) * G] = x[1];
        to[(2 * t + 8) * G] = x[2], to[(2 * t + 9) * G] = x[3];
      }
      R.add(x, vs, v);
    }
  }
  join_rows<D, G, F8, kWarps>(B, R, ctas, rank, p.out + ((int64_t)token * p.n_kv + h) * G * D);

  // the weights of this CTA's keys
  float* w = p.weights + ((int64_t)s * p.n_kv + h) * p.weights_stride + (first << 4);
  const int keys = min(pages << 4, L - (first << 4));
  const int fresh = L - 1 - (first << 4);  // the new token
  {
    float m[G], inv[G];
#pragma unroll
    for (int i = 0; i < G; ++i) m[i] = B.cta_m[i], inv[i] = 1.f / B.cta_l[i];
    const int kept = min(keys, p.kept_pages << 4);
    for (int j = threadIdx.x; j < kept; j += kWarps * 32) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const float x = scores_s[j * G + i];
        sum += x == -INFINITY ? 0.f : fast_exp2(x - m[i]) * inv[i];
      }
      w[j] = (j == fresh ? 0.f : w[j]) + sum;
    }
  }
  if (pages <= p.kept_pages) return;
  const float m = g < G ? B.cta_m[g] : 0.f, inv = g < G ? 1.f / B.cta_l[g] : 0.f;
  for (int i = p.kept_pages + warp; i < pages; i += kWarps) {
    const int page = look_up(i, false);
    if (page < 0) continue;
    const int64_t off = page * page_bytes;
    R.load_k(kc + off, vc + off, p.n_kv, h);
    float x[4], vs[4];
    R.scores(x, vs);
    float sum[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      sum[c] = g < G && x[c] != -INFINITY ? fast_exp2(x[c] - m) * inv : 0.f;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], o);
    }
    if (g == 0) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j = i * 16 + 2 * t + (c & 1) + (c >> 1) * 8;
        if (j < keys) w[j] = (j == fresh ? 0.f : w[j]) + sum[c];
      }
    }
  }
}

// Shared memory for scores: what three CTAs of an SM can have beside the rest.
constexpr size_t kScoreBytes = 48 * 1024;

template <int D, int G>
cudaError_t launch_t(WeighArgs p, int ctas, cudaStream_t stream) {
  const int pages = (p.max_seq_len + 15) / 16;
  const int share = (pages + ctas - 1) / ctas;
  const int most = (int)(kScoreBytes / (16 * G * sizeof(float)));
  p.kept_pages = share < most ? share : most;
  const size_t smem = (size_t)p.kept_pages * 16 * G * sizeof(float);
  auto kern = p.fp8 ? weigh_kernel<D, G, true> : weigh_kernel<D, G, false>;
  if (smem > 16 * 1024) {
    // (always the most any call takes, so that calls on other threads agree)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)kScoreBytes);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((unsigned)((long long)p.num_seqs * p.n_kv * ctas));
  return launch_early(kern, grid, dim3(kWarps * 32), smem, stream, ctas, p);
}
template <int D>
cudaError_t launch_d(const WeighArgs& p, int ctas, cudaStream_t stream) {
  switch (p.group) {
    case 1: return launch_t<D, 1>(p, ctas, stream);
    case 2: return launch_t<D, 2>(p, ctas, stream);
    case 4: return launch_t<D, 4>(p, ctas, stream);
    default: return launch_t<D, 8>(p, ctas, stream);
  }
}

}  // namespace

cudaError_t launch_weigh(const WeighArgs& p, int sm_count, cudaStream_t stream) {
  const long long units = (long long)p.num_seqs * p.n_kv;
  const long long pages = ((long long)p.max_seq_len + 15) / 16;
  int ctas = 1;
  while (ctas < 8 && pages > 2ll * ctas * kWarps &&
         (units * ctas < 4ll * sm_count || pages > 64ll * ctas * kWarps))
    ctas *= 2;
  return p.head_dim == 128 ? launch_d<128>(p, ctas, stream) : launch_d<64>(p, ctas, stream);
}

}  // namespace pa
