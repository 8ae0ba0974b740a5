// pa_sparse.cu -- attention over chosen blocks of the paged cache: each token's query
// heads of a kv head read the blocks that are listed for them and no others.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q k_j),
//
// j over the listed blocks' positions up to the token's own.  Each listed K and V row
// is read once for the group's heads; at 4 d flops a head and key the memory is the
// bound.  A cluster of CTAs takes a (token, kv head); its warps take the list's
// 16-token pages in turn, and the pieces are joined through shared memory of the
// cluster, so there is no workspace and no second kernel.
#include <cstdint>

#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;

template <int D, int G, bool F8>
__global__ void __launch_bounds__(kWarps * 32) sparse_kernel(const SparseArgs p) {
  using Rows = WarpRows<D, G, F8>;
  __shared__ RowsShared<D, G, kWarps> B;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ctas = cluster_size(), rank = cluster_rank();
  const long long unit = blockIdx.x / ctas;
  const int h = (int)(unit % p.n_kv), t = (int)(unit / p.n_kv);
  after_prior_kernels();
  TokenRequest req;
  if (!find_request(p.query_start_loc, p.seq_lens, p.num_seqs, p.num_tokens,
                    ((long long)p.max_blocks << p.block_shift) * 16, t, p.err,
                    threadIdx.x == 0 && rank == 0 && h == 0, req))
    return;
  const int32_t* table = p.block_tables + (int64_t)req.s * p.max_blocks;
  const int32_t* list = p.selected + ((int64_t)t * p.n_kv + h) * p.num_selected;
  const int pages = p.num_selected << p.block_shift;
  const int half = (1 << p.block_shift) - 1;  // 16-token pages of a block, less one
  const uint8_t* kc = static_cast<const uint8_t*>(p.k_cache);
  const uint8_t* vc = static_cast<const uint8_t*>(p.v_cache);
  const int64_t page_bytes = Rows::page_bytes(p.n_kv);

  Rows R;
  R.begin(p.q + ((int64_t)t * p.n_kv + h) * G * D, p.scale_log2);
  const int stride = (int)ctas * kWarps;
  for (int base = (int)rank * kWarps + warp; base < pages; base += 32 * stride) {
    // lane i looks up the warp's i-th page from here
    const int i = base + lane * stride;
    int page = -1, live = 0;
    if (i < pages) {
      const int e = list[i >> p.block_shift];
      if (e > req.pos >> (4 + p.block_shift)) {
        flag_error(p.err, DEVERR_BOUNDS);
      } else if (e >= 0) {
        const int b = table[e];
        live = req.pos + 1 - (((e << p.block_shift) + (i & half)) << 4);
        if (b < 0 || b >= p.num_blocks)
          flag_error(p.err, DEVERR_BOUNDS);
        else if (live > 0)
          page = (b << p.block_shift) + (i & half);
      }
    }
    unsigned todo = __ballot_sync(0xffffffffu, page >= 0);
    if (!todo) continue;
    int at = __ffs(todo) - 1;
    int64_t off = __shfl_sync(0xffffffffu, page, at) * page_bytes;
    R.load_k(kc + off, vc + off, p.n_kv, h);
    while (todo) {
      todo &= todo - 1;
      const int n = __shfl_sync(0xffffffffu, live, at);
      uint32_t v[4][Rows::VW];
      R.load_v(vc + off, p.n_kv, h, v);
      float x[4], vs[4] = {0.f, 0.f, 0.f, 0.f};
      R.scores(x, vs);
      if (todo) {
        at = __ffs(todo) - 1;
        off = __shfl_sync(0xffffffffu, page, at) * page_bytes;
        R.load_k(kc + off, vc + off, p.n_kv, h);
      }
      if (n < 16) R.hide(n, x, vs, v);
      R.add(x, vs, v);
    }
  }
  join_rows<D, G, F8, kWarps>(B, R, ctas, rank, p.out + ((int64_t)t * p.n_kv + h) * G * D);
}

template <int D, int G>
cudaError_t launch_t(const SparseArgs& p, int ctas, cudaStream_t stream) {
  const dim3 grid((unsigned)((long long)p.num_tokens * p.n_kv * ctas));
  return p.fp8 ? launch_early(sparse_kernel<D, G, true>, grid, dim3(kWarps * 32), 0, stream, ctas, p)
               : launch_early(sparse_kernel<D, G, false>, grid, dim3(kWarps * 32), 0, stream, ctas,
                              p);
}
template <int D>
cudaError_t launch_d(const SparseArgs& p, int ctas, cudaStream_t stream) {
  switch (p.group) {
    case 1: return launch_t<D, 1>(p, ctas, stream);
    case 2: return launch_t<D, 2>(p, ctas, stream);
    case 4: return launch_t<D, 4>(p, ctas, stream);
    default: return launch_t<D, 8>(p, ctas, stream);
  }
}

}  // namespace

cudaError_t launch_sparse(const SparseArgs& p, int sm_count, cudaStream_t stream) {
  const long long units = (long long)p.num_tokens * p.n_kv;
  const long long pages = (long long)p.num_selected << p.block_shift;
  int ctas = 1;
  while (ctas < 8 && units * ctas < 4ll * sm_count && pages > 2ll * ctas * kWarps) ctas *= 2;
  return p.head_dim == 128 ? launch_d<128>(p, ctas, stream) : launch_d<64>(p, ctas, stream);
}

}  // namespace pa
