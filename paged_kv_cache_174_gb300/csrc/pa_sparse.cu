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
// 512 pairs of 128 blocks of 16 (32 q / 8 kv heads of 128): 84 us, 95% of the copy rate;
// 8-bit 59 us, 70%: each warp's chain of conversions and products, 3 warps a scheduler (48% issue).
#include <cstdint>

#include "pa_rows.cuh"
#include "pa_tma_host.h"

namespace pa {
namespace {

// CTAs of an SM, and the bytes of a warp's ring that leaves: three pages in flight a warp.  512
// pairs with rings of 16, 24 and 32 KB (3, 2 and 1 CTAs) 91 84* 98 us; 256 pairs, 8-bit, with
// 8, 12 and 16 KB (5, 4 and 3) 36.4 31.9* 38.8.  Heads of 64, with 8, 12, 16 and 24 KB (5, 4, 3
// and 2 CTAs): 512 pairs 50.1 49.9* 57.2 50.1, 8-bit 40.4 36.8* 51.8 51.9; 256 pairs, 8-bit, 27.0
// 26.1* 29.2 29.2.
template <int D, bool F8>
constexpr int kCtas = D == 128 && !F8 ? 2 : 4;
template <int D, bool F8>
constexpr int kRing = (D == 128 && !F8 ? 24 : 12) * 1024;

template <int D, int G, bool F8>
__global__ void __launch_bounds__(kRowsWarps * 32, kCtas<D, F8>)
    sparse_kernel(const SparseArgs p, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
  using Ring = RowsRing<D, F8, kRing<D, F8>>;
  extern __shared__ __align__(1024) unsigned char rings[];
  __shared__ Ring B;
  __shared__ RowsShared<D, G> J;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ctas = cluster_size(), rank = cluster_rank();
  const long long unit = blockIdx.x / ctas;
  const int h = (int)(unit % p.n_kv), t = (int)(unit / p.n_kv);
  init_rings(B, &J.found, &kmap, &vmap);
  after_prior_kernels();
  const int32_t* list = p.selected + ((int64_t)t * p.n_kv + h) * p.num_selected;
  const int pages = p.num_selected << p.block_shift;
  const int stride = (int)ctas * kRowsWarps;
  // lane i has the warp's i-th page of the list; the first ones are on their way while the
  // request is found
  int base = (int)rank * kRowsWarps + warp + lane * stride;
  int entry = base < pages ? list[base >> p.block_shift] : -1;
  TokenRequest req;
  if (!find_request(p.query_start_loc, p.seq_lens, p.num_seqs, p.num_tokens,
                    ((long long)p.max_blocks << p.block_shift) * 16, t, p.err,
                    threadIdx.x == 0 && rank == 0 && h == 0, &J.found, req))
    return;
  if (ctas > 1) cluster_arrive();
  const int32_t* table = p.block_tables + (int64_t)req.s * p.max_blocks;
  const int half = (1 << p.block_shift) - 1;  // 16-token pages of a block, less one
  RowsStream<D, F8, kRing<D, F8>> S{
      B,     rings + warp * Ring::BYTES, static_cast<const uint8_t*>(p.k_cache),
      static_cast<const uint8_t*>(p.v_cache), &kmap, &vmap, p.err, p.n_kv, h, warp, lane};
  int page = -1, live = 0;
  unsigned todo = 0;  // lanes that hold pages to come
  const auto issue_next = [&] {
    while (!todo) {
      if (base - lane * stride >= pages) return;
      page = -1;
      if (entry > req.pos >> (4 + p.block_shift)) {
        flag_error(p.err, DEVERR_BOUNDS);
      } else if (entry >= 0) {
        const int b = table[entry];
        live = req.pos + 1 - (((entry << p.block_shift) + (base & half)) << 4);
        if (b < 0 || b >= p.num_blocks)
          flag_error(p.err, DEVERR_BOUNDS);
        else if (live > 0)
          page = (b << p.block_shift) + (base & half);
      }
      base += 32 * stride;
      entry = base < pages ? list[base >> p.block_shift] : -1;
      todo = __ballot_sync(0xffffffffu, page >= 0);
    }
    const int at = __ffs(todo) - 1;
    todo &= todo - 1;
    const int pg = __shfl_sync(0xffffffffu, page, at);
    const int lv = __shfl_sync(0xffffffffu, live, at);
    S.issue(pg, lv, true);
  };
#pragma unroll 1
  for (int i = 0; i < Ring::STAGES; ++i) issue_next();
  WarpRows<D, G, F8> R;
  R.begin(p.q + ((int64_t)t * p.n_kv + h) * G * D, p.scale_log2);
  for (uint32_t c = 0; c < S.issued; ++c) {
    int n;
    bool here;
    const uint32_t at = S.wait(c, n, here);
    float x[4];
    R.scores(at, S.scales(c), x);
    if (n < 16) {
      R.hide(n, x);
      S.clear_v(c, n);
    }
    R.add(x, at + Ring::PAGE, S.scales(c));
    if (!__all_sync(0xffffffffu, here)) break;  // (and the stage has been read)
    issue_next();
  }
  S.settle();
  join_rows<Ring::BYTES, D, G, F8>(J, R, rings, ctas, rank,
                                   p.out + ((int64_t)t * p.n_kv + h) * G * D);
}

template <int D, int G, bool F8>
cudaError_t launch_t(const SparseArgs& p, int ctas, cudaStream_t stream) {
  CUtensorMap km, vm;
  const int64_t pages = (int64_t)p.num_blocks << p.block_shift;
  cudaError_t e = encode_page_map(&km, p.k_cache, F8, pages, p.n_kv, D);
  if (e == cudaSuccess) e = encode_page_map(&vm, p.v_cache, F8, pages, p.n_kv, D);
  if (e != cudaSuccess) return e;
  constexpr int smem = kRowsWarps * RowsRing<D, F8, kRing<D, F8>>::BYTES;
  auto kern = sparse_kernel<D, G, F8>;
  if (ctas > 8) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((long long)p.num_tokens * p.n_kv * ctas));
  return launch_early(kern, grid, dim3(kRowsWarps * 32), smem, stream, ctas, p, km, vm);
}
template <int D, int G>
cudaError_t launch_f(const SparseArgs& p, int ctas, cudaStream_t stream) {
  return p.fp8 ? launch_t<D, G, true>(p, ctas, stream) : launch_t<D, G, false>(p, ctas, stream);
}
template <int D>
cudaError_t launch_d(const SparseArgs& p, int ctas, cudaStream_t stream) {
  switch (p.group) {
    case 1: return launch_f<D, 1>(p, ctas, stream);
    case 2: return launch_f<D, 2>(p, ctas, stream);
    case 4: return launch_f<D, 4>(p, ctas, stream);
    default: return launch_f<D, 8>(p, ctas, stream);
  }
}

}  // namespace

cudaError_t launch_sparse(const SparseArgs& p, int sm_count, cudaStream_t stream) {
  const long long units = (long long)p.num_tokens * p.n_kv;
  const long long pages = (long long)p.num_selected << p.block_shift;
  // CTAs of a cluster, until every SM has one and while each warp has two pages.  One, two,
  // four, eight and 16 for lists of 128 pages: 512 pairs 82* 93 101 132 260 us; 256 pairs,
  // 8-bit, 31.8* 32.1 39 54 94; 128 pairs 26.6 27.6* 31 40 71; 64 pairs 21.4 17.8 16.9* 21.6
  // 38; 8 pairs 19.0 13.4 9.3 7.3 7.3*.
  int ctas = 1;
  while (ctas < kRowsMaxCtas && units * ctas < sm_count && pages > 2ll * ctas * kRowsWarps)
    ctas *= 2;
  return p.head_dim == 128 ? launch_d<128>(p, ctas, stream) : launch_d<64>(p, ctas, stream);
}

}  // namespace pa
