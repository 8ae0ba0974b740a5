// pa_evict.cu -- eviction: of each request past its budget the tokens of least
// accumulated attention weight go, kv head by kv head, the rest move together in
// order, and the blocks that this empties return to the free list.
//
// Kept are the first num_sinks tokens, the last num_recent ones and, of those
// between, the heaviest (ties: the lowest index).  Kept token i (in order) becomes
// token i of the request: source(i) >= i, and the sources increase.  So a copy in
// place needs no second buffer: the rows of a tile are read before any of them is
// written, and rows read for later tiles lie behind every row written so far.
//
// A cluster takes a (request, kv head): its CTAs choose alike, each from the same
// weights, and move a part of the rows each (K or V, or a range of their bytes).
// The bytes of the weights and of the rows that move, read and written once, are the
// bound.
#include <cstdint>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_select.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;        // 16-byte pieces of a thread in a tile

template <int TILE>
struct EvictShared {
  SelectShared select;
  int stay;  // tokens before the first that goes
  int64_t from[2][TILE], to[2][TILE];  // byte offsets of a tile's rows, or -1
};

// Bit n (from 0) of the set bits of x, which has more than n.
__device__ __forceinline__ int nth_bit(uint32_t x, int n) {
  int at = 0;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const int c = __popc(x & ((1u << w) - 1u));
    if (n >= c) n -= c, x >>= w, at += w;
  }
  return at;
}

// The request's place in the call, or false where there is nothing to do.
struct EvictRequest {
  int len, budget;
};
__device__ __forceinline__ bool evict_request(const EvictArgs& p, int s, EvictRequest& R,
                                              bool report) {
  R.len = p.seq_lens[s];
  R.budget = p.budgets[s];
  if (R.len < 0 || R.len > p.max_seq_len || R.len > (long long)p.max_blocks << p.block_log2 ||
      R.budget < p.num_sinks + p.num_recent) {
    if (report) flag_error(p.err, DEVERR_BOUNDS);
    return false;
  }
  return R.len > R.budget;
}

// New lengths, blocks returned, position offsets: by one CTA.
__device__ void keep_books(const EvictArgs& p, SelectShared& B) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int raw = *p.free_count;
  const bool ok = raw >= 0 && raw <= p.num_blocks;
  if (!ok && tid == 0) flag_error(p.err, DEVERR_BOUNDS);
  long long total = 0;
  __shared__ int first_s[kThreads], freed_s[kThreads];
  __shared__ uint32_t before_s[kThreads];
  for (int s0 = 0; s0 < p.num_seqs; s0 += kThreads) {
    const int s = s0 + tid;
    int first = 0, freed = 0;
    if (s < p.num_seqs) {
      EvictRequest R;
      const bool over = evict_request(p, s, R, true);
      if (over) {
        const int bs = (1 << p.block_log2) - 1;
        first = (R.budget + bs) >> p.block_log2;
        freed = (int)(((long long)R.len + bs) >> p.block_log2) - first;
        if (p.position_offsets) p.position_offsets[s] += R.len - R.budget;
      }
      p.seq_lens_out[s] = over ? R.budget : R.len;
    }
    uint32_t before, unused, all, unused2;
    block_scan2(B, (uint32_t)freed, 0u, before, unused, all, unused2);
    first_s[tid] = first, freed_s[tid] = freed, before_s[tid] = before;
    __syncthreads();
    for (int r = warp; r < kThreads; r += kThreads / 32) {
      const int n = freed_s[r];
      if (n <= 0) continue;
      const int32_t* table = p.block_tables + (int64_t)(s0 + r) * p.max_blocks + first_s[r];
      const long long at = (long long)raw + total + before_s[r];
      for (int i = lane; i < n; i += 32) {
        const int id = table[i];
        if (id < 0 || id >= p.num_blocks || !ok || at + i >= p.num_blocks)
          flag_error(p.err, DEVERR_BOUNDS);
        if (ok && at + i < p.num_blocks) p.free_blocks[at + i] = id;
      }
    }
    total += all;
    __syncthreads();
  }
  if (tid == 0) {
    const long long count = (long long)raw + total;
    *p.free_count_out = !ok ? raw : count > p.num_blocks ? p.num_blocks : (int)count;
  }
}

// PARTS: ranges of a row's bytes, a CTA each for K and for V.
template <int D, bool F8, int PARTS>
__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs p) {
  constexpr int ROW = F8 ? D : 2 * D;
  constexpr int BYTES = ROW / PARTS;
  constexpr int CPR = BYTES / 16;             // pieces of a row
  constexpr int TILE = kThreads * kVecs / CPR;  // rows of a tile
  static_assert(BYTES >= 32, "a part of a row is a sector at least");
  extern __shared__ uint32_t words[];
  __shared__ EvictShared<TILE> B;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr uint32_t CTAS = 2 * PARTS;
  const uint32_t rank = cluster_rank();
  const long long unit = blockIdx.x / CTAS;
  after_prior_kernels();
  if (unit >= (long long)p.num_seqs * p.n_kv) {
    if (rank == 0) keep_books(p, B.select);
    return;
  }
  const int s = (int)(unit / p.n_kv), h = (int)(unit % p.n_kv);
  EvictRequest R;
  if (!evict_request(p, s, R, false)) return;  // (flagged with the books)
  const int L = R.len, budget = R.budget;
  float* w = p.weights + ((int64_t)s * p.n_kv + h) * p.weights_stride;
  const int first = p.num_sinks, last = L - p.num_recent;  // the ones to choose from
  const int K = budget - p.num_sinks - p.num_recent;
  const int nw = (L + 31) >> 5;
  uint32_t* above = words;         // a bit for each token: kept
  uint32_t* equal = above + nw;    // at the threshold; then the count of kept tokens before a word
  uint32_t* keys = equal + nw;     // the weights' keys, where they fit
  const bool staged = p.staged;
  if (staged)
    for (int j = tid; j < L; j += kThreads) keys[j] = ordered_key(w[j]);
  const auto key = [&](int j) { return staged ? keys[j] : ordered_key(w[j]); };
  __syncthreads();
  Threshold th{0xffffffffu, 0u};
  if (K > 0)
    th = select_threshold(B.select, last - first, (uint32_t)K,
                          [&](int i) { return key(first + i); });
  for (int k = warp; k < nw; k += kThreads / 32) {
    const int j = k * 32 + lane;
    const bool middle = j >= first && j < last;
    const uint32_t x = middle ? key(j) : 0u;
    const unsigned a = __ballot_sync(0xffffffffu, j < L && (!middle || x > th.key));
    const unsigned e = __ballot_sync(0xffffffffu, middle && x == th.key);
    if (lane == 0) above[k] = a, equal[k] = e;
  }
  // every CTA of the cluster has read the weights: they may change from here on
  cluster_sync();
  // Words in runs of one thread each: the first th.equal of those at the threshold
  // are kept, and each word gets the number of kept tokens before it.
  {
    const int run = (nw + kThreads - 1) / kThreads | 1;
    const int lo = min(tid * run, nw), hi = min(lo + run, nw);
    uint32_t ne = 0, na = 0, pre_e, pre_a, all_e, all_a;
    for (int k = lo; k < hi; ++k) ne += __popc(equal[k]), na += __popc(above[k]);
    block_scan2(B.select, ne, na, pre_e, pre_a, all_e, all_a);
    uint32_t kept = pre_a + min(pre_e, th.equal);
    uint32_t room = th.equal - min(pre_e, th.equal);
    for (int k = lo; k < hi; ++k) {
      uint32_t e = equal[k];
      uint32_t take = __popc(e);
      if (take > room) {  // the lowest `room` of them
        uint32_t some = 0;
        for (uint32_t i = 0; i < room; ++i) {
          some |= e & (0u - e);
          e &= e - 1;
        }
        e = some;
        take = room;
      }
      room -= take;
      const uint32_t bits = above[k] | e;
      above[k] = bits;
      equal[k] = kept;
      kept += __popc(bits);
    }
    if (tid == 0) B.stay = budget;
    __syncthreads();
    for (int k = lo; k < hi; ++k) {
      // (the last word's bits past the end are clear too)
      if (above[k] != 0xffffffffu) {
        atomicMin(&B.stay, (int)(equal[k] + __ffs(~above[k]) - 1));
        break;
      }
    }
    __syncthreads();
  }
  const int stay = B.stay;
  // The token that becomes token i: the i-th bit.
  const auto source = [&](int i) {
    int lo = 0, hi = nw;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int)equal[mid] <= i)
        lo = mid;
      else
        hi = mid;
    }
    return lo * 32 + nth_bit(above[lo], i - (int)equal[lo]);
  };
  const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
  const int bmask = (1 << p.block_log2) - 1;
  unsigned char* cache = static_cast<unsigned char*>(rank & 1 ? p.v_cache : p.k_cache);
  const int part = rank >> 1;
  bool bad = false;
  // Byte offset of the part of token j's row, or -1.
  const auto row_of = [&](int j) -> int64_t {
    const int b = table[j >> p.block_log2];
    if (b < 0 || b >= p.num_blocks) {
      bad = true;
      return -1;
    }
    if constexpr (F8) {
      const int64_t page = ((int64_t)b << (p.block_log2 - 4)) + ((j & bmask) >> 4);
      return page * fp8_page_bytes(p.n_kv, D) + ((int64_t)(j & 15) * p.n_kv + h) * D + part * BYTES;
    } else {
      return ((((int64_t)b << p.block_log2) + (j & bmask)) * p.n_kv + h) * ROW + part * BYTES;
    }
  };
  // A tile's rows, looked up a tile ahead of its loads.
  const auto look_up = [&](int tile) {
    const int base = stay + tile * TILE;
    for (int i = tid; i < TILE; i += kThreads) {
      int64_t from = -1, to = -1;
      if (base + i < budget) {
        from = row_of(source(base + i));
        to = from < 0 ? -1 : row_of(base + i);
      }
      B.from[tile & 1][i] = from;
      B.to[tile & 1][i] = to;
    }
  };
  const int tiles = (budget - stay + TILE - 1) / TILE;
  uint4 now[kVecs], next[kVecs];
  const auto load = [&](int tile, uint4 (&x)[kVecs]) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int c = v * kThreads + tid;
      const int64_t from = B.from[tile & 1][c / CPR];
      if (from >= 0 && B.to[tile & 1][c / CPR] >= 0)
        x[v] = *reinterpret_cast<const uint4*>(cache + from + (c % CPR) * 16);
    }
  };
  const auto store = [&](int tile, const uint4 (&x)[kVecs]) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int c = v * kThreads + tid;
      const int64_t to = B.to[tile & 1][c / CPR];
      if (to >= 0) *reinterpret_cast<uint4*>(cache + to + (c % CPR) * 16) = x[v];
    }
  };
  if (tiles > 0) look_up(0);
  __syncthreads();
  if (tiles > 0) load(0, now);
  for (int k = 0; k < tiles; ++k) {
    if (k + 1 < tiles) look_up(k + 1);
    __syncthreads();  // the tile's rows have been read; the next one's places are known
    if (k + 1 < tiles) load(k + 1, next);
    store(k, now);
    __syncthreads();  // the tile's places have been read (the tile after next takes them)
#pragma unroll
    for (int v = 0; v < kVecs; ++v) now[v] = next[v];
  }
  // the rows' scales (8-bit cache) and, beside K, the weights: four bytes a token
  const auto move_words = [&](auto place) {
    for (int base = stay; base < budget; base += kThreads * kVecs) {
      uint32_t x[kVecs];
      uint32_t* to[kVecs];
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const int i = base + v * kThreads + tid;
        to[v] = nullptr;
        if (i < budget) {
          const uint32_t* from = place(source(i));
          to[v] = from ? place(i) : nullptr;
          if (to[v]) x[v] = *from;
        }
      }
      __syncthreads();
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        if (to[v]) *to[v] = x[v];
    }
  };
  if constexpr (F8) {
    if (part == 0)
      move_words([&](int j) -> uint32_t* {
        const int b = table[j >> p.block_log2];
        if (b < 0 || b >= p.num_blocks) return nullptr;
        const int64_t page = ((int64_t)b << (p.block_log2 - 4)) + ((j & bmask) >> 4);
        return reinterpret_cast<uint32_t*>(cache + page * fp8_page_bytes(p.n_kv, D) +
                                           fp8_scales_offset(p.n_kv, D)) +
               (j & 15) * p.n_kv + h;
      });
  }
  if (rank == 0) move_words([&](int j) { return reinterpret_cast<uint32_t*>(w + j); });
  if (bad) flag_error(p.err, DEVERR_BOUNDS);
}

__global__ void __launch_bounds__(kThreads) books_kernel(const EvictArgs p) {
  __shared__ SelectShared B;
  after_prior_kernels();
  keep_books(p, B);
}

constexpr size_t kEvictSmemMost = 2 * (size_t)kEvictMaxLen / 8;
static_assert(kEvictSmemMost >= kEvictStaged && kEvictSmemMost <= 160 * 1024, "");

template <int D, bool F8, int PARTS>
cudaError_t launch_t(const EvictArgs& p, size_t smem, bool books, cudaStream_t stream) {
  auto kern = evict_kernel<D, F8, PARTS>;
  if (smem > 8 * 1024) {
    // (always the most any call takes, so that calls on other threads agree)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)kEvictSmemMost);
    if (e != cudaSuccess) return e;
  }
  const long long units = (long long)p.num_seqs * p.n_kv + (books ? 1 : 0);
  return launch_early(kern, dim3((unsigned)(units * 2 * PARTS)), dim3(kThreads), smem, stream,
                      2 * PARTS, p);
}
template <int D, bool F8>
cudaError_t launch_p(const EvictArgs& p, int parts, size_t smem, bool books, cudaStream_t stream) {
  switch (parts) {
    case 1: return launch_t<D, F8, 1>(p, smem, books, stream);
    case 2: return launch_t<D, F8, 2>(p, smem, books, stream);
    default:
      if constexpr (F8 && D == 64)
        return launch_t<D, F8, 2>(p, smem, books, stream);
      else
        return launch_t<D, F8, 4>(p, smem, books, stream);
  }
}

}  // namespace

cudaError_t launch_evict(EvictArgs p, int sm_count, cudaStream_t stream) {
  // lengths that the call changes are written by a kernel of their own, behind the one
  // that reads them
  const bool in_place = p.seq_lens_out == p.seq_lens;
  const size_t bits = 2 * (((size_t)p.max_seq_len + 31) / 32) * 4;
  const size_t with_keys = bits + (size_t)p.max_seq_len * 4;
  p.staged = with_keys <= kEvictStaged;
  const size_t smem = p.staged ? with_keys : bits;
  const long long units = (long long)p.num_seqs * p.n_kv;
  int parts = 1;
  while (parts < 4 && units * 2 * parts < 2ll * sm_count) parts *= 2;
  cudaError_t e;
  if (p.head_dim == 128)
    e = p.fp8 ? launch_p<128, true>(p, parts, smem, !in_place, stream)
              : launch_p<128, false>(p, parts, smem, !in_place, stream);
  else
    e = p.fp8 ? launch_p<64, true>(p, parts, smem, !in_place, stream)
              : launch_p<64, false>(p, parts, smem, !in_place, stream);
  if (e != cudaSuccess || !in_place) return e;
  return launch_early(books_kernel, dim3(1), dim3(kThreads), 0, stream, 1, p);
}

}  // namespace pa
