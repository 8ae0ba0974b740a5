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
// bound: 64 requests of 1900 to 2304 tokens down to 2048, 8 heads of 128, 125 us, 79% of the
// copy rate; 8 requests of 16K to 32K tokens, 8-bit, down to 4096, 55 us, half of it the
// choice, which every CTA of a cluster waits for.
#include <cstdint>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_select.cuh"

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kWindow = 2048;            // rows whose places are looked up together
constexpr int kTileBytes = 16 * 1024;    // rows read together
// Tiles of the ring, all but one in flight while that is stored: few where an SM has two
// CTAs, many where it has one.
constexpr int kFewTiles = 4, kManyTiles = 8;

struct EvictShared {
  SelectShared select;
  int stay;  // tokens before the first that goes
  // a window's rows: the token that moves, its slot and the one it goes to (or -1)
  int token[kWindow], from[kWindow], to[kWindow];
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
  const int tid = threadIdx.x;
  const int raw = *p.free_count;
  const bool ok = raw >= 0 && raw <= p.num_blocks;
  if (!ok && tid == 0) flag_error(p.err, DEVERR_BOUNDS);
  long long total = 0;
  __shared__ int first_s[kThreads];
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
    first_s[tid] = first, before_s[tid] = before;
    __syncthreads();
    // item k of these requests' blocks: the owner is the last that begins at or before it
    // (one with blocks, as later ones begin past it)
    const auto owner = [&](uint32_t k) {
      int lo = 0, hi = kThreads;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before_s[mid] <= k)
          lo = mid;
        else
          hi = mid;
      }
      return lo;
    };
    for (uint32_t k0 = 0; k0 < all; k0 += 4 * kThreads) {
      int id[4];  // (several loads in flight)
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t k = k0 + i * kThreads + tid;
        id[i] = -1;
        if (k < all) {
          const int r = owner(k);
          id[i] = p.block_tables[(int64_t)(s0 + r) * p.max_blocks + first_s[r] + (k - before_s[r])];
          bad |= id[i] < 0 || id[i] >= p.num_blocks;
        }
      }
      // (an entry that names no block is not pushed, and the others move together)
      const bool some_bad = __syncthreads_or(bad);
      if (bad) flag_error(p.err, DEVERR_BOUNDS);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t k = k0 + i * kThreads;
        if (k >= all) continue;
        const bool push = id[i] >= 0 && id[i] < p.num_blocks;
        uint32_t nth = tid, unused3, pushed = min(all - k, (uint32_t)kThreads), unused4;
        if (some_bad) block_scan2(B, push, 0u, nth, unused3, pushed, unused4);
        const long long at = (long long)raw + total + nth;
        if (push && (!ok || at >= p.num_blocks)) flag_error(p.err, DEVERR_BOUNDS);
        if (push && ok && at < p.num_blocks) p.free_blocks[at] = id[i];
        total += pushed;
      }
    }
    __syncthreads();
  }
  if (tid == 0) {
    const long long count = (long long)raw + total;
    *p.free_count_out = !ok ? raw : count > p.num_blocks ? p.num_blocks : (int)count;
  }
}

__device__ __forceinline__ void copy_async16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void commit_copies() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// All of this thread's groups of copies but the last N are complete.
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// PARTS: ranges of a row's bytes, a CTA each for K and for V.
template <int D, bool F8, int PARTS, int kTiles>
__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const EvictArgs p) {
  constexpr int ROW = F8 ? D : 2 * D;
  constexpr int BYTES = ROW / PARTS;
  constexpr int CPR = BYTES / 16;               // pieces of a row
  constexpr int TILE = kTileBytes / BYTES;      // rows of a tile
  constexpr int PIECES = kTileBytes / 16 / kThreads;  // of a thread in a tile
  static_assert(BYTES >= 32, "a part of a row is a sector at least");
  static_assert(kWindow % TILE == 0 && PIECES >= 1, "");
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ EvictShared B;
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
  uint32_t* above = reinterpret_cast<uint32_t*>(smem);  // a bit for each token: kept
  uint32_t* equal = above + nw;  // at the threshold; then the kept tokens before a word
  // then the weights where they fit, and later the ring in their place
  unsigned char* ring = smem + ((8 * (size_t)nw + 15) & ~size_t(15));
  uint32_t* held = equal + nw;
  const bool staged = p.staged;
  if (staged) {  // (four bytes a copy: a row of weights begins at any multiple of them)
    for (int j = tid; j < L; j += kThreads)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(held + j)), "l"(w + j)
                   : "memory");
    commit_copies();
    wait_copies<0>();
  }
  // keys in the weights' place, each by the thread that brought it
  KeyBits seen;
#pragma unroll 4
  for (int j = tid; j < L; j += kThreads) {
    const uint32_t k = ordered_key(staged ? __uint_as_float(held[j]) : w[j]);
    if (staged) held[j] = k;
    if (j >= first && j < last) seen.see(k);
  }
  const auto key = [&](int j) { return staged ? held[j] : ordered_key(w[j]); };
  __syncthreads();
  Threshold th{0xffffffffu, 0u};
  static_assert(kWindow >= kSelectBins, "the histogram lies where rows' places will");
  if (K > 0)
    th = select_threshold(B.select, reinterpret_cast<uint32_t*>(B.token), last - first, (uint32_t)K,
                          [&](int i) { return key(first + i); }, seen);
  for (int k0 = warp; k0 < nw; k0 += 4 * (kThreads / 32)) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = (k0 + i * (kThreads / 32)) * 32 + lane;
      x[i] = j >= first && j < last ? key(j) : 0u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + i * (kThreads / 32), j = k * 32 + lane;
      const bool middle = j >= first && j < last;
      const unsigned a = __ballot_sync(0xffffffffu, j < L && (!middle || x[i] > th.key));
      const unsigned e = __ballot_sync(0xffffffffu, middle && x[i] == th.key);
      if (lane == 0 && k < nw) above[k] = a, equal[k] = e;
    }
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
  const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
  const int bmask = (1 << p.block_log2) - 1;
  unsigned char* cache = static_cast<unsigned char*>(rank & 1 ? p.v_cache : p.k_cache);
  const int part = rank >> 1;
  const int64_t page_bytes = fp8_page_bytes(p.n_kv, D);
  // This CTA's part of the row of a slot.
  const auto row_at = [&](int slot) {
    if constexpr (F8)
      return cache + (slot >> 4) * page_bytes + ((slot & 15) * p.n_kv + h) * D + part * BYTES;
    else
      return cache + ((int64_t)slot * p.n_kv + h) * ROW + part * BYTES;
  };
  bool bad = false;
  for (int base = stay; base < budget; base += kWindow) {
    const int rows = min(kWindow, budget - base);
    __syncthreads();  // (the last window's places, and the keys, have been read)
    constexpr int MINE = kWindow / kThreads;  // rows of a thread, looked up side by side
    {
      // the token that becomes token i: the i-th bit, in the last word with no more before it
      int lo[MINE], hi[MINE];
#pragma unroll
      for (int v = 0; v < MINE; ++v) lo[v] = 0, hi[v] = nw;
      for (int n = nw; n > 1; n = (n + 1) >> 1) {
#pragma unroll
        for (int v = 0; v < MINE; ++v) {
          const int mid = (lo[v] + hi[v]) >> 1;
          const bool right = (int)equal[mid] <= base + v * kThreads + tid;
          // (done where they are neighbours: mid is lo, and its count is not above)
          if (right)
            lo[v] = mid;
          else
            hi[v] = mid;
        }
      }
      int token[MINE], from[MINE], to[MINE];
#pragma unroll
      for (int v = 0; v < MINE; ++v) {
        const int i = v * kThreads + tid;
        token[v] = 0, from[v] = to[v] = -1;
        if (i < rows) {
          token[v] = lo[v] * 32 + nth_bit(above[lo[v]], base + i - (int)equal[lo[v]]);
          from[v] = table[token[v] >> p.block_log2];
          to[v] = table[(base + i) >> p.block_log2];
        }
      }
#pragma unroll
      for (int v = 0; v < MINE; ++v) {
        const int i = v * kThreads + tid;
        const bool good = (unsigned)from[v] < (unsigned)p.num_blocks &&
                          (unsigned)to[v] < (unsigned)p.num_blocks;
        bad |= i < rows && !good;
        B.token[i] = token[v];
        B.from[i] = good ? (from[v] << p.block_log2) + (token[v] & bmask) : -1;
        B.to[i] = good ? (to[v] << p.block_log2) + ((base + i) & bmask) : -1;
      }
    }
    __syncthreads();
    // The rows' scales (8-bit cache) and, beside K, the weights, four bytes a token: a window's
    // are read before any is written (the barriers of the tiles lie between).
    uint32_t x[MINE], y[MINE];
    const auto scale_at = [&](int slot) {
      return reinterpret_cast<uint32_t*>(cache + (slot >> 4) * page_bytes +
                                         fp8_scales_offset(p.n_kv, D)) +
             (slot & 15) * p.n_kv + h;
    };
    const bool scales = F8 && part == 0, weights = rank == 0;
#pragma unroll
    for (int v = 0; v < MINE; ++v) {
      const int i = v * kThreads + tid;
      if (i >= rows) continue;
      if (scales && B.to[i] >= 0) x[v] = *scale_at(B.from[i]);
      if (weights && B.to[i] >= 0) y[v] = __float_as_uint(w[B.token[i]]);
    }
    const int tiles = (rows + TILE - 1) / TILE;
    // A tile's rows are read before any of them is written, and rows read for later tiles lie
    // behind every row written so far, so tiles may be read ahead.
    const auto fetch = [&](int k) {
      if (k < tiles) {
        const uint32_t to = smem_addr(ring + (k % kTiles) * kTileBytes);
#pragma unroll
        for (int v = 0; v < PIECES; ++v) {
          const int c = v * kThreads + tid, r = k * TILE + c / CPR;
          if (B.to[r] >= 0) copy_async16(to + c * 16, row_at(B.from[r]) + (c % CPR) * 16);
        }
      }
      commit_copies();
    };
#pragma unroll
    for (int k = 0; k < kTiles - 1; ++k) fetch(k);
    for (int k = 0; k < tiles; ++k) {
      wait_copies<kTiles - 2>();
      __syncthreads();  // the tile is here; the one before it has been stored
      fetch(k + kTiles - 1);
      const unsigned char* at = ring + (k % kTiles) * kTileBytes;
#pragma unroll
      for (int v = 0; v < PIECES; ++v) {
        const int c = v * kThreads + tid, r = k * TILE + c / CPR;
        const int to = B.to[r];
        if (to >= 0)
          *reinterpret_cast<uint4*>(row_at(to) + (c % CPR) * 16) =
              *reinterpret_cast<const uint4*>(at + c * 16);
      }
    }
    wait_copies<0>();
#pragma unroll
    for (int v = 0; v < MINE; ++v) {
      const int i = v * kThreads + tid;
      if (i >= rows) continue;
      if (scales && B.to[i] >= 0) *scale_at(B.to[i]) = x[v];
      if (weights && B.to[i] >= 0) w[base + i] = __uint_as_float(y[v]);
    }
  }
  if (bad) flag_error(p.err, DEVERR_BOUNDS);
}

__global__ void __launch_bounds__(kThreads) books_kernel(const EvictArgs p) {
  __shared__ SelectShared B;
  after_prior_kernels();
  keep_books(p, B);
}

// Shared memory of a CTA beside its static part: the bits and prefix counts of the longest
// request with the ring, or with its weights.
constexpr size_t kEvictSmemMost = 2 * (size_t)kEvictMaxLen / 8 + 16 + kFewTiles * kTileBytes;
static_assert(kEvictSmemMost + sizeof(EvictShared) <= 227 * 1024, "");

template <int D, bool F8, int PARTS, int TILES>
cudaError_t launch_t(const EvictArgs& p, size_t smem, bool books, cudaStream_t stream) {
  auto kern = evict_kernel<D, F8, PARTS, TILES>;
  // (always the most any call takes, so that calls on other threads agree)
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kEvictSmemMost);
  if (e != cudaSuccess) return e;
  const long long units = (long long)p.num_seqs * p.n_kv + (books ? 1 : 0);
  return launch_early(kern, dim3((unsigned)(units * 2 * PARTS)), dim3(kThreads), smem, stream,
                      2 * PARTS, p);
}
template <int D, bool F8, int TILES>
cudaError_t launch_p(const EvictArgs& p, int parts, size_t smem, bool books, cudaStream_t stream) {
  switch (parts) {
    case 1: return launch_t<D, F8, 1, TILES>(p, smem, books, stream);
    case 2: return launch_t<D, F8, 2, TILES>(p, smem, books, stream);
    default:
      if constexpr (F8 && D == 64)
        return launch_t<D, F8, 2, TILES>(p, smem, books, stream);
      else
        return launch_t<D, F8, 4, TILES>(p, smem, books, stream);
  }
}
template <int D, bool F8>
cudaError_t launch_r(const EvictArgs& p, int parts, bool many, size_t smem, bool books,
                     cudaStream_t stream) {
  return many ? launch_p<D, F8, kManyTiles>(p, parts, smem, books, stream)
              : launch_p<D, F8, kFewTiles>(p, parts, smem, books, stream);
}

}  // namespace

cudaError_t launch_evict(EvictArgs p, int sm_count, cudaStream_t stream) {
  // lengths that the call changes are written by a kernel of their own, behind the one
  // that reads them
  const bool in_place = p.seq_lens_out == p.seq_lens;
  const size_t bits = (2 * (((size_t)p.max_seq_len + 31) / 32) * 4 + 15) & ~size_t(15);
  const size_t with_keys = bits + (size_t)p.max_seq_len * 4;
  p.staged = with_keys <= kEvictSmemMost;
  const long long units = (long long)p.num_seqs * p.n_kv;
  // A row's bytes in one, two or four ranges, as CTAs are few (each chooses for itself): 512
  // pairs of about 2048 tokens 125* 140 205 us, 64 pairs of 16K to 32K tokens, 8-bit, 57*
  // 82 176, 8 pairs of 32K 42 36 30*.
  int parts = 1;
  while (parts < 4 && units * 4 * parts < sm_count) parts *= 2;
  const size_t few = bits + kFewTiles * kTileBytes, more = bits + kManyTiles * kTileBytes;
  const bool many = units * 2 * parts <= sm_count && more <= kEvictSmemMost;
  const size_t ring = many ? more : few;
  const size_t smem = p.staged && with_keys > ring ? with_keys : ring;
  cudaError_t e = cudaSuccess;
  if (units > 0 || !in_place) {  // (else only the books)
    if (p.head_dim == 128)
      e = p.fp8 ? launch_r<128, true>(p, parts, many, smem, !in_place, stream)
                : launch_r<128, false>(p, parts, many, smem, !in_place, stream);
    else
      e = p.fp8 ? launch_r<64, true>(p, parts, many, smem, !in_place, stream)
                : launch_r<64, false>(p, parts, many, smem, !in_place, stream);
  }
  if (e != cudaSuccess || !in_place) return e;
  return launch_early(books_kernel, dim3(1), dim3(kThreads), 0, stream, 1, p);
}

}  // namespace pa
