// pa_weights_chunk.cu -- accumulated attention weights of prompt chunks (requests with
// q_len >= 2) on the tcgen05 tensor cores.
//
//   weights[s, h, j] += sum over the chunk's rows i that see key j, and over the q heads
//                       of kv head h, of exp(x_ij) / sum_k exp(x_ik),  x = scale q k
//
// A weight needs its row's sum over all keys, so there are two passes over S = Q K^T,
// neither of which needs V or P in shared memory:
//  * rows: a tile of 128 / G tokens x G heads stays, key tiles of 128 stream past; each
//    thread keeps the running max and sum of a row.
//  * columns: a tile of 128 keys stays, query tiles of 128 rows stream past; S^T puts a key
//    in each TMEM lane, so the sum over rows is a thread's own.
// In both the CTAs of a cluster share a unit's tiles where units are few, and add up at its
// end: no atomics, and one order.
// The passes share the code below.  The tile that stays is A, copied to TMEM once a unit, so
// that a product reads only B from shared memory; S has three buffers, for two groups of
// eight warps that take the sums.  The warps that bring tiles and issue products run ahead
// of a unit's end.  8-bit cache: K codes are converted to bf16 (exact) and the keys' scales
// multiply the scores.
// The waits of the warps that sum, for TMEM and for one another, bound it, and in 8-bit
// caches the conversion, which shares the exponentials' pipe: 4096 rows and keys, 32 q / 8 kv
// heads of 128, take 92 us for the rows and 80 for the columns (the products alone 34 each),
// 8-bit 166 and 84.  Measured in the same terms: A in shared memory and two CTAs an SM 82 and
// 134 (8-bit 214 and 157); a tile of 256 by products of 64 columns, which took about three
// times as long a score, 114 and 117; accumulators read as 16 x 256 bits, for fewer reads of
// a column's value, 87 and 158; codes converted by shifts and one product 198 in place of 167.
#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_select.cuh"
#include "pa_tcgen05.cuh"
#include "pa_tma_host.h"

namespace pa {
namespace {

constexpr int kTile = 128;          // rows of A and of B: a product's lanes and columns
constexpr int kSumWarps = 16;       // warps 2-17: for each S buffer two a TMEM lane quarter
constexpr int kFirstKWarp = 18;
constexpr int kBuffers = 3;         // of S in TMEM
// Barriers of their products: each is of one group of sum warps, which so meets every phase
// (of a buffer's barrier it would meet every other one, and take one parity for another).
constexpr int kFulls = 2 * kBuffers;
constexpr int kSide = 12;           // slots of the values that go with a B tile's columns
constexpr int kListed = 512;        // chunk requests of a launch

// Warps that bring K tiles, eight pages between them.  Of an 8-bit cache each has the codes and
// scales of its next kRaw tiles' pages on their way to shared memory, and converts them.
template <bool F8>
struct Roles {
  static constexpr int kKWarps = F8 ? 8 : 2;
  static constexpr int kPages = 8 / kKWarps;
  static constexpr int kStages = F8 ? 3 : 4;  // B tiles on their way or in use
  static constexpr int kThreads = (kFirstKWarp + kKWarps) * 32;
};
constexpr int kRaw = 3;
template <int D>
struct Raw {  // a warp's codes and scales of a tile
  static constexpr int kBytes = Roles<true>::kPages * 16 * D + 128;
  static_assert(kBytes % 128 == 0, "tensor copies start on 128 bytes");
};

struct alignas(16) ChunkShared {
  uint64_t a_full, a_ready, b_full[4], b_empty[4], s_full[kFulls], s_empty[kBuffers];
  uint64_t side_full[kSide], raw_full[8][kRaw];
  uint32_t tmem_slot;
  int abort_flag;
  int late;  // a wait for the last copies was given up too
  int listed;
  // rows pass: the keys' scales times the scores'; columns pass: the rows' log sums
  alignas(16) float side[kSide][kTile];
  // by units in turn: rows pass (max, sum) by sum warps' share; columns pass [0] sums
  float part[2][2][4][kTile];
  int list_seq[kListed];
  int list_base[kListed + 1]; // first tile of each listed request
  SelectShared scan;
};

// Byte offset of 16-byte chunk c of row r in a [rows][64 x bf16] block with the
// 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}

// The codes of a page of one kv head.
__device__ __forceinline__ void load_codes(uint32_t dst, const CUtensorMap* map, int head,
                                           int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(head), "r"(0), "r"(page), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void cp_async4(float* to, const float* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(to)), "l"(from)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// S = A B^T: 128 rows of A in TMEM, two values a column, and tile B [half of head_dim][128][64].
template <int D>
__device__ __forceinline__ void issue_products(uint32_t d_tmem, uint32_t a_tmem, tc::Desc b) {
  constexpr uint32_t HALF = kTile * 128;
  constexpr uint32_t IDESC = tc::idesc_bf16_f32(kTile, kTile, 0, 0);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off_b = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
    if (kk == 0)
      tc::mma_bf16_tmem_a_pair<false>(d_tmem, a_tmem, b, off_b, IDESC);
    else
      tc::mma_bf16_tmem_a_pair<true>(d_tmem, a_tmem + kk * 8, b, off_b, IDESC);
  }
}

struct ChunkUnit {
  int s, h, a, ql, L, c0;  // request, kv head, first token, rows, length, cached before
  int q0, ntok;            // rows pass: first token and tokens of the query tile
  int key0;                // columns pass: first key of the tile
  int first, step, count;  // B tiles of this CTA: first, first + step, ...
};

template <int D, int G, bool F8, bool COLS>
__global__ void __launch_bounds__(Roles<F8>::kThreads, 1)
    chunk_kernel(const ChunkArgs p, const __grid_constant__ CUtensorMap qmap,
                 const __grid_constant__ CUtensorMap kmap) {
  constexpr int TM = kTile / G;  // tokens of a query tile
  constexpr int NH = D / 64;
  constexpr uint32_t HALF = kTile * 128, TILE = NH * HALF;
  constexpr int NB = Roles<F8>::kStages;
  constexpr int KW = Roles<F8>::kKWarps;
  constexpr int PAGES = Roles<F8>::kPages;  // of a K tile for a warp
  constexpr int RAW = Raw<D>::kBytes;
  constexpr int THREADS = Roles<F8>::kThreads;
  constexpr uint32_t A_COLS = kBuffers * kTile;
  constexpr uint32_t TMEM_COLS = 512;       // S, then A

  extern __shared__ unsigned char smem_raw[];
  unsigned char* a_s = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* b_s = a_s + TILE;
  unsigned char* raw_s = b_s + NB * TILE;  // (8-bit cache) [K warp][kRaw][RAW]
  ChunkShared& B = *reinterpret_cast<ChunkShared*>(raw_s + (F8 ? KW * kRaw * RAW : 0));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ctas = cluster_size(), rank = cluster_rank();

  if (tid == 0) {
    mbar_init(smem_addr(&B.a_full), COLS ? KW : 1);
    mbar_init(smem_addr(&B.a_ready), kSumWarps);
    for (int i = 0; i < NB; ++i) {
      mbar_init(smem_addr(&B.b_full[i]), COLS ? 1 : KW);
      mbar_init(smem_addr(&B.b_empty[i]), 1);
    }
    for (int i = 0; i < kFulls; ++i) mbar_init(smem_addr(&B.s_full[i]), 1);
    for (int i = 0; i < kBuffers; ++i) mbar_init(smem_addr(&B.s_empty[i]), kSumWarps / 2);
    for (int i = 0; i < kSide; ++i) mbar_init(smem_addr(&B.side_full[i]), COLS ? 1 : KW);
    for (int i = 0; i < 8 * kRaw; ++i) mbar_init(smem_addr(&B.raw_full[i / kRaw][i % kRaw]), 1);
    B.abort_flag = B.late = 0;
    fence_mbar_init();
  }
  after_prior_kernels();
  // (only now: a CTA that held columns while it waited for a kernel whose CTA on this
  // SM waits for columns would never end)
  if (warp == 1) {
    tc::tmem_alloc(smem_addr(&B.tmem_slot), TMEM_COLS);
    tc::tmem_relinquish();
  }
  // the launch's chunk requests and their tiles, in order
  int tiles_all = 0;
  {
    int listed = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += THREADS) {
      const int s = s0 + tid;
      int n = 0;
      if (s < p.num_seqs) {
        const int a = p.query_start_loc[s], b = p.query_start_loc[s + 1], L = p.seq_lens[s];
        if (b - a >= 2 && a >= 0 && b <= p.num_tokens && L >= b - a && L <= p.max_seq_len &&
            L <= ((long long)p.max_blocks << p.block_shift) * 16)
          n = COLS ? (L + kTile - 1) / kTile : (b - a + TM - 1) / TM;
      }
      uint32_t before_n, unused, all_n, unused2;
      block_scan2(B.scan, n > 0, 0u, before_n, unused, all_n, unused2);
      const int at = listed + (int)before_n - p.skip;
      // (requests before this launch's take no tiles of it)
      if (n > 0 && at >= 0 && at < kListed) B.list_seq[at] = s, B.list_base[at] = n;
      listed += (int)all_n;
    }
    const int mine = min(max(listed - p.skip, 0), kListed);
    __syncthreads();
    // counts to first tiles
    uint32_t run = 0;
    for (int i0 = 0; i0 < mine; i0 += THREADS) {
      const int i = i0 + tid;
      const uint32_t n = i < mine ? (uint32_t)B.list_base[i] : 0u;
      uint32_t before, unused, all, unused2;
      block_scan2(B.scan, n, 0u, before, unused, all, unused2);
      if (i < mine) B.list_base[i] = (int)(run + before);
      run += all;
    }
    tiles_all = (int)run;
    if (tid == 0) B.list_base[mine] = tiles_all, B.listed = mine;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = B.tmem_slot;
  volatile int* abort_flag = &B.abort_flag;
  const long long units = (long long)tiles_all * p.n_kv;
  const long long groups = gridDim.x / ctas, group = blockIdx.x / ctas;

  uint32_t c0 = 0;      // B tiles of this CTA before this unit
  uint32_t loaded = 0;  // units before this one that it loaded an A tile for
  uint32_t raw0 = 0;    // (8-bit cache) K tiles before this unit
  bool arrived = false; // at the end of a unit not waited for
  for (long long round = 0; round * groups < units; ++round) {
    // long units first; every other round backwards, to even the sums out
    long long u = round * groups + (round & 1 ? groups - 1 - group : group);
    if (u >= units) continue;
    if (!COLS) u = units - 1 - u;
    ChunkUnit U;
    {
      const int tile = (int)(u / p.n_kv);
      int lo = 0, hi = B.listed;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (B.list_base[mid] <= tile)
          lo = mid;
        else
          hi = mid;
      }
      U.s = B.list_seq[lo];
      U.h = (int)(u % p.n_kv);
      U.a = p.query_start_loc[U.s];
      U.ql = p.query_start_loc[U.s + 1] - U.a;
      U.L = p.seq_lens[U.s];
      U.c0 = U.L - U.ql;
      const int nth = tile - B.list_base[lo];
      if constexpr (COLS) {
        U.key0 = nth * kTile;
        U.q0 = U.ntok = 0;
        const int from = max(0, U.key0 - U.c0) / TM, tiles = (U.ql + TM - 1) / TM;
        U.first = from + (int)rank;
        U.step = (int)ctas;
        U.count = U.first < tiles ? (tiles - U.first + U.step - 1) / U.step : 0;
      } else {
        U.key0 = 0;
        U.q0 = U.a + nth * TM;
        U.ntok = min(TM, U.ql - nth * TM);
        const int tiles = (U.c0 + nth * TM + U.ntok + kTile - 1) / kTile;
        U.first = (int)((long long)rank * tiles / ctas);
        U.step = 1;
        U.count = (int)((long long)(rank + 1) * tiles / ctas) - U.first;
      }
    }
    if (*abort_flag) U.count = 0;  // (a wait was given up: nothing more is begun)
    const int32_t* table = p.block_tables + (int64_t)U.s * p.max_blocks;
    // tokens of query tile i of the request, and how many (columns pass)
    const auto tokens_of = [&](int i) { return min(TM, U.ql - i * TM); };

    if (warp == 0) {
      // ------------------------------------------------ query tiles
      if constexpr (COLS) {
        // the log sums of a query tile's rows, two columns a lane, a tile ahead
        const auto log_sums = [&](int i) {
          float4 v = make_float4(INFINITY, INFINITY, INFINITY, INFINITY);  // (no row: weight 0)
          if (i < U.count) {
            const int qt = U.first + i * U.step, n = tokens_of(qt) * G;
            const float* at = p.sums + ((int64_t)U.h * p.num_tokens + U.a + qt * TM) * G + lane * 4;
            if (lane * 4 < n) v.x = at[0];
            if (lane * 4 + 1 < n) v.y = at[1];
            if (lane * 4 + 2 < n) v.z = at[2];
            if (lane * 4 + 3 < n) v.w = at[3];
          }
          return v;
        };
        float4 ls = log_sums(0);
        for (int i = 0; i < U.count; ++i) {
          const uint32_t c = c0 + i, st = c % NB;
          const int q0 = U.a + (U.first + i * U.step) * TM;
          // Their slot's last tile, kSide earlier, is done with: this warp has waited for a
          // stage that the product NB + 1 tiles back freed, which needed that S buffer's
          // tile before to have been read, by warps that were done with all earlier ones.
          static_assert(kSide >= NB + 6 && kSide % 2 == 0, "");
          *reinterpret_cast<float4*>(B.side[c % kSide] + lane * 4) = ls;
          ls = log_sums(i + 1);
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_addr(&B.side_full[c % kSide]));
            if (c >= NB)
              mbar_wait(smem_addr(&B.b_empty[st]), (c / NB - 1) & 1, p.err, abort_flag);
            const uint32_t bar = smem_addr(&B.b_full[st]);
            mbar_arrive_expect_tx(bar, TILE);
#pragma unroll
            for (int hf = 0; hf < NH; ++hf)
              tc::tma_load_3d(smem_addr(b_s + st * TILE + hf * HALF), &qmap, hf * 64, U.h * G,
                              q0, bar);
          }
          __syncwarp();
        }
      } else if (lane == 0 && U.count > 0) {
        const uint32_t bar = smem_addr(&B.a_full);
        // (the unit before has copied its tile away)
        if (loaded == 0 ||
            mbar_wait(smem_addr(&B.a_ready), (loaded - 1) & 1, p.err, abort_flag)) {
          mbar_arrive_expect_tx(bar, TILE);
#pragma unroll
          for (int hf = 0; hf < NH; ++hf)
            tc::tma_load_3d(smem_addr(a_s + hf * HALF), &qmap, hf * 64, U.h * G, U.q0, bar);
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------ products
      if (lane == 0 && U.count > 0) {
        const tc::Desc bd = tc::sw128_desc_pair(smem_addr(b_s), 16, 1024);
        const bool ok = mbar_wait_spin(smem_addr(&B.a_ready), loaded & 1, p.err, abort_flag);
        for (int i = 0; ok && i < U.count; ++i) {
          const uint32_t c = c0 + i, st = c % NB, sb = c % kBuffers;
          if (!mbar_wait_spin(smem_addr(&B.b_full[st]), (c / NB) & 1, p.err, abort_flag)) break;
          if (c >= kBuffers && !mbar_wait_spin(smem_addr(&B.s_empty[sb]), (c / kBuffers - 1) & 1,
                                               p.err, abort_flag))
            break;
          tc::fence_after_sync();
          issue_products<D>(tmem + sb * kTile, tmem + A_COLS,
                            tc::Desc{bd.lo + st * (TILE >> 4), bd.hi});
          tc::commit(smem_addr(&B.s_full[c % kFulls]));
          tc::commit(smem_addr(&B.b_empty[st]));
        }
      }
    } else if (warp >= kFirstKWarp) {
      // ------------------------------------------------ key tiles
      const int idx = warp - kFirstKWarp;
      const int first = COLS ? U.key0 / kTile : U.first;
      const int tiles = U.count == 0 ? 0 : COLS ? 1 : U.count;
      // Page k of this warp's of K tile first + i: its place in the pool (-1: none).
      const auto look_up = [&](int i, int k) {
        const int lp = (first + i) * (kTile / 16) + idx * PAGES + k;
        if (i >= tiles || k >= PAGES || lp * 16 >= U.L) return -1;
        const int b = table[lp >> p.block_shift];
        if (b >= 0 && b < p.num_blocks)
          return (b << p.block_shift) + (lp & ((1 << p.block_shift) - 1));
        flag_error(p.err, DEVERR_BOUNDS);
        return -1;
      };
      // Where K tile i goes, and its barrier: A, or a stage of B, waited for.
      const auto tile_bar = [&](int i) {
        return smem_addr(COLS ? &B.a_full : &B.b_full[(c0 + i) % NB]);
      };
      const auto tile_at = [&](int i) {
        const uint32_t c = c0 + i, st = c % NB;
        if (lane == 0 && COLS && loaded > 0)
          mbar_wait(smem_addr(&B.a_ready), (loaded - 1) & 1, p.err, abort_flag);
        if (lane == 0 && !COLS && c >= NB)
          mbar_wait(smem_addr(&B.b_empty[st]), (c / NB - 1) & 1, p.err, abort_flag);
        __syncwarp();
        return COLS ? a_s : b_s + st * TILE;
      };
      if constexpr (!F8) {
        // a lane for each half of a page, with its place looked up a tile ahead
        int page = look_up(0, lane / NH);
        for (int i = 0; i < tiles; ++i) {
          const int here = page;
          page = look_up(i + 1, lane / NH);
          unsigned char* dst = tile_at(i);
          const uint32_t bar = tile_bar(i);
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, here >= 0)) * 2048;
          if (lane == 0) {
            if (bytes)
              mbar_arrive_expect_tx(bar, bytes);
            else
              mbar_arrive(bar);
          }
          __syncwarp();
          if (here >= 0)
            tc::tma_load_3d(smem_addr(dst + (lane % NH) * HALF + (idx * PAGES + lane / NH) * 2048),
                            &kmap, (lane % NH) * 64, U.h, here * 16, bar);
          __syncwarp();
        }
      } else {
        unsigned char* raw = raw_s + idx * kRaw * RAW;
        // lane 0 brings a page's codes, lane l < 16 the scale of token l
        static_assert(PAGES == 1, "");
        const auto start = [&](int i, int page) {
          const uint32_t slot = (raw0 + i) % kRaw;
          unsigned char* to = raw + slot * RAW;
          const uint32_t bar = smem_addr(&B.raw_full[idx][slot]);
          const int mine = __shfl_sync(0xffffffffu, page, 0);
          if (i < tiles) {
            const uint32_t n = __popc(__ballot_sync(0xffffffffu, page >= 0));
            if (lane == 0) {
              if (n)
                mbar_arrive_expect_tx(bar, n * 16 * D);
              else
                mbar_arrive(bar);
            }
            __syncwarp();
            if (page >= 0)
              load_codes(smem_addr(to + lane * 16 * D), &kmap, U.h, page, bar);
            if (!COLS && lane < 16) {
              float* sc = reinterpret_cast<float*>(to + PAGES * 16 * D) + lane;
              if (mine >= 0)
                cp_async4(sc, reinterpret_cast<const float*>(
                                  static_cast<const uint8_t*>(p.k_cache) +
                                  mine * fp8_page_bytes(p.n_kv, D) + fp8_scales_offset(p.n_kv, D)) +
                                  (lane & 15) * p.n_kv + U.h);
              else
                *sc = 0.f;
            }
          }
          cp_async_commit();
        };
        for (int i = 0; i < kRaw; ++i) start(i, look_up(i, lane));
        int page = look_up(kRaw, lane);
        constexpr int CPR = D / 16, RPL = 32 / CPR;
        const int c16 = lane % CPR, c8 = (c16 & 3) * 2;
        for (int i = 0; i < tiles; ++i) {
          const uint32_t slot = (raw0 + i) % kRaw;
          const unsigned char* from = raw + slot * RAW;
          cp_async_wait<kRaw - 1>();
          __syncwarp();
          mbar_wait(smem_addr(&B.raw_full[idx][slot]), ((raw0 + i) / kRaw) & 1, p.err, abort_flag);
          unsigned char* dst = tile_at(i);
          if (!COLS && lane < 16)
            B.side[(c0 + i) % kSide][idx * PAGES * 16 + lane] =
                reinterpret_cast<const float*>(from + PAGES * 16 * D)[lane] * p.scale_log2;
#pragma unroll
          for (int k = 0; k < PAGES; ++k) {
            unsigned char* to = dst + (c16 >> 2) * HALF + (idx * PAGES + k) * 2048;
#pragma unroll
            for (int j = 0; j < 16 / RPL; ++j) {
              const uint4 w =
                  *reinterpret_cast<const uint4*>(from + k * 16 * D + j * 512 + lane * 16);
              const uint32_t src[4] = {w.x, w.y, w.z, w.w};
              uint32_t out[8];
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                uint32_t x, y;
                f16x2x2_from_e4m3x4(src[n], x, y);
                const float2 f = half2_bits_to_float2(x), g = half2_bits_to_float2(y);
                out[2 * n] = pack_bf16x2(f.x, f.y);
                out[2 * n + 1] = pack_bf16x2(g.x, g.y);
              }
              const uint32_t at = swizzled(j * RPL + lane / CPR, c8);
              *reinterpret_cast<uint4*>(to + at) = make_uint4(out[0], out[1], out[2], out[3]);
              *reinterpret_cast<uint4*>(to + (at ^ 16u)) =
                  make_uint4(out[4], out[5], out[6], out[7]);
            }
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(tile_bar(i));
            if (!COLS) mbar_arrive(smem_addr(&B.side_full[(c0 + i) % kSide]));
          }
          // (every lane has read the slot: its next tile may come)
          start(i + kRaw, page);
          page = look_up(i + kRaw + 1, lane);
        }
        cp_async_wait<0>();
      }
    } else {
      // ------------------------------------------------ sums
      const int quarter = warp & 3, share = (warp - 2) >> 2;
      const int cols = (share & 1) * (kTile / 2), group = share >> 1;
      const int r = quarter * 32 + lane;
      const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
      if (U.count > 0) {
        // A to TMEM: 32 values of a row, 16 columns, each
        mbar_wait(smem_addr(&B.a_full), loaded & 1, p.err, abort_flag);
        if (share < D / 32) {
          uint32_t x[16];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(
                a_s + (share >> 1) * HALF + swizzled(r, (share & 1) * 4 + c));
            x[4 * c] = v.x, x[4 * c + 1] = v.y, x[4 * c + 2] = v.z, x[4 * c + 3] = v.w;
          }
          tc::tmem_st16(tmem + lane_addr + A_COLS + share * 16, x);
          tc::tmem_wait_st();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&B.a_ready));
      }
      float top = -INFINITY, sum = 0.f, mul = p.scale_log2;
      int p_row = 0;  // rows pass: the row's position
      if constexpr (!COLS) {
        p_row = U.c0 + (U.q0 - U.a) + r / G;
      } else if constexpr (F8) {
        const int j = U.key0 + r;
        float ks = 0.f;
        if (j < U.L) {
          const int b = table[j >> (4 + p.block_shift)];
          if (b >= 0 && b < p.num_blocks) {
            const int64_t page =
                ((int64_t)b << p.block_shift) + ((j >> 4) & ((1 << p.block_shift) - 1));
            ks = __ldg(reinterpret_cast<const float*>(static_cast<const uint8_t*>(p.k_cache) +
                                                      page * fp8_page_bytes(p.n_kv, D) +
                                                      fp8_scales_offset(p.n_kv, D)) +
                       (j & 15) * p.n_kv + U.h);
          }
        }
        mul *= ks;
      }
      for (int i = (c0 & 1) ^ group; i < U.count; i += 2) {
        const uint32_t c = c0 + i, sb = c % kBuffers;
        const int tile = U.first + i * U.step;
        const float* side = B.side[c % kSide] + cols;
        mbar_wait(smem_addr(&B.s_full[c % kFulls]), (c / kFulls) & 1, p.err, abort_flag);
        if (COLS || F8)
          mbar_wait(smem_addr(&B.side_full[c % kSide]), (c / kSide) & 1, p.err, abort_flag);
        tc::fence_after_sync();
        // of this warp's columns lo .. hi - 1 count for a row
        int lo = 0, hi;
        if constexpr (COLS) {
          const int p0 = U.c0 + tile * TM;  // position of the query tile's first token
          lo = (U.key0 + r - p0) * G - cols;
          hi = tokens_of(tile) * G - cols;
        } else {
          hi = p_row + 1 - tile * kTile - cols;
        }
        const bool whole = __all_sync(0xffffffffu, lo <= 0 && hi >= 64);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          uint32_t x[32];
          tc::tmem_ld32(tmem + lane_addr + sb * kTile + cols + part * 32, x);
          tc::tmem_wait_ld();
          if (part == 1) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&B.s_empty[sb]));
          }
          if constexpr (COLS) {
            if (whole) {
              float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
              const float2 m2 = make_float2(mul, mul);
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 ls = *reinterpret_cast<const float4*>(side + part * 32 + j);
                const float2 u = __ffma2_rn(
                    make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), m2,
                    make_float2(-ls.x, -ls.y));
                const float2 v = __ffma2_rn(
                    make_float2(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])), m2,
                    make_float2(-ls.z, -ls.w));
                acc[0] = __fadd2_rn(acc[0], make_float2(fast_exp2(u.x), fast_exp2(u.y)));
                acc[1] = __fadd2_rn(acc[1], make_float2(fast_exp2(v.x), fast_exp2(v.y)));
              }
              sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const int col = part * 32 + j;
                const float e = fast_exp2(fmaf(__uint_as_float(x[j]), mul, -side[col]));
                sum += col >= lo && col < hi ? e : 0.f;
              }
            }
          } else {
            // With a positive factor the largest raw score gives the largest scaled one and the
            // factor goes into the exponent's FMA; else (and with the keys' scales) the scores
            // are scaled first.
            const bool raw = !F8 && mul > 0.f;
            if (!raw) {
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                float4 f = make_float4(mul, mul, mul, mul);
                if constexpr (F8) f = *reinterpret_cast<const float4*>(side + part * 32 + j);
                const float2 u = __fmul2_rn(
                    make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])),
                    make_float2(f.x, f.y));
                const float2 v = __fmul2_rn(
                    make_float2(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])),
                    make_float2(f.z, f.w));
                x[j] = __float_as_uint(u.x), x[j + 1] = __float_as_uint(u.y);
                x[j + 2] = __float_as_uint(v.x), x[j + 3] = __float_as_uint(v.y);
              }
            }
            if (!whole) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (part * 32 + j >= hi) x[j] = __float_as_uint(-INFINITY);
            }
            float m4[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              m4[0] = fmax3(m4[0], __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
              m4[1] = fmax3(m4[1], __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
            }
            const float f = raw ? mul : 1.f;
            const float mx = fmaxf(m4[0], m4[1]) * f;
            if (mx > top) {
              sum *= fast_exp2(top - mx);  // (0 from -inf)
              top = mx;
            }
            const float ref = top == -INFINITY ? 0.f : top;
            const float2 f2 = make_float2(f, f), r2 = make_float2(-ref, -ref);
            float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float2 u = __ffma2_rn(
                  make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), f2, r2);
              const float2 v = __ffma2_rn(
                  make_float2(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])), f2, r2);
              add[0] = __fadd2_rn(add[0], make_float2(fast_exp2(u.x), fast_exp2(u.y)));
              add[1] = __fadd2_rn(add[1], make_float2(fast_exp2(v.x), fast_exp2(v.y)));
            }
            add[0] = __fadd2_rn(add[0], add[1]);
            sum += add[0].x + add[0].y;
          }
        }
      }
      float(&part)[2][4][kTile] = B.part[round & 1];
      part[0][share][r] = COLS ? sum : top;
      if (!COLS) part[1][share][r] = sum;
      // The unit's sums are in place, and its products done: A may be written again.
      tc::fence_before_sync();
      if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
      } else {
        asm volatile("bar.sync 1, %0;" ::"n"(kSumWarps * 32) : "memory");
      }
      tc::fence_after_sync();
      // number what of row t, from share k & 3 of CTA k / 4's columns
      const int t = tid - 64;
      const auto part_of = [&](int what, uint32_t k) {
        const float* at = &part[what][k & 3][t];
        return ctas > 1 ? ld_cluster_f32(cluster_addr(smem_addr(at), k >> 2)) : *at;
      };
      if constexpr (COLS) {
        const int j = U.key0 + t;
        if (rank == 0 && t < kTile && j < U.L) {
          float all = 0.f;
          for (uint32_t k = 0; k < 4 * ctas; ++k) all += part_of(0, k);
          float* w = p.weights + ((int64_t)U.s * p.n_kv + U.h) * p.weights_stride + j;
          *w = (j < U.c0 ? *w : 0.f) + all;
        }
      } else if (rank == 0 && t < U.ntok * G) {
        // the row's log sum over the shares, and the cluster's pieces of its keys
        float m = -INFINITY, all = 0.f;
        for (uint32_t k = 0; k < 4 * ctas; ++k) {
          const float pm = part_of(0, k), ps = part_of(1, k);
          const float to = fmaxf(m, pm);
          all = (m == -INFINITY ? all : all * fast_exp2(m - to)) +
                (pm == -INFINITY ? ps : ps * fast_exp2(pm - to));
          m = to;
        }
        p.sums[((int64_t)U.h * p.num_tokens + U.q0) * G + t] = m + __log2f(all);
      }
    }
    // (the warps that bring tiles and issue products do not wait for a unit's end: of a
    // cluster they arrive, and wait for the end of the unit before)
    if (ctas > 1 && (warp < 2 || warp >= kFirstKWarp)) {
      __syncwarp();
      if (arrived) cluster_wait();
      cluster_arrive();
      arrived = true;
    }
    c0 += U.count;
    loaded += U.count > 0;
    if (U.count > 0) raw0 += COLS ? 1 : U.count;
  }
  if (arrived) cluster_wait();
  if (ctas > 1) cluster_sync();  // (the first CTA has read the others' last sums)
  tc::fence_before_sync();
  __syncthreads();
  // Every product is done and so every copy landed, unless a wait was given up: then the
  // last copies into each stage are waited for (again with a limit).
  if (*abort_flag && tid == 0) {
    for (uint32_t c = c0 > NB ? c0 - NB : 0; c < c0; ++c)
      mbar_wait_landed(smem_addr(&B.b_full[c % NB]), (c / NB) & 1, p.err, &B.late);
    if (loaded) mbar_wait_landed(smem_addr(&B.a_full), (loaded - 1) & 1, p.err, &B.late);
    for (int w = 0; F8 && w < KW; ++w)
      for (uint32_t c = raw0 > kRaw ? raw0 - kRaw : 0; c < raw0; ++c)
        mbar_wait_landed(smem_addr(&B.raw_full[w][c % kRaw]), (c / kRaw) & 1, p.err, &B.late);
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int D, int G, bool F8, bool COLS>
cudaError_t launch_pass(const ChunkArgs& p, const CUtensorMap& qm, const CUtensorMap& km, int grid,
                        int ctas, cudaStream_t stream) {
  using R = Roles<F8>;
  constexpr size_t used = 1024 + (size_t)(D / 64) * 128 * (kTile + kTile * R::kStages) +
                          (F8 ? R::kKWarps * kRaw * Raw<D>::kBytes : 0) + sizeof(ChunkShared);
  constexpr size_t smem = std::max<size_t>(used, 120 * 1024);
  static_assert(offsetof(ChunkShared, side) % 16 == 0, "alignment");
  // (one CTA an SM, which has all of TMEM)
  static_assert(smem < 227 * 1024, "");
  auto kern = chunk_kernel<D, G, F8, COLS>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_early(kern, dim3(grid), dim3(Roles<F8>::kThreads), smem, stream, ctas, p, qm, km);
}

template <int D, int G, bool F8>
cudaError_t launch_t(ChunkArgs p, int max_q_len, int sm_count, cudaStream_t stream) {
  const cuuint64_t nkv = (cuuint64_t)p.n_kv;
  const cuuint64_t slots = ((cuuint64_t)p.num_blocks << p.block_shift) * 16;
  CUtensorMap qm, km;
  {
    const cuuint64_t dims[3] = {D, (cuuint64_t)p.n_q, (cuuint64_t)p.num_tokens};
    const cuuint64_t strides[2] = {D * 2, (cuuint64_t)p.n_q * D * 2};
    const cuuint32_t box[3] = {64, G, kTile / G};
    const cudaError_t e = encode_map<3>(&qm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.q, dims, strides,
                                        box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
  }
  if (!F8) {
    const cuuint64_t dims[3] = {D, nkv, slots};
    const cuuint64_t strides[2] = {D * 2, nkv * D * 2};
    const cuuint32_t box[3] = {64, 1, 16};
    const cudaError_t e = encode_map<3>(&km, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.k_cache, dims,
                                        strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
  } else {
    const cuuint64_t dims[4] = {D, nkv, 16, slots / 16};
    const cuuint64_t strides[3] = {D, D * nkv, (cuuint64_t)fp8_page_bytes(p.n_kv, D)};
    const cuuint32_t box[4] = {D, 1, 16, 1};
    const cudaError_t e =
        encode_map<4>(&km, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.k_cache, dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_NONE,
                      D == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                               : CU_TENSOR_MAP_L2_PROMOTION_L2_64B);
    if (e != cudaSuccess) return e;
  }
  // upper bounds of the units: the kernel has the exact count
  const long long row_units = ((long long)p.num_tokens / (kTile / G) + p.num_seqs) * p.n_kv;
  const long long most_chunks = std::min<long long>(p.num_seqs, p.num_tokens / 2);
  const long long key_tiles = ((long long)p.max_seq_len + kTile - 1) / kTile;
  const long long col_units = most_chunks * key_tiles * p.n_kv;
  // CTAs of a cluster, while they leave SMs idle without: pieces of a row's keys, and of a key
  // tile's query tiles.  A chunk of 64 after 4096 tokens, 8 kv heads (24 units of rows): 47.8
  // us with 1 piece, 41.2 with 2, 39.2 with 4, 47.8 with 8.  Where the units fill the SMs a
  // cluster costs: 4096 rows in 2 pieces 347 us, in one 322; with clusters of 4 for the columns
  // 408, of 2 322, alone 320.
  const long long least = ((long long)p.num_tokens / (kTile / G) + 1) * p.n_kv;
  int pieces = 1;
  while (pieces < 4 && least * pieces * 2 <= sm_count && key_tiles >= 4ll * pieces) pieces *= 2;
  const int tiles = (max_q_len + kTile / G - 1) / (kTile / G);
  int ctas = 1;
  while (ctas < 4 && key_tiles * p.n_kv * ctas * 2 <= sm_count && tiles >= 8 * ctas) ctas *= 2;
  for (p.skip = 0; p.skip < most_chunks; p.skip += kListed) {
    long long groups = std::min<long long>(row_units, sm_count / pieces);
    cudaError_t e =
        launch_pass<D, G, F8, false>(p, qm, km, (int)(groups * pieces), pieces, stream);
    if (e != cudaSuccess) return e;
    groups = std::min<long long>(col_units, sm_count / ctas);
    e = launch_pass<D, G, F8, true>(p, qm, km, (int)(groups * ctas), ctas, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int D, int G>
cudaError_t launch_f(const ChunkArgs& p, int max_q_len, int sm_count, cudaStream_t stream) {
  return p.fp8 ? launch_t<D, G, true>(p, max_q_len, sm_count, stream)
               : launch_t<D, G, false>(p, max_q_len, sm_count, stream);
}
template <int D>
cudaError_t launch_d(const ChunkArgs& p, int max_q_len, int sm_count, cudaStream_t stream) {
  switch (p.group) {
    case 1: return launch_f<D, 1>(p, max_q_len, sm_count, stream);
    case 2: return launch_f<D, 2>(p, max_q_len, sm_count, stream);
    case 4: return launch_f<D, 4>(p, max_q_len, sm_count, stream);
    default: return launch_f<D, 8>(p, max_q_len, sm_count, stream);
  }
}

}  // namespace

cudaError_t launch_chunk_weights(const ChunkArgs& p, int max_q_len, int sm_count,
                                 cudaStream_t stream) {
  return p.head_dim == 128 ? launch_d<128>(p, max_q_len, sm_count, stream)
                           : launch_d<64>(p, max_q_len, sm_count, stream);
}

}  // namespace pa
