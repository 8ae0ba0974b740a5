// pa_weights_chunk.cu -- accumulated attention weights of prompt chunks (requests with
// q_len >= 2) on the tcgen05 tensor cores.
//
//   weights[s, h, j] += sum over the chunk's rows i that see key j, and over the q heads
//                       of kv head h, of exp(x_ij) / sum_k exp(x_ik),  x = scale q k
//
// A weight needs its row's sum over all keys, so there are two passes over S = Q K^T,
// neither of which needs V or P in shared memory:
//  * rows: a tile of 128 / G tokens x G heads stays, key tiles of 128 stream past; each
//    thread keeps the running max and sum of half a row (the halves of the key tile).
//    The keys may be cut into pieces for more units; pieces are (max, sum) pairs.
//  * columns: a tile of 128 keys stays, query tiles stream past; S^T puts a key in
//    each TMEM lane, so the sum over rows is a thread's own.  A cluster's CTAs take
//    query tiles in turn and add their sums up at the end: no atomics, and one order.
// Both share the code below: the tile that stays is A (128 lanes), those that stream
// are B (128 columns), bf16 with 128-byte swizzle, two S buffers in TMEM, and two CTAs
// an SM, so that one's waits, and the drain between units, are the other's work.
// 8-bit cache: K codes are converted to bf16 (exact) and the keys' scales multiply
// the scores.  An exponential for each (row, head, key) in each pass is the bound.
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

constexpr int kTile = 128;          // lanes and columns of a product
constexpr int kEpilogueWarps = 8;   // warps 2-9: two for each TMEM lane quarter
constexpr int kFirstKWarp = 10;
constexpr int kSide = 8;            // slots of the values that go with a B tile's columns
constexpr int kListed = 512;        // chunk requests of a launch

template <bool F8>
struct Roles {
  static constexpr int kKWarps = F8 ? 4 : 2;  // load K tiles: eight pages between them
  static constexpr int kThreads = (kFirstKWarp + kKWarps) * 32;
};

struct alignas(16) ChunkShared {
  uint64_t a_full, b_full[4], b_empty[4], s_full[2], s_empty[2], side_full[kSide];
  uint32_t tmem_slot;
  int abort_flag;
  int listed;
  // rows pass: the keys' scales; columns pass: the rows' log sums (read four at a time)
  alignas(16) float side[kSide][kTile];
  float part[2][2][kTile];    // rows pass: (max, sum); columns pass: [0][half] sums
  int list_seq[kListed];
  int list_base[kListed + 1]; // first tile of each listed request
  SelectShared scan;
};

// Byte offset of 16-byte chunk c of row r in a [rows][64 x bf16] block with the
// 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}

// S = A B^T, both tiles [half of head_dim][128 rows][64].
template <int D>
__device__ __forceinline__ void issue_products(uint32_t d_tmem, tc::Desc a, tc::Desc b) {
  constexpr uint32_t HALF = kTile * 128;
  constexpr uint32_t IDESC = tc::idesc_bf16_f32(kTile, kTile, 0, 0);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
    if (kk == 0)
      tc::mma_bf16_pair<false>(d_tmem, a, off, b, off, IDESC);
    else
      tc::mma_bf16_pair<true>(d_tmem, a, off, b, off, IDESC);
  }
}

struct ChunkUnit {
  int s, h, a, ql, L, c0;  // request, kv head, first token, rows, length, cached before
  int q0, ntok;            // rows pass: first token and tokens of the query tile
  int key0;                // columns pass: first key of the tile
  int first, step, count;  // B tiles of this CTA: first, first + step, ...
  int piece;               // rows pass: piece of the keys
};

template <int D, int G, bool F8, bool COLS>
__global__ void __launch_bounds__(Roles<F8>::kThreads, 2)
    chunk_kernel(const ChunkArgs p, const __grid_constant__ CUtensorMap qmap,
                 const __grid_constant__ CUtensorMap kmap) {
  constexpr int TM = kTile / G;
  constexpr int NH = D / 64;
  constexpr uint32_t HALF = kTile * 128;
  constexpr uint32_t TILE = NH * HALF;
  constexpr int NB = D == 64 ? 4 : 2;      // B stages
  constexpr int KW = Roles<F8>::kKWarps;
  constexpr int PAGES = 8 / KW;            // pages of a K tile for a warp
  constexpr int THREADS = Roles<F8>::kThreads;
  constexpr uint32_t TMEM_COLS = 256;

  extern __shared__ unsigned char smem_raw[];
  unsigned char* a_s = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* b_s = a_s + TILE;
  ChunkShared& B = *reinterpret_cast<ChunkShared*>(b_s + NB * TILE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ctas = cluster_size(), rank = cluster_rank();

  if (tid == 0) {
    mbar_init(smem_addr(&B.a_full), COLS ? KW : 1);
    for (int i = 0; i < NB; ++i) {
      mbar_init(smem_addr(&B.b_full[i]), COLS ? 1 : KW);
      mbar_init(smem_addr(&B.b_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&B.s_full[i]), 1);
      mbar_init(smem_addr(&B.s_empty[i]), kEpilogueWarps);
    }
    for (int i = 0; i < kSide; ++i) mbar_init(smem_addr(&B.side_full[i]), COLS ? 1 : KW);
    B.abort_flag = 0;
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
    int listed = 0, tiles = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += THREADS) {
      const int s = s0 + tid;
      int n = 0;
      if (s < p.num_seqs) {
        const int a = p.query_start_loc[s], b = p.query_start_loc[s + 1], L = p.seq_lens[s];
        if (b - a >= 2 && a >= 0 && b <= p.num_tokens && L >= b - a && L <= p.max_seq_len &&
            L <= ((long long)p.max_blocks << p.block_shift) * 16)
          n = COLS ? (L + kTile - 1) / kTile : (b - a + TM - 1) / TM;
      }
      uint32_t before_n, before_t, all_n, all_t;
      block_scan2(B.scan, n > 0, (uint32_t)n, before_n, before_t, all_n, all_t);
      const int at = listed + (int)before_n - p.skip;
      // (requests before this launch's take no tiles of it)
      if (n > 0 && at >= 0 && at < kListed) B.list_seq[at] = s, B.list_base[at] = n;
      listed += (int)all_n;
      tiles += (int)all_t;
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
    (void)tiles;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = B.tmem_slot;
  volatile int* abort_flag = &B.abort_flag;
  const int pieces = COLS ? 1 : p.pieces;
  const long long units = (long long)tiles_all * p.n_kv * pieces;
  const long long groups = gridDim.x / ctas, group = blockIdx.x / ctas;

  uint32_t c0 = 0;      // B tiles of this CTA before this unit
  uint32_t loaded = 0;  // units before this one that it loaded an A tile for
  for (long long round = 0; round * groups < units; ++round) {
    // long units first; every other round backwards, to even the sums out
    long long u = round * groups + (round & 1 ? groups - 1 - group : group);
    if (u >= units) continue;
    if (!COLS) u = units - 1 - u;
    ChunkUnit U;
    {
      const int per = p.n_kv * pieces;
      const int tile = (int)(u / per), rem = (int)(u % per);
      int lo = 0, hi = B.listed;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (B.list_base[mid] <= tile)
          lo = mid;
        else
          hi = mid;
      }
      U.s = B.list_seq[lo];
      U.h = rem / pieces;
      U.piece = rem % pieces;
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
        U.first = (int)((long long)U.piece * tiles / pieces);
        U.step = 1;
        U.count = (int)((long long)(U.piece + 1) * tiles / pieces) - U.first;
      }
    }
    const int32_t* table = p.block_tables + (int64_t)U.s * p.max_blocks;
    // tokens of query tile i of the request, and how many (columns pass)
    const auto tokens_of = [&](int i) { return min(TM, U.ql - i * TM); };

    if (warp == 0) {
      // ------------------------------------------------ query tiles
      if constexpr (COLS) {
        for (int i = 0; i < U.count; ++i) {
          const uint32_t c = c0 + i, st = c % NB;
          const int qt = U.first + i * U.step, q0 = U.a + qt * TM, ntok = tokens_of(qt);
          // The log sums of the tile's rows.  Their slot's last tile, kSide earlier, is done
          // with: this warp has waited for a stage that a product NB + 1 tiles back freed,
          // which needed the S buffer of the tile two before that to have been read.
          static_assert(kSide >= 4 + 4, "");
          float* side = B.side[c % kSide];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int col = lane * 4 + j, tl = col / G;
            float v = INFINITY;  // (no such row: weight 0)
            if (tl < ntok) {
              const int64_t row = (int64_t)(q0 + tl) * p.n_q + U.h * G + col % G;
              float m = -INFINITY, sum = 0.f;
              for (int k = 0; k < p.pieces; ++k)
                m = fmaxf(m, p.sums[(int64_t)k * p.num_tokens * p.n_q + row].x);
              for (int k = 0; k < p.pieces; ++k) {
                const float2 ml = p.sums[(int64_t)k * p.num_tokens * p.n_q + row];
                if (ml.x != -INFINITY || ml.y != 0.f) sum += ml.y * fast_exp2(ml.x - m);
              }
              v = m + __log2f(sum);
            }
            side[col] = v;
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_addr(&B.side_full[c % kSide]));
            if (c >= NB)
              mbar_wait(smem_addr(&B.b_empty[st]), (c / NB - 1) & 1, p.err, abort_flag);
            const uint32_t bar = smem_addr(&B.b_full[st]);
            mbar_arrive_expect_tx(bar, TILE);
#pragma unroll
            for (int hf = 0; hf < NH; ++hf)
              tc::tma_load_3d(smem_addr(b_s + st * TILE + hf * HALF), &qmap, hf * 64, U.h * G, q0,
                              bar);
          }
          __syncwarp();
        }
      } else if (lane == 0 && U.count > 0) {
        const uint32_t bar = smem_addr(&B.a_full);
        mbar_arrive_expect_tx(bar, TILE);
#pragma unroll
        for (int hf = 0; hf < NH; ++hf)
          tc::tma_load_3d(smem_addr(a_s + hf * HALF), &qmap, hf * 64, U.h * G, U.q0, bar);
      }
    } else if (warp == 1) {
      // ------------------------------------------------ products
      if (lane == 0 && U.count > 0) {
        const tc::Desc ad = tc::sw128_desc_pair(smem_addr(a_s), 16, 1024);
        const tc::Desc bd = tc::sw128_desc_pair(smem_addr(b_s), 16, 1024);
        mbar_wait_spin(smem_addr(&B.a_full), loaded & 1, p.err, abort_flag);
        for (int i = 0; i < U.count; ++i) {
          const uint32_t c = c0 + i, st = c % NB, sb = c & 1;
          mbar_wait_spin(smem_addr(&B.b_full[st]), (c / NB) & 1, p.err, abort_flag);
          if (c >= 2)
            mbar_wait_spin(smem_addr(&B.s_empty[sb]), ((c >> 1) - 1) & 1, p.err, abort_flag);
          tc::fence_after_sync();
          issue_products<D>(tmem + sb * kTile, ad, tc::Desc{bd.lo + st * (TILE >> 4), bd.hi});
          tc::commit(smem_addr(&B.s_full[sb]));
          tc::commit(smem_addr(&B.b_empty[st]));
        }
      }
    } else if (warp >= kFirstKWarp) {
      // ------------------------------------------------ key tiles
      const int idx = warp - kFirstKWarp;
      // Pages idx * PAGES .. of the K tile at key0 into dst, completion on bar.
      const auto load_tile = [&](int key0, unsigned char* dst, uint32_t bar, float* scales) {
        int page[PAGES];
        uint32_t bytes = 0;
#pragma unroll
        for (int i = 0; i < PAGES; ++i) {
          const int lp = key0 / 16 + idx * PAGES + i;
          page[i] = -1;
          if (lp * 16 < U.L) {
            const int b = table[lp >> p.block_shift];
            if (b >= 0 && b < p.num_blocks) {
              page[i] = (b << p.block_shift) + (lp & ((1 << p.block_shift) - 1));
              bytes += NH * 2048;
            } else if (lane == 0) {
              flag_error(p.err, DEVERR_BOUNDS);
            }
          }
        }
        if constexpr (!F8) {
          if (lane != 0) return;
          if (bytes)
            mbar_arrive_expect_tx(bar, bytes);
          else
            mbar_arrive(bar);
#pragma unroll
          for (int i = 0; i < PAGES; ++i) {
            if (page[i] < 0) continue;
#pragma unroll
            for (int hf = 0; hf < NH; ++hf)
              tc::tma_load_3d(smem_addr(dst + hf * HALF + (idx * PAGES + i) * 2048), &kmap,
                              hf * 64, U.h, page[i] * 16, bar);
          }
        } else {
          constexpr int CPR = D / 16, RPL = 32 / CPR, LOADS = 16 / RPL;
          uint4 w[PAGES][LOADS];
          float sc[PAGES];
#pragma unroll
          for (int i = 0; i < PAGES; ++i) {
            sc[i] = 0.f;
            if (page[i] < 0) continue;
            const uint8_t* at = static_cast<const uint8_t*>(p.k_cache) +
                                page[i] * fp8_page_bytes(p.n_kv, D);
            sc[i] = __ldg(reinterpret_cast<const float*>(at + fp8_scales_offset(p.n_kv, D)) +
                          (lane & 15) * p.n_kv + U.h);
#pragma unroll
            for (int j = 0; j < LOADS; ++j)
              w[i][j] = __ldg(reinterpret_cast<const uint4*>(
                  at + ((int64_t)(j * RPL + lane / CPR) * p.n_kv + U.h) * D + (lane % CPR) * 16));
          }
#pragma unroll
          for (int i = 0; i < PAGES; ++i) {
            if (scales && lane < 16) scales[(idx * PAGES + i) * 16 + lane] = sc[i];
            if (page[i] < 0) continue;
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
              const uint32_t src[4] = {w[i][j].x, w[i][j].y, w[i][j].z, w[i][j].w};
              uint32_t out[8];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t x, y;
                f16x2x2_from_e4m3x4(src[k], x, y);
                const float2 f = half2_bits_to_float2(x), g = half2_bits_to_float2(y);
                out[2 * k] = pack_bf16x2(f.x, f.y);
                out[2 * k + 1] = pack_bf16x2(g.x, g.y);
              }
              const int c16 = lane % CPR, c8 = (c16 & 3) * 2;
              unsigned char* to = dst + (c16 >> 2) * HALF + (idx * PAGES + i) * 2048;
              const uint32_t at = swizzled(j * RPL + lane / CPR, c8);
              *reinterpret_cast<uint4*>(to + at) = make_uint4(out[0], out[1], out[2], out[3]);
              *reinterpret_cast<uint4*>(to + (at ^ 16u)) =
                  make_uint4(out[4], out[5], out[6], out[7]);
            }
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar);
        }
      };
      if constexpr (COLS) {
        if (U.count > 0) load_tile(U.key0, a_s, smem_addr(&B.a_full), nullptr);
      } else {
        for (int i = 0; i < U.count; ++i) {
          const uint32_t c = c0 + i, st = c % NB;
          if (lane == 0 && c >= NB)
            mbar_wait(smem_addr(&B.b_empty[st]), (c / NB - 1) & 1, p.err, abort_flag);
          __syncwarp();
          load_tile((U.first + i) * kTile, b_s + st * TILE, smem_addr(&B.b_full[st]),
                    F8 ? B.side[c % kSide] : nullptr);
          if constexpr (F8) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&B.side_full[c % kSide]));
          }
        }
      }
    } else {
      // ------------------------------------------------ sums
      const int quarter = warp & 3, half = (warp - 2) >> 2;
      const int r = quarter * 32 + lane;
      const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
      float top = -INFINITY, sum = 0.f;
      float mul = p.scale_log2;
      int p_row = 0;  // rows pass: the row's position
      if constexpr (COLS) {
        if constexpr (F8) {
          const int j = U.key0 + r;
          float ks = 0.f;
          if (j < U.L) {
            const int b = table[j >> (4 + p.block_shift)];
            if (b >= 0 && b < p.num_blocks) {
              const int64_t page = ((int64_t)b << p.block_shift) +
                                   ((j >> 4) & ((1 << p.block_shift) - 1));
              ks = __ldg(reinterpret_cast<const float*>(
                             static_cast<const uint8_t*>(p.k_cache) +
                             page * fp8_page_bytes(p.n_kv, D) + fp8_scales_offset(p.n_kv, D)) +
                         (j & 15) * p.n_kv + U.h);
            }
          }
          mul *= ks;
        }
      } else {
        p_row = U.c0 + (U.q0 - U.a) + r / G;
      }
      for (int i = 0; i < U.count; ++i) {
        const uint32_t c = c0 + i, sb = c & 1;
        const int tile = U.first + i * U.step;
        const float* side = B.side[c % kSide] + half * 64;
        mbar_wait(smem_addr(&B.s_full[sb]), (c >> 1) & 1, p.err, abort_flag);
        if (COLS || F8)
          mbar_wait(smem_addr(&B.side_full[c % kSide]), (c / kSide) & 1, p.err, abort_flag);
        tc::fence_after_sync();
        // columns lo .. hi - 1 of this half count for this lane
        int lo = 0, hi = 64;
        if constexpr (COLS) {
          const int p0 = U.c0 + tile * TM;  // position of the query tile's first token
          lo = (U.key0 + r - p0) * G - half * 64;
          hi = tokens_of(tile) * G - half * 64;
        } else {
          hi = p_row + 1 - (tile * kTile + half * 64);
        }
        const bool whole = __all_sync(0xffffffffu, lo <= 0 && hi >= 64);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          uint32_t x[32];
          tc::tmem_ld32(tmem + lane_addr + sb * kTile + half * 64 + part * 32, x);
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
                const float2 a = __ffma2_rn(
                    make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), m2,
                    make_float2(-ls.x, -ls.y));
                const float2 b = __ffma2_rn(
                    make_float2(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])), m2,
                    make_float2(-ls.z, -ls.w));
                acc[0].x += fast_exp2(a.x), acc[0].y += fast_exp2(a.y);
                acc[1].x += fast_exp2(b.x), acc[1].y += fast_exp2(b.y);
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
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              float v = __uint_as_float(x[j]) * mul;
              if constexpr (F8) v *= side[part * 32 + j];
              if (!whole) v = part * 32 + j < hi ? v : -INFINITY;
              x[j] = __float_as_uint(v);
              mx = fmaxf(mx, v);
            }
            if (mx > top) {
              sum *= fast_exp2(top - mx);  // (0 from -inf)
              top = mx;
            }
            const float ref = top == -INFINITY ? 0.f : top;
            float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 32; ++j) add[j & 3] += fast_exp2(__uint_as_float(x[j]) - ref);
            sum += (add[0] + add[1]) + (add[2] + add[3]);
          }
        }
      }
      if constexpr (COLS) {
        B.part[0][half][r] = sum;
      } else {
        B.part[0][half][r] = top;
        B.part[1][half][r] = sum;
      }
    }
    c0 += U.count;
    loaded += U.count > 0;
    group_sync(ctas);
    if constexpr (COLS) {
      const int j = U.key0 + tid;
      if (rank == 0 && tid < kTile && j < U.L) {
        float sum = 0.f;
        for (uint32_t k = 0; k < ctas; ++k)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            sum += ctas > 1 ? ld_cluster_f32(cluster_addr(smem_addr(&B.part[0][hf][tid]), k))
                            : B.part[0][hf][tid];
        float* w = p.weights + ((int64_t)U.s * p.n_kv + U.h) * p.weights_stride + j;
        *w = (j < U.c0 ? *w : 0.f) + sum;
      }
    } else if (tid < kTile && tid < U.ntok * G) {
      const float m0 = B.part[0][0][tid], m1 = B.part[0][1][tid], m = fmaxf(m0, m1);
      const float s0 = B.part[1][0][tid], s1 = B.part[1][1][tid];
      const float sum = (m0 == -INFINITY ? s0 : s0 * fast_exp2(m0 - m)) +
                        (m1 == -INFINITY ? s1 : s1 * fast_exp2(m1 - m));
      const int64_t row = (int64_t)(U.q0 + tid / G) * p.n_q + U.h * G + tid % G;
      p.sums[(int64_t)U.piece * p.num_tokens * p.n_q + row] = make_float2(m, sum);
    }
    group_sync(ctas);
  }
  // A unit ends with every product done and so every copy landed, unless a wait was
  // given up: then the last copies into each stage are waited for (again with a limit).
  if (B.abort_flag && tid == 0) {
    for (uint32_t c = c0 > NB ? c0 - NB : 0; c < c0; ++c)
      mbar_wait(smem_addr(&B.b_full[c % NB]), (c / NB) & 1, p.err, abort_flag);
    if (loaded) mbar_wait(smem_addr(&B.a_full), (loaded - 1) & 1, p.err, abort_flag);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int D, int G, bool F8, bool COLS>
cudaError_t launch_pass(const ChunkArgs& p, const CUtensorMap& qm, const CUtensorMap& km, int grid,
                        int ctas, cudaStream_t stream) {
  constexpr size_t tile = (size_t)(D / 64) * kTile * 128;
  constexpr size_t smem = 1024 + tile * (1 + (D == 64 ? 4 : 2)) + sizeof(ChunkShared);
  static_assert(offsetof(ChunkShared, side) % 16 == 0 && tile % 1024 == 0, "alignment");
  static_assert(smem > 80 * 1024 && smem < 113 * 1024, "two CTAs an SM, not three");
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
  km = qm;
  if (!F8) {
    const cuuint64_t dims[3] = {D, nkv, slots};
    const cuuint64_t strides[2] = {D * 2, nkv * D * 2};
    const cuuint32_t box[3] = {64, 1, 16};
    const cudaError_t e = encode_map<3>(&km, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.k_cache, dims,
                                        strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
  }
  const long long slots_of_sms = 2ll * sm_count;
  const ChunkPlan plan = chunk_plan(p.num_tokens, p.n_q, p.n_kv, p.max_seq_len, sm_count);
  // upper bounds of the units: the kernel has the exact count
  const long long q_tiles = (long long)p.num_tokens / (kTile / G) + p.num_seqs;
  const long long row_units = q_tiles * p.n_kv * plan.pieces;
  const long long most_chunks = std::min<long long>(p.num_seqs, p.num_tokens / 2);
  const long long col_units =
      most_chunks * (((long long)p.max_seq_len + kTile - 1) / kTile) * p.n_kv;
  // query tiles that a key tile may see: their cluster's CTAs take them in turn
  const int tiles = (max_q_len + kTile / G - 1) / (kTile / G);
  int ctas = 1;
  while (ctas < 4 && tiles >= 4 * ctas) ctas *= 2;
  p.pieces = plan.pieces;
  for (p.skip = 0; p.skip < most_chunks; p.skip += kListed) {
    cudaError_t e = launch_pass<D, G, F8, false>(
        p, qm, km, (int)std::min(row_units, slots_of_sms), 1, stream);
    if (e != cudaSuccess) return e;
    const long long groups = std::min(col_units, slots_of_sms / ctas);
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

ChunkPlan chunk_plan(int num_tokens, int num_q_heads, int num_kv_heads, int max_seq_len,
                     int sm_count) {
  const int per_tile = kTile / (num_q_heads / num_kv_heads);
  const long long units = ((long long)num_tokens / per_tile + 1) * num_kv_heads;
  const long long key_tiles = ((long long)max_seq_len + kTile - 1) / kTile;
  ChunkPlan plan{1, 0};
  while (plan.pieces < kMaxChunkPieces && units * plan.pieces < 2ll * sm_count &&
         key_tiles >= 8ll * plan.pieces)
    plan.pieces *= 2;
  plan.bytes = (size_t)num_tokens * num_q_heads * plan.pieces * sizeof(float2);
  return plan;
}

cudaError_t launch_chunk_weights(const ChunkArgs& p, int max_q_len, int sm_count,
                                 cudaStream_t stream) {
  return p.head_dim == 128 ? launch_d<128>(p, max_q_len, sm_count, stream)
                           : launch_d<64>(p, max_q_len, sm_count, stream);
}

}  // namespace pa
