// pa_step.cu -- a step's integer inputs built on the GPU from the requests'
// lengths: block-table entries of newly needed blocks (popped from a free
// list), sequence lengths, query start locations, the slot of every new token
// and its positions.  The host-side step driver does the same with lists; with
// these arrays made on the device, a captured loop of steps needs no host work
// between replays.
//
// Request s holds c_s cached tokens and gets n_s new ones, so it needs
//   need_s = ceil((c_s + n_s) / bs) - ceil(c_s / bs)
// blocks.  With B_s and T_s the exclusive prefix sums of need and n, request s
// is served when B_s + need_s <= free count and T_s + n_s <= num_tokens (both
// sums only grow, so the served requests are a prefix of the list), its k-th
// new block is free[count - 1 - (B_s + k)] (last in, first out, as the host
// allocator hands blocks out), and its i-th new token is row T_s + i.
//
// Kilobytes move, so a launch's latency is all there is: one CTA scans the
// lengths into shared memory, then its threads walk the flat lists of new
// blocks and of token rows, each finding its request by a binary search of the
// prefix sums.
#include <cstdint>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// The last index s in [0, n) with pre[s] <= x (pre[0] = 0 <= x, non-decreasing).
__device__ __forceinline__ int owner_of(const int* pre, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) build_step_kernel(const StepPlanArgs p) {
  extern __shared__ int smem_i[];
  int* ctx_s = smem_i;                     // [num_seqs]
  int* tok_s = ctx_s + p.num_seqs;         // [num_seqs + 1] exclusive prefix of new tokens
  int* blk_s = tok_s + p.num_seqs + 1;     // [num_seqs + 1] exclusive prefix of new blocks
  __shared__ long long warp_t[kPlanWarps], warp_b[kPlanWarps];
  __shared__ int served_t, served_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bs = p.block_size;

  const int raw_count = *p.free_count;
  const bool count_ok = raw_count >= 0 && raw_count <= p.num_blocks;
  const int count = count_ok ? raw_count : 0;
  bool bad = !count_ok;
  if (tid == 0) served_t = 0, served_b = 0;

  long long run_t = 0, run_b = 0;  // totals of the chunks before this one
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    long long nt = 0, nb = 0;
    bool ok = false;
    if (s < p.num_seqs) {
      const int c = p.context_lens[s], n = p.new_lens[s];
      ctx_s[s] = c;
      ok = c >= 0 && n >= 0 && (long long)c + n <= (long long)p.max_blocks * bs;
      if (ok) {
        nt = n;
        nb = ((long long)c + n + bs - 1) / bs - ((long long)c + bs - 1) / bs;
      } else {
        bad = true;  // a length out of range: no rows, no blocks
      }
    }
    long long it = nt, ib = nb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, it, o);
      const long long b = __shfl_up_sync(0xffffffffu, ib, o);
      if (lane >= o) it += a, ib += b;
    }
    __syncthreads();  // the last chunk's warp totals have been read
    if (lane == 31) warp_t[warp] = it, warp_b[warp] = ib;
    __syncthreads();
    long long bt = run_t, bb = run_b;
    for (int w = 0; w < kPlanWarps; ++w) {
      if (w < warp) bt += warp_t[w], bb += warp_b[w];
      run_t += warp_t[w], run_b += warp_b[w];
    }
    it += bt, ib += bb;
    if (s < p.num_seqs) {
      const bool served = it <= p.num_tokens && ib <= count;
      // inclusive sums at s + 1; past the served prefix a mark, replaced below
      tok_s[s + 1] = served ? (int)it : -1;
      blk_s[s + 1] = served ? (int)ib : -1;
      if (served) {
        atomicMax(&served_t, (int)it);
        atomicMax(&served_b, (int)ib);
      } else {
        bad = true;
      }
    }
  }
  if (tid == 0) tok_s[0] = 0, blk_s[0] = 0;
  __syncthreads();
  const int total_t = served_t, total_b = served_b;
  for (int s = tid; s < p.num_seqs; s += kPlanThreads) {
    if (tok_s[s + 1] < 0) tok_s[s + 1] = total_t, blk_s[s + 1] = total_b;
  }
  __syncthreads();

  for (int s = tid; s <= p.num_seqs; s += kPlanThreads) {
    p.query_start_loc[s] = tok_s[s];
    if (s < p.num_seqs) p.seq_lens[s] = ctx_s[s] + (tok_s[s + 1] - tok_s[s]);
  }
  if (tid == 0) *p.free_count_out = raw_count - total_b;

  // new blocks, in the order of the requests
  for (int k = tid; k < total_b; k += kPlanThreads) {
    const int s = owner_of(blk_s, p.num_seqs, k);
    const int col = (int)(((long long)ctx_s[s] + bs - 1) / bs) + (k - blk_s[s]);
    int id = p.free_blocks[count - 1 - k];
    if (id < 0 || id >= p.num_blocks) bad = true, id = -1;
    p.block_tables[(int64_t)s * p.max_blocks + col] = id;
  }
  // token rows; those past the last new token are padding
  for (int t = tid; t < p.num_tokens; t += kPlanThreads) {
    int slot = -1, pos = 0;
    if (t < total_t) {
      const int s = owner_of(tok_s, p.num_seqs, t);
      const int c = ctx_s[s];
      const int at = c + (t - tok_s[s]);
      const int col = at / bs;
      const int first = (int)(((long long)c + bs - 1) / bs);
      const int id = col >= first ? p.free_blocks[count - 1 - (blk_s[s] + col - first)]
                                  : p.block_tables[(int64_t)s * p.max_blocks + col];
      if (id < 0 || id >= p.num_blocks)
        bad = true;
      else
        slot = id * bs + at % bs;
      pos = at + (p.position_offsets ? p.position_offsets[s] : 0);
    }
    p.slot_mapping[t] = slot;
    for (int a = 0; a < p.num_axes; ++a) p.positions[(int64_t)a * p.num_tokens + t] = pos;
  }
  if (bad) flag_error(p.err, DEVERR_BOUNDS);
}

}  // namespace

cudaError_t launch_build_step(const StepPlanArgs& p, cudaStream_t stream) {
  const size_t smem = ((size_t)3 * p.num_seqs + 2) * sizeof(int);
  if (smem > 48 * 1024) {
    // (always the most any call takes, so that calls on other threads agree)
    cudaError_t e = cudaFuncSetAttribute(build_step_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)((3 * kMaxPlanSeqs + 2) * sizeof(int)));
    if (e != cudaSuccess) return e;
  }
  build_step_kernel<<<1, kPlanThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
