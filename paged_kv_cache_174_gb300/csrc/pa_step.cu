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
// Kilobytes move, so latency is all there is (64 decodes 3.1 us back to back;
// 256 requests with 20K token rows on three axes 7.0 us, 30.8 with one CTA).  Every
// CTA scans all the lengths into its shared memory (cheaper than handing the sums
// over), then the CTAs' threads walk the flat lists of new blocks and of token rows,
// each finding its request by a binary search of the prefix sums.  The grid is one cluster, so
// that its barrier can keep every write behind every CTA's reads: seq_lens may
// be context_lens, and free_count_out free_count.
#include <cstdint>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kPlanWarps = 32;  // at most
// Up to this many token rows one CTA of 512 threads does the step; past it a
// cluster of eight of 1024.
constexpr int kPlanOneCta = 1024;

// What a block holds in shared memory beside the requests' words.
struct PlanShared {
  long long warp_t[kPlanWarps], warp_b[kPlanWarps];
  int served_t, served_b;
};
// Dynamic shared memory that a launch may take without asking for more: a block's
// 48 KB hold its static part and the padding between the two as well.
constexpr size_t kPlanSmemPlain = 47 * 1024;
static_assert(sizeof(PlanShared) + 128 <= 48 * 1024 - kPlanSmemPlain, "");

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

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kPlanWarps * 32) build_step_kernel(const StepPlanArgs p) {
  extern __shared__ int smem_i[];
  int* ctx_s = smem_i;                     // [num_seqs]
  int* tok_s = ctx_s + p.num_seqs;         // [num_seqs + 1] exclusive prefix of new tokens
  int* blk_s = tok_s + p.num_seqs + 1;     // [num_seqs + 1] exclusive prefix of new blocks
  __shared__ PlanShared B;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int threads = blockDim.x, warps = threads >> 5;
  const int me = blockIdx.x * threads + tid, all = gridDim.x * threads;
  const int bs = p.block_size;

  after_prior_kernels();
  const int raw_count = *p.free_count;
  const bool count_ok = raw_count >= 0 && raw_count <= p.num_blocks;
  const int count = count_ok ? raw_count : 0;
  bool bad = !count_ok;
  if (tid == 0) B.served_t = 0, B.served_b = 0, tok_s[0] = 0, blk_s[0] = 0;

  bool cut = false;                // a request of this thread was not served
  long long run_t = 0, run_b = 0;  // totals of the chunks before this one
  for (int s0 = 0; s0 < p.num_seqs; s0 += threads) {
    const int s = s0 + tid;
    long long nt = 0, nb = 0;
    if (s < p.num_seqs) {
      const int c = p.context_lens[s], n = p.new_lens[s];
      ctx_s[s] = c;
      if (c >= 0 && n >= 0 && (long long)c + n <= (long long)p.max_blocks * bs) {
        // (at most 2^31 - 1 positions: no overflow in 32 bits, unsigned)
        nt = n;
        nb = ((unsigned)c + n + bs - 1) / (unsigned)bs - ((unsigned)c + bs - 1) / (unsigned)bs;
      } else {
        bad = true;  // a length out of range: no rows, no blocks
      }
    }
    long long it = warp_scan(nt, lane), ib = warp_scan(nb, lane);
    if (s0) __syncthreads();  // the last chunk's warp totals have been read
    if (lane == 31) B.warp_t[warp] = it, B.warp_b[warp] = ib;
    __syncthreads();
    const long long wt = warp_scan(lane < warps ? B.warp_t[lane] : 0, lane);
    const long long wb = warp_scan(lane < warps ? B.warp_b[lane] : 0, lane);
    const int before = warp > 0 ? warp - 1 : 0;
    const long long pt = __shfl_sync(0xffffffffu, wt, before);
    const long long pb = __shfl_sync(0xffffffffu, wb, before);
    it += run_t + (warp > 0 ? pt : 0), ib += run_b + (warp > 0 ? pb : 0);
    run_t += __shfl_sync(0xffffffffu, wt, 31), run_b += __shfl_sync(0xffffffffu, wb, 31);
    const bool mine = s < p.num_seqs;
    const bool served = mine && it <= p.num_tokens && ib <= count;
    const unsigned ball = __ballot_sync(0xffffffffu, served);
    if (served) {
      tok_s[s + 1] = (int)it;
      blk_s[s + 1] = (int)ib;
      if ((ball >> lane) == 1u) {  // the warp's last served request
        atomicMax(&B.served_t, (int)it);
        atomicMax(&B.served_b, (int)ib);
      }
    } else if (mine) {
      tok_s[s + 1] = -1;  // past the served prefix: the totals, below
      cut = true;
    }
  }
  const int any_cut = __syncthreads_or(cut);
  const int total_t = B.served_t, total_b = B.served_b;
  if (any_cut) {
    bad |= cut;
    for (int s = tid; s < p.num_seqs; s += threads)
      if (tok_s[s + 1] < 0) tok_s[s + 1] = total_t, blk_s[s + 1] = total_b;
    __syncthreads();
  }
  if (gridDim.x > 1) cluster_barrier();

  for (int s = me; s <= p.num_seqs; s += all) {
    p.query_start_loc[s] = tok_s[s];
    if (s < p.num_seqs) p.seq_lens[s] = ctx_s[s] + (tok_s[s + 1] - tok_s[s]);
  }
  if (me == 0) *p.free_count_out = raw_count - total_b;

  // new blocks, in the order of the requests
  for (int64_t k64 = me; k64 < total_b; k64 += all) {
    const int k = (int)k64;
    const int s = owner_of(blk_s, p.num_seqs, k);
    const int col = (int)(((unsigned)ctx_s[s] + bs - 1) / (unsigned)bs) + (k - blk_s[s]);
    int id = p.free_blocks[count - 1 - k];
    if (id < 0 || id >= p.num_blocks) bad = true, id = -1;
    p.block_tables[(int64_t)s * p.max_blocks + col] = id;
  }
  // token rows; those past the last new token are padding
  for (int64_t t64 = me; t64 < p.num_tokens; t64 += all) {
    const int t = (int)t64;
    int slot = -1, pos = 0;
    if (t < total_t) {
      const int s = owner_of(tok_s, p.num_seqs, t);
      const int c = ctx_s[s];
      const int at = c + (t - tok_s[s]);
      const int col = (unsigned)at / (unsigned)bs;
      const int first = (int)(((unsigned)c + bs - 1) / (unsigned)bs);
      const int id = col >= first ? p.free_blocks[count - 1 - (blk_s[s] + col - first)]
                                  : p.block_tables[(int64_t)s * p.max_blocks + col];
      if (id < 0 || id >= p.num_blocks)
        bad = true;
      else
        slot = id * bs + (at - col * bs);
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
  if (smem > kPlanSmemPlain) {
    // (always the most any call takes, so that calls on other threads agree)
    cudaError_t e = cudaFuncSetAttribute(build_step_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)((3 * kMaxPlanSeqs + 2) * sizeof(int)));
    if (e != cudaSuccess) return e;
  }
  const bool one = p.num_tokens <= kPlanOneCta;
  return launch_early(build_step_kernel, dim3(one ? 1 : 8), dim3(one ? 512 : kPlanWarps * 32), smem,
                      stream, one ? 1 : 8, p);
}

}  // namespace pa
