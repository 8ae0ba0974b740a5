// pa_select.cuh -- the K largest of n 32-bit keys, by a block or by a warp (used by the
// choice of blocks and by the eviction of tokens), and what a cluster's CTAs do together.
//
// Keys are unsigned (ordered_key() maps floats to them in their order); a key of all bits
// set is always chosen.  The K-th largest key is found from the top: by a block digit by
// digit (a histogram of the digit among the keys that agree with what is known, and the
// digit where the count from above passes K), by a warp bit by bit over registers.  Both
// begin below the bits that all keys share and end as soon as a count comes out even.
// Ties go to the lowest index, so what is chosen depends on the keys alone: counts are
// integers, whatever the order of the atomics.
#pragma once

#include <cstdint>

#include "pa_common.cuh"

namespace pa {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared-memory address `local` of this CTA, in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t local, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// The two halves of a cluster barrier, apart.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// Over the cluster, or (one CTA) the block.
__device__ __forceinline__ void group_sync(uint32_t ctas) {
  if (ctas > 1)
    cluster_sync();
  else
    __syncthreads();
}

// Floats as unsigned numbers in the same order: -0 is 0, every NaN is the largest.
__device__ __forceinline__ uint32_t ordered_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

constexpr uint32_t kAlways = 0xffffffffu;  // the key that is chosen whatever K

struct SelectShared {
  uint32_t warp_a[32], warp_b[32];
  uint32_t all, any, always;  // bits of all keys, of any; keys that are always chosen
  uint32_t digit, above, here;
};

// Exclusive prefix sums of a and b over the block's threads (in order of threadIdx.x);
// the block's totals in all_a, all_b.
__device__ __forceinline__ void block_scan2(SelectShared& B, uint32_t a, uint32_t b, uint32_t& pre_a,
                                            uint32_t& pre_b, uint32_t& all_a, uint32_t& all_b) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  uint32_t ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t va = __shfl_up_sync(0xffffffffu, ia, o);
    const uint32_t vb = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) ia += va, ib += vb;
  }
  __syncthreads();  // (an earlier call's sums have been read)
  if (lane == 31) B.warp_a[warp] = ia, B.warp_b[warp] = ib;
  __syncthreads();
  uint32_t before_a = 0, before_b = 0;
  all_a = all_b = 0;
  for (int w = 0; w < warps; ++w) {
    const uint32_t wa = B.warp_a[w], wb = B.warp_b[w];
    if (w < warp) before_a += wa, before_b += wb;
    all_a += wa, all_b += wb;
  }
  pre_a = before_a + ia - a;
  pre_b = before_b + ib - b;
}

// What a thread has seen of the keys: the bits of all of them and of any, but for those that
// are always chosen, which it counts.
struct KeyBits {
  uint32_t all = kAlways, any = 0, always = 0;
  __device__ __forceinline__ void see(uint32_t k) {
    if (k == kAlways)
      ++always;
    else
      all &= k, any |= k;
  }
};

// The threshold that leaves the K largest of n keys, read by key(i): those above `key`, and
// the first `equal` of those that are `key` itself.  0 < K <= n.  Every thread of the block,
// of kSelectBins / 8 threads at least; seen: of the block's threads together every key once;
// hist: kSelectBins words of shared memory.
struct Threshold {
  uint32_t key, equal;
};
constexpr int kSelectDigit = 11, kSelectBins = 1 << kSelectDigit;
template <class Key>
__device__ Threshold select_threshold(SelectShared& B, uint32_t* hist, int n, uint32_t K, Key key,
                                      KeyBits seen) {
  const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
  const int per = kSelectBins / threads;  // bins of a thread
  for (int i = tid; i < kSelectBins; i += threads) hist[i] = 0;
  if (tid == 0) B.all = kAlways, B.any = 0, B.always = 0;
  __syncthreads();
  {
    const uint32_t all = __reduce_and_sync(kAlways, seen.all);
    const uint32_t any = __reduce_or_sync(kAlways, seen.any);
    const uint32_t always = __reduce_add_sync(kAlways, seen.always);
    if (lane == 0) {
      atomicAnd(&B.all, all);
      atomicOr(&B.any, any);
      if (always) atomicAdd(&B.always, always);
    }
  }
  __syncthreads();
  const uint32_t all = B.all, any = B.any;
  // (at most as many as there are are asked for: the others of them are ties at the top)
  if (B.always >= K) return Threshold{kAlways, K};
  uint32_t left = K - B.always;  // how many of the keys that agree with `known` are to be kept
  int top = all == any ? 0 : 32 - __clz(all ^ any);  // bits still open
  uint32_t mask = top == 32 ? 0u : kAlways << top, known = all & mask;
  while (top > 0) {
    const int shift = top > kSelectDigit ? top - kSelectDigit : 0;
    // (of the digit's bits, those above `top` are zeros)
    const auto count = [&](uint32_t k) {
      if (k != kAlways && (k & mask) == known) atomicAdd(&hist[(k & ~mask) >> shift], 1u);
    };
    int i = tid;
    for (; i + 3 * threads < n; i += 4 * threads) {  // (several loads in flight)
      const uint32_t k0 = key(i), k1 = key(i + threads), k2 = key(i + 2 * threads),
                     k3 = key(i + 3 * threads);
      count(k0), count(k1), count(k2), count(k3);
    }
    for (; i < n; i += threads) count(key(i));
    __syncthreads();
    // thread 0 has the highest bins
    uint32_t c[8], sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= per) continue;
      const int d = kSelectBins - 1 - (tid * per + j);
      sum += c[j] = hist[d];
      hist[d] = 0;
    }
    uint32_t before, unused, total, unused2;
    block_scan2(B, sum, 0u, before, unused, total, unused2);
    if (before < left && left <= before + sum) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= per) continue;
        if (before < left && left <= before + c[j])
          B.digit = kSelectBins - 1 - (tid * per + j), B.above = before, B.here = c[j];
        before += c[j];
      }
    }
    __syncthreads();
    known |= B.digit << shift;
    mask |= kAlways << shift;
    left -= B.above;
    top = shift;
    // all that agree so far are kept: no lower digit matters
    if (left == B.here && known != 0) return Threshold{known - 1, 0u};
  }
  return Threshold{known, left};
}

// The K largest over a warp's registers: k[j] of lane i is key 32 j + i, those from n on are
// not there.  Sets bit j of the result for the lane's chosen ones: K in all, never more (of
// more keys that are always chosen the first K).  0 < K <= n.
template <int NJ>
__device__ __forceinline__ uint32_t select_in_warp(const uint32_t (&k)[NJ], int n, int K) {
  const int lane = threadIdx.x & 31;
  uint32_t chosen = 0, all = kAlways, any = 0;
  int fixed = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool there = 32 * j + lane < n;
    if (there && k[j] == kAlways) chosen |= 1u << j, ++fixed;
    if (there && k[j] != kAlways) all &= k[j], any |= k[j];
  }
  // of the keys that are T the first `left`
  const auto take_first = [&](uint32_t T, int left) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const bool tie = 32 * j + lane < n && k[j] == T;
      const uint32_t ball = __ballot_sync(kAlways, tie);
      if (tie && __popc(ball & ((1u << lane) - 1u)) < left) chosen |= 1u << j;
      left -= __popc(ball);
    }
  };
  fixed = __reduce_add_sync(kAlways, fixed);
  if (fixed > K) {
    chosen = 0;
    take_first(kAlways, K);
    return chosen;
  }
  K -= fixed;
  if (K == 0) return chosen;
  all = __reduce_and_sync(kAlways, all);
  any = __reduce_or_sync(kAlways, any);
  // the bits that all keys share, then bit by bit: the largest T with at least K keys >= T
  int bit = all == any ? -1 : 31 - __clz(all ^ any);
  uint32_t T = bit < 0 ? all : bit == 31 ? 0u : all & (kAlways << (bit + 1));
  bool exact = false;
  for (; bit >= 0 && !exact; --bit) {
    const uint32_t t = T | 1u << bit;
    int count = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      count += 32 * j + lane < n && k[j] >= t && k[j] != kAlways;
    count = __reduce_add_sync(kAlways, count);
    if (count >= K) T = t;
    exact = count == K;
  }
  // all above T, and of those at T the first
  int above = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool there = 32 * j + lane < n && k[j] != kAlways;
    if (there && (k[j] > T || (exact && k[j] == T))) chosen |= 1u << j, ++above;
  }
  if (exact) return chosen;
  // (there are keys below kAlways, as K of them are left to choose, so T is one of them)
  take_first(T, K - __reduce_add_sync(kAlways, above));
  return chosen;
}

}  // namespace pa
