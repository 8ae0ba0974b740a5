// pa_select.cuh -- the K largest of n 32-bit keys spread over the CTAs of a cluster
// (used by the choice of blocks and by the eviction of tokens).
//
// Keys are unsigned (ordered_key() maps floats to them in their order).  The K-th
// largest key is found digit by digit from the top: a histogram of the digit among
// the keys that still agree with what is known, added up over the cluster through
// distributed shared memory, and the digit where the count from above passes K.
// Ties at that key go to the lowest index, so what is chosen depends on the keys
// alone: counts are integers, whatever the order of the atomics.
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
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
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

struct SelectShared {
  uint32_t hist[2][256];
  uint32_t total[256];
  uint32_t warp_a[32], warp_b[32];
  uint32_t digit, above;
  uint32_t mine[2];  // this CTA's counts above the threshold and at it
};

// The threshold that leaves the K largest keys of the cluster: those above `key`,
// and the first `equal` of those that are `key` itself.  n: keys of this CTA, read
// by key(i).  0 < K <= keys of the cluster.  Every thread of the cluster calls it;
// blockDim.x is at least 256.
struct Threshold {
  uint32_t key, equal;
};
template <class Key>
__device__ Threshold select_threshold(SelectShared& B, int n, uint32_t K, uint32_t ctas, Key key) {
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t known = 0, mask = 0;
  uint32_t left = K;  // how many of the keys that agree with `known` are to be kept
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    uint32_t* hist = B.hist[pass & 1];
    // (remote reads of this buffer, two passes ago, ended before the barrier of the last pass)
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += blockDim.x) {
      const uint32_t k = key(i);
      if ((k & mask) == known) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    group_sync(ctas);
    if (tid < 256) {
      uint32_t sum = 0;
      if (ctas > 1) {
        const uint32_t at = smem_addr(&hist[tid]);
        for (uint32_t r = 0; r < ctas; ++r) sum += ld_cluster_u32(cluster_addr(at, r));
      } else {
        sum = hist[tid];
      }
      B.total[tid] = sum;
    }
    __syncthreads();
    if (tid < 32) {
      // lane 0 holds the highest eight digits
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += c[j] = B.total[255 - (lane * 8 + j)];
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      uint32_t before = incl - sum;
      if (before < left && left <= incl) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (before < left && left <= before + c[j]) {
            B.digit = 255 - (lane * 8 + j);
            B.above = before;
          }
          before += c[j];
        }
      }
    }
    __syncthreads();
    known |= B.digit << shift;
    mask |= 255u << shift;
    left -= B.above;
  }
  return Threshold{known, left};
}

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

}  // namespace pa
