// pa_window.cu -- attention with a sliding window and sink tokens over the
// paged cache: the row at position p attends to positions j <= p with
// p - j < window or j < num_sinks.
//
// One warp per (token, q head) walks the visible keys; lanes own head_dim / 32
// elements each, the dot product is a shuffle reduction, the softmax is online
// (base 2, fp32).
#include <cstdint>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kWarps = 4;

template <int D, bool F8>
__global__ void __launch_bounds__(kWarps * 32) window_kernel(const AttnArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= (int64_t)a.num_tokens * a.num_q_heads) return;
  const int t = (int)(row / a.num_q_heads), h = (int)(row % a.num_q_heads);
  if (t < a.query_start_loc[0] || t >= a.query_start_loc[a.num_seqs]) return;
  int lo = 0, hi = a.num_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.query_start_loc[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int begin = a.query_start_loc[lo], ql = a.query_start_loc[lo + 1] - begin;
  const int L = a.seq_lens[lo];
  const int bs = 16 << a.block_shift;
  if (L < ql || L > a.max_seq_len || (int64_t)L > (int64_t)a.max_blocks * bs || begin < 0 ||
      begin + ql > a.num_tokens || (a.no_decode && ql == 1)) {
    if (lane == 0) flag_error(a.err, DEVERR_BOUNDS);
    return;
  }
  const int p = L - ql + (t - begin);
  const int g = h / (a.num_q_heads / a.num_kv_heads);
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float((uint32_t)a.q[row * D + lane * E + e] << 16) *
           (a.scale * 1.4426950408889634f);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int w0 = max(0, p - a.window + 1);
  for (int j = min(a.num_sinks, w0) > 0 ? 0 : w0; j <= p; j = (j + 1 == a.num_sinks && j + 1 < w0) ? w0 : j + 1) {
    const int b = a.block_tables[(int64_t)lo * a.max_blocks + j / bs];
    if (b < 0 || b >= a.num_blocks) {
      if (lane == 0) flag_error(a.err, DEVERR_BOUNDS);
      continue;
    }
    const int64_t slot = (int64_t)b * bs + j % bs;
    float k[E], v[E];
    if (F8) {
      const int64_t page = slot / kFp8PageTokens;
      const int64_t r = (slot % kFp8PageTokens) * a.num_kv_heads + g;
      const unsigned char* kp = static_cast<const unsigned char*>(a.k_cache) +
                                page * fp8_page_bytes(a.num_kv_heads, D);
      const unsigned char* vp = static_cast<const unsigned char*>(a.v_cache) +
                                page * fp8_page_bytes(a.num_kv_heads, D);
      const float ks = *reinterpret_cast<const float*>(
          kp + fp8_scales_offset(a.num_kv_heads, D) + r * 4);
      const float vs = *reinterpret_cast<const float*>(
          vp + fp8_scales_offset(a.num_kv_heads, D) + r * 4);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        uint32_t x, y;
        f16x2x2_from_e4m3x4(kp[r * D + lane * E + e], x, y);
        k[e] = half2_bits_to_float2(x).x * ks;
        f16x2x2_from_e4m3x4(vp[r * D + lane * E + e], x, y);
        v[e] = half2_bits_to_float2(x).x * vs;
      }
    } else {
      const int64_t off = (slot * a.num_kv_heads + g) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        k[e] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.k_cache)[off + e] << 16);
        v[e] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.v_cache)[off + e] << 16);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * k[e];
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s), al = exp2f(m - mn), pr = exp2f(s - mn);
    l = l * al + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * al + pr * v[e];
    m = mn;
  }
  if (l == 0.f) return;  // every block id of the row was out of range
#pragma unroll
  for (int e = 0; e < E; ++e) a.out[row * D + lane * E + e] = float_to_bf16_rn(o[e] / l);
}

}  // namespace

cudaError_t launch_window(const AttnArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.num_tokens * a.num_q_heads;
  const unsigned grid = (unsigned)((rows + kWarps - 1) / kWarps);
  if (a.head_dim == 128 && a.fp8)
    window_kernel<128, true><<<grid, kWarps * 32, 0, stream>>>(a);
  else if (a.head_dim == 128)
    window_kernel<128, false><<<grid, kWarps * 32, 0, stream>>>(a);
  else if (a.fp8)
    window_kernel<64, true><<<grid, kWarps * 32, 0, stream>>>(a);
  else
    window_kernel<64, false><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pa
