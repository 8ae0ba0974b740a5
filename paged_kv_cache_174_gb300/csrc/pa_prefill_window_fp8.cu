// pa_prefill_window_fp8.cu -- the chunked-prefill kernel's sliding-window instance for the
// 8-bit cache, in a translation unit of its own so that the instances compile
// in parallel.
#include "pa_prefill_kernel.cuh"

namespace pa {

cudaError_t launch_prefill_window_fp8(const AttnArgs& a, const PrefillPlan& plan, void* ws,
                                  int sm_count, cudaStream_t stream) {
  const int group = a.num_q_heads / a.num_kv_heads;
#define PA_PREFILL_WINDOW_FP8_CASE(D_, G_)                                            \
  if (a.head_dim == D_ && group == G_)                                                  \
    return pair_query_tiles<D_, G_, kKindFp8>(a, plan, sm_count)                      \
               ? launch_prefill_t<D_, G_, kKindFp8, true, 2>(a, plan, ws, sm_count, stream) \
               : launch_prefill_t<D_, G_, kKindFp8, true, 1>(a, plan, ws, sm_count, stream);
  PA_PREFILL_WINDOW_FP8_CASE(128, 1)
  PA_PREFILL_WINDOW_FP8_CASE(128, 2)
  PA_PREFILL_WINDOW_FP8_CASE(128, 4)
  PA_PREFILL_WINDOW_FP8_CASE(128, 8)
  PA_PREFILL_WINDOW_FP8_CASE(64, 1)
  PA_PREFILL_WINDOW_FP8_CASE(64, 2)
  PA_PREFILL_WINDOW_FP8_CASE(64, 4)
  PA_PREFILL_WINDOW_FP8_CASE(64, 8)
#undef PA_PREFILL_WINDOW_FP8_CASE
  return cudaErrorInvalidValue;
}

}  // namespace pa
