// pa_decode_window_fp8.cu -- the sliding-window instantiations of the split-KV decode kernel
// (pa_decode_kernel.cuh) over the 8-bit cache.  A translation unit of its own
// so that the instantiations compile in parallel.
#include "pa_decode_kernel.cuh"

namespace pa {

cudaError_t launch_decode_window_fp8(const AttnArgs& a, const DecodeWorkspace& ws, int ctas,
                                 cudaStream_t stream) {
  return launch_decode_any<true, false, true>(a, ws, ctas, stream);
}

}  // namespace pa
