// pa_tma_host.h -- tensor maps, which the host encodes before a launch: the driver's
// function, and the caches' maps of the kernels of the long-context operators.
#pragma once

#include <cuda.h>  // CUtensorMap (types only; nothing is linked from the driver)
#include <cuda_runtime.h>
#include <mutex>

#include "pa_internal.h"

namespace pa {

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(f);
  });
  return fn;
}

template <int RANK>
cudaError_t encode_map(CUtensorMap* m, CUtensorMapDataType type, const void* ptr,
                       const cuuint64_t (&dims)[RANK], const cuuint64_t (&strides)[RANK - 1],
                       const cuuint32_t (&box)[RANK], CUtensorMapSwizzle swizzle,
                       CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  EncodeTiled enc = encode_tiled();
  if (!enc) return cudaErrorNotSupported;
  cuuint32_t es[RANK];
  for (int i = 0; i < RANK; ++i) es[i] = 1;
  const CUresult r = enc(m, type, RANK, const_cast<void*>(ptr), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A box is a 16-token page of one kv head: bf16 [64-channel half][16][64] at (0, h, first
// row, 0), 8-bit codes [16][head_dim] at (0, h, 0, page); 128-byte rows with the 128-byte
// swizzle (64-byte rows: the 64-byte one).  L2 fetches no more than a row: the next head's
// row beside it may never be read.
inline cudaError_t encode_page_map(CUtensorMap* m, const void* cache, bool fp8, int64_t pages,
                                   int n_kv, int head_dim) {
  const cuuint64_t d = (cuuint64_t)head_dim, h = (cuuint64_t)n_kv, n = (cuuint64_t)pages;
  if (fp8) {
    const cuuint64_t dims[4] = {d, h, 16, n};
    const cuuint64_t strides[3] = {d, h * d, (cuuint64_t)fp8_page_bytes(n_kv, head_dim)};
    const cuuint32_t box[4] = {(cuuint32_t)d, 1, 16, 1};
    return encode_map<4>(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache, dims, strides, box,
                         head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         head_dim == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                         : CU_TENSOR_MAP_L2_PROMOTION_L2_64B);
  }
  const cuuint64_t dims[4] = {64, h, n * 16, d / 64};
  const cuuint64_t strides[3] = {d * 2, h * d * 2, 128};
  const cuuint32_t box[4] = {64, 1, 16, (cuuint32_t)(d / 64)};
  return encode_map<4>(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cache, dims, strides, box,
                       CU_TENSOR_MAP_SWIZZLE_128B,
                       head_dim == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                       : CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
}

}  // namespace pa
