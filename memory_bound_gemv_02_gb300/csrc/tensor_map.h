// Tensor maps of the TMA copies, encoded per call.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "ops_internal.h"

namespace gemvk {

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (looked up once).
inline EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// A map of `rank` dimensions (innermost first, strides in bytes from the second
// on); what lies outside reads as zero.
inline bool encode_map(CUtensorMap *map, const void *p, int type, int rank, const cuuint64_t *dims,
                       const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const CUtensorMapDataType t = type == GEMV_TYPE_F16    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                : type == GEMV_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                : type == GEMV_TYPE_F32  ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                         : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, t, (cuuint32_t)rank, const_cast<void *>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gemvk
