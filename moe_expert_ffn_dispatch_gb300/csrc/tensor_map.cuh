// Host side: tensor maps of the TMA copies.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace moe {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, asked for once; nullptr if there is none.
inline EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool got = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                         cudaSuccess &&
                     q == cudaDriverEntryPointSuccess;
    return got ? reinterpret_cast<EncodeTiledFn>(f) : nullptr;
  }();
  return fn;
}

// 2-D row-major [rows][cols] tensor, rows `stride` elements apart (dense without it), box {box_cols, box_rows}
inline bool encode_2d(CUtensorMap* m, const void* base, CUtensorMapDataType dt, size_t elem, uint64_t rows, uint64_t cols,
                      uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle sw, uint64_t stride = 0) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {(stride ? stride : cols) * elem};
  const cuuint32_t box[2] = {box_cols, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
