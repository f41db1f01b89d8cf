// Host helper: tensor maps for tiled TMA loads of strided [batch, rows, columns] arrays.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
  }();
  return fn;
}

// Map of base[batch][rows][cols] with the given strides (elements; the columns are contiguous) in boxes of
// box_rows x box_cols, zeros outside.  The caller has checked that base and strides are multiples of 16
// bytes.  False where CUDA does not take it (an axis that is broadcast, for one).
bool make_tensor_map(CUtensorMap* m, bool bf16, const void* base, int64_t batch, int64_t rows, int64_t cols,
                            int64_t batch_stride, int64_t row_stride, int box_rows, int box_cols) {
  const auto encode = tensor_map_encoder();
  const int64_t e = bf16 ? 2 : 4;
  if (!encode || (rows > 1 && row_stride <= 0) || (batch > 1 && batch_stride <= 0)) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
  // an axis of one element never uses its stride: any valid one
  const cuuint64_t row_bytes = rows > 1 ? (cuuint64_t)(row_stride * e) : 16;
  const cuuint64_t strides[2] = {row_bytes, batch > 1 ? (cuuint64_t)(batch_stride * e) : row_bytes};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
  return encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace ssd
