// Host side shared by the GEMM launches: tensor maps of the operands and the
// output, the SM count and the shared-memory opt-in.
#pragma once

#include "context.h"
#include "kernels.h"

namespace fp8blk {

// 2-D map over a row-major [rows][cols] E4M3 matrix, box = box_rows x 128 bytes, 128-byte swizzle.
inline bool make_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_rows) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of the output for the TMA-store epilogue: bf16 [rows][ld], boxes of 32
// rows x 64 columns (128 bytes) in the 128-byte swizzle.  An fp32 output
// leaves by plain stores; its map (the same extent read as bf16, the fp32 row
// pitch) is never used.
inline bool make_out_map(CUtensorMap* map, void* base, int64_t rows, int64_t cols, int64_t ld, bool f32) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld * (f32 ? 4 : 2))};
  const cuuint32_t box[2] = {64, 32};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SM count of the current device (cached per context).
inline int num_sms() {
  static PerContext<int> cache;
  int sms = 0;
  const cudaError_t e = cache.get(&sms, [](int* v) {
    int dev = 0;
    cudaError_t r = cudaGetDevice(&dev);
    if (r == cudaSuccess) r = cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
    return r;
  });
  return (e == cudaSuccess && sms > 0) ? sms : 1;
}

// Opts a kernel into `bytes` of dynamic shared memory, once per context.
template <typename Kernel>
cudaError_t set_smem_once(PerContext<int>& cache, Kernel kernel, int bytes) {
  int done = 0;
  return cache.get(&done, [&](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}

}  // namespace fp8blk
