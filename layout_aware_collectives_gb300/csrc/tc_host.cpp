// Tensor maps of the tensor-core kernels' operands.
#include "tc_host.h"

namespace tide {
namespace {

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess) {
      cudaGetLastError();
      return (EncodeTiled) nullptr;
    }
    return found == cudaDriverEntryPointSuccess ? (EncodeTiled)p : (EncodeTiled) nullptr;
  }();
  return fn;
}

}  // namespace

bool make_map(CUtensorMap* map, const void* p, int elem, int64_t cols, int64_t rows, int64_t ld, uint32_t box_cols,
              uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  const EncodeTiled encode = encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * elem};
  const cuuint32_t box[2] = {box_cols, box_rows}, step[2] = {1, 1};
  return encode(map, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_slab_map(CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t ld, uint32_t box_rows) {
  const EncodeTiled encode = encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(cols / 64)};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, 128};
  const cuuint32_t box[3] = {64, box_rows, 2}, step[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_stack_map(CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t count, int64_t ld,
                    uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  const EncodeTiled encode = encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(ld * rows) * 2};
  const cuuint32_t box[3] = {box_cols, box_rows, 1}, step[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_slab_stack_map(CUtensorMap* map, const void* p, int64_t rows, int64_t count, int64_t ld, uint32_t box_rows,
                         uint32_t box_slabs) {
  const EncodeTiled encode = encoder();
  if (!encode) return false;
  const cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)(ld / 64), (cuuint64_t)count};
  const cuuint64_t strides[3] = {(cuuint64_t)ld * 2, 128, (cuuint64_t)(ld * rows) * 2};
  const cuuint32_t box[4] = {64, box_rows, box_slabs, 1}, step[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(p), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t held_clusters(const void* kernel, int threads, size_t smem, int most, int* held) {
  for (int s = 2; s <= most; ++s) {
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim = {2u * s, 1, 1};
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(2 * s);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.attrs = &cluster;
    c.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&held[s], kernel, &c);
    if (e == cudaSuccess) continue;
    if (s <= 4) return e;
    held[s] = 0;  // more CTAs than any device has to take in one cluster
    (void)cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace tide
