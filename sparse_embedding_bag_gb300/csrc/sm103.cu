// Host side of sm103.cuh: tensor maps, and what is asked of a device once.
#include "sm103.cuh"

#include <atomic>

namespace embbwd {

namespace {

cudaError_t encode(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t width, uint64_t rows,
                   uint64_t row_bytes, uint32_t box_width, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static std::atomic<void*> entry{nullptr};
  void* fn = entry.load(std::memory_order_acquire);
  if (!fn) {
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    entry.store(fn, std::memory_order_release);
  }
  const cuuint64_t dims[2] = {width, rows}, strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_width, box_rows}, step[2] = {1, 1};
  const CUresult r = reinterpret_cast<Encode>(fn)(map, type, 2, const_cast<void*>(base), dims, strides, box, step,
                                                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t byte_matrix_map(CUtensorMap* map, const void* base, int64_t rows, int64_t row_bytes, int box_rows) {
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, row_bytes, rows, row_bytes, 128, box_rows,
                CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t tile_matrix_map(CUtensorMap* map, const void* base, int64_t rows, int64_t tiles, int box_rows,
                            int box_tiles) {
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_INT64, base, tiles * 64, rows, tiles * 512, box_tiles * 64, box_rows,
                CU_TENSOR_MAP_SWIZZLE_NONE);
}

int sm_count(int device) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  if (device < kDevices) {
    const int n = known[device].load(std::memory_order_relaxed);
    if (n) return n;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1) n = 1;
  if (device < kDevices) known[device].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace embbwd
