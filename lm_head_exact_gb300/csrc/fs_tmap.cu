// TMA tensor-map encoding through the driver entry point obtained from the
// runtime, so the library needs no link-time dependency on libcuda.
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "fs_tmap.h"

namespace fs {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 find_encode() {
  cudaDriverEntryPointQueryResult q;
  void* ptr = nullptr;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
}

// The driver encodes under the calling thread's context.  A host thread whose
// first CUDA work is this call has none bound yet (the runtime's queries made
// before it bind none), so a failure binds the device's and tries once more.
bool bind_context() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
}

bool encode(CUtensorMap* tm, CUtensorMapDataType type, int width, const void* base, int64_t rows, int64_t cols,
            int64_t pitch, int box_cols, int box_rows) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = find_encode();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * width};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t steps[2] = {1, 1};
  const auto run = [&]() {
    return encode(tm, type, 2, const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  return run() || (bind_context() && run());
}

}  // namespace

bool encode_rows_bf16(CUtensorMap* tm, const void* base, int64_t rows, int64_t cols, int64_t pitch, int box_cols,
                      int box_rows) {
  return encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, rows, cols, pitch, box_cols, box_rows);
}

bool encode_rows_u8(CUtensorMap* tm, const void* base, int64_t rows, int64_t cols, int64_t pitch, int box_cols,
                    int box_rows) {
  return encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, rows, cols, pitch, box_cols, box_rows);
}

bool encode_kmajor_bf16(CUtensorMap* tm, const void* base, int64_t rows, int64_t d, int box_cols, int box_rows) {
  return encode_rows_bf16(tm, base, rows, d, d, box_cols, box_rows);
}

}  // namespace fs
