// TMA tensor maps: the driver's encoder, looked up once (libcuda is not linked).
#include "tensor_map.cuh"

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

namespace fljsd {

bool make_tensor_map(CUtensorMap* m, MapType type, const void* ptr, int64_t inner, int64_t outer,
                     int64_t ld, int box_inner, int box_outer, bool swizzle) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  if (!encode) return false;
  const int size = type == MapType::kF32 ? 4 : type == MapType::kBf16 ? 2 : 1;
  const CUtensorMapDataType t = type == MapType::kF32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : type == MapType::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)ld * size};
  cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_outer};
  cuuint32_t estr[2] = {1, 1};
  return encode(m, t, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE,
                swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace fljsd
