// tma.cu -- tensor maps (see tma.h).  The driver's encoder is reached through
// the runtime's driver entry point, so the library does not link the driver
// library.
#include "tma.h"

#include <mutex>

namespace bakron {

cudaError_t make_tensor_map(CUtensorMap* out, const TileMap& t) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Encode encode = nullptr;
  static cudaError_t lookup = cudaSuccess;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    lookup = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (lookup == cudaSuccess && q == cudaDriverEntryPointSuccess) encode = reinterpret_cast<Encode>(f);
    if (lookup == cudaSuccess && !encode) lookup = cudaErrorSymbolNotFound;
  });
  if (lookup != cudaSuccess) return lookup;
  const int64_t bytes = t.type == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)t.cols, (cuuint64_t)t.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(t.ld * bytes)};
  const cuuint32_t box[2] = {t.box_cols, t.box_rows}, step[2] = {1, 1};
  const CUresult r = encode(out, t.type, 2, const_cast<void*>(t.base), dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE,
                            t.swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace bakron
