// fp8_codes.cuh -- e4m3 codes with one scale for a block of values:
//     scale = fp32(max |x| / 448),  code = e4m3(fp32(x r)),  r = fp32(1 / scale),
// rounded to nearest, ties to even.  A block of zeros (or so small that r would
// overflow) has scale 0 and codes 0; a block that holds a NaN or an infinity
// has scale NaN and codes 0, so that what is computed from it is NaN.
#pragma once

#include <cuda_fp8.h>

#include "elem.cuh"

namespace bakron {

constexpr int kFp8Block = 128;

// top: the largest magnitude's bits, which order as the magnitudes do, with
// infinity and then NaN above all.
__device__ __forceinline__ void block_scale(uint32_t top, float& scale, float& inv) {
  scale = __fdiv_rn(__uint_as_float(top), 448.f);
  inv = 0.f;
  if (top >= 0x7f800000u)
    scale = __int_as_float(0x7fffffff);
  else if (scale >= 1.17549435e-38f)
    inv = __fdiv_rn(1.f, scale);
  else
    scale = 0.f;
}
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t fp8_pair(float a, float b, float inv_a, float inv_b) {
  // A block without a reciprocal may hold what is not finite, and 0 times that is no number.
  const float2 q = make_float2(inv_a > 0.f ? a * inv_a : 0.f, inv_b > 0.f ? b * inv_b : 0.f);
  return (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
}
// Eight codes as bytes.
__device__ __forceinline__ uint2 fp8_codes8(const float (&x)[8], float inv) {
  return make_uint2(fp8_pair(x[0], x[1], inv, inv) | (fp8_pair(x[2], x[3], inv, inv) << 16),
                    fp8_pair(x[4], x[5], inv, inv) | (fp8_pair(x[6], x[7], inv, inv) << 16));
}

}  // namespace bakron
