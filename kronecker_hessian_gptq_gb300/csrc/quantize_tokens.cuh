// quantize_tokens.cuh -- 8-bit codes of activations, one scale for each token.
#pragma once

#include "elem.cuh"

namespace bakron {

// Scale of a row whose largest magnitude is `top`: fp32(top / 127), NaN
// where the row holds a NaN or an infinity (`top` is then one of them), so
// that everything computed from the row's codes is NaN and no other row is.
__device__ __forceinline__ float token_scale(float top) {
  return top < INFINITY ? __fdiv_rn(top, 127.f) : __int_as_float(0x7fffffff);
}
// Reciprocal for token_code(): 0 for a row without a positive finite scale,
// whose codes are all 0.
__device__ __forceinline__ float token_inv(float s) { return s > 0.f ? __fdiv_rn(1.f, s) : 0.f; }

// The 8-bit code of x for the scale s: fp32(x / s) rounded to nearest, ties
// to even, kept within +-127; `inv` is token_inv(s).  x * inv is within
// 2^-23 |x / s| of the quotient and the quotient's own rounding within 2^-24
// of it, 2.3e-5 in all for a code, so both round to the same integer unless
// x * inv lies within 2^-14 of a half-integer; only then (and where 1 / s
// overflows) is the division carried out.
__device__ __forceinline__ int token_code(float x, float s, float inv) {
  if (inv == 0.f) return 0;
  const float q = x * inv;
  float r = rintf(q);
  if (!(fabsf(fabsf(q - r) - 0.5f) > 6.1035e-5f) || !(fabsf(q) < 128.f)) r = rintf(__fdiv_rn(x, s));
  return (int)fminf(fmaxf(r, -127.f), 127.f);
}

}  // namespace bakron
