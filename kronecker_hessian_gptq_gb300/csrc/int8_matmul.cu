// int8_matmul.cu -- the product of quantized activations and quantized weights,
//     Y[t, o] = s_t w_o sum_k c[t, k] v[o, k] + b_o,
// for 8-bit codes c (one scale s_t for each token) and v (one scale w_o for
// each output), and the codes of activations,
//     s_t = fp32(max_k |x_tk| / 127), c_tk = rint(fp32(x_tk / s_t)).
// The integer sums are exact.
#include <algorithm>

#include "bakron.h"
#include "elem.cuh"
#include "layers.h"
#include "quantize_tokens.cuh"
#include "tile_product.cuh"

namespace bakron {
namespace {

template <class T>
__global__ void __launch_bounds__(256) quantize_tokens_kernel(const T* X, int64_t K, int64_t ldx, int8_t* C, int64_t ldc,
                                                              float* s) {
  __shared__ float red[32];
  const T* x = X + (int64_t)blockIdx.x * ldx;
  float top[1] = {0.f};
  for (int64_t k = threadIdx.x; k < K; k += 256) top[0] = MaxOp()(fabsf(to_f32<T>(x[k])), top[0]);
  block_reduce<1>(top, red, MaxOp());
  const float scale = token_scale(top[0]), inv = token_inv(scale);
  if (threadIdx.x == 0) s[blockIdx.x] = scale;
  int8_t* c = C + (int64_t)blockIdx.x * ldc;
  for (int64_t k = threadIdx.x; k < K; k += 256) c[k] = (int8_t)token_code(to_f32<T>(x[k]), scale, inv);
}

struct Codes {
  const int8_t* p;
  int64_t ld;
  __device__ int operator()(int64_t r, int64_t k) const { return p[r * ld + k]; }
};
struct CodesT {
  const int8_t* p;
  int64_t ld;
  __device__ int operator()(int64_t k, int64_t r) const { return p[r * ld + k]; }
};
template <class T>
struct PutScaled {
  const float *s, *w, *b;
  T* y;
  int64_t ld;
  __device__ void operator()(int64_t t, int64_t o, int v) const {
    y[t * ld + o] = from_f32<T>(fmaf((float)v * s[t], w[o], b ? b[o] : 0.f));
  }
};

template <class T>
void product(const Int8Matmul& p, const int8_t* C, int64_t ldc, const float* s, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.N + 63) / 64), (unsigned)((p.T + 63) / 64));
  tile_product_kernel<int><<<grid, 256, 0, stream>>>(p.T, p.N, p.K, Codes{C, ldc}, CodesT{p.V, p.ldv},
                                                     PutScaled<T>{s, p.scales, p.bias, static_cast<T*>(p.Y), p.ldy});
}

}  // namespace

cudaError_t quantize_tokens_launch(const void* X, int dtype, int64_t T, int64_t K, int64_t ldx, int8_t* C, int64_t ldc,
                                   float* s, cudaStream_t stream) {
  const unsigned grid = (unsigned)T;
  switch (dtype) {
    case kF32: quantize_tokens_kernel<<<grid, 256, 0, stream>>>((const float*)X, K, ldx, C, ldc, s); break;
    case kF16: quantize_tokens_kernel<<<grid, 256, 0, stream>>>((const __half*)X, K, ldx, C, ldc, s); break;
    default: quantize_tokens_kernel<<<grid, 256, 0, stream>>>((const __nv_bfloat16*)X, K, ldx, C, ldc, s);
  }
  return cudaGetLastError();
}

size_t int8_matmul_workspace_bytes(int64_t T, int64_t K, int64_t N) { return (size_t)(T * K + 255) / 256 * 256 + T * 4; }

cudaError_t int8_matmul_launch(const Int8Matmul& p, void* ws, int32_t* status_dev, cudaStream_t stream) {
  cudaError_t e = cudaMemsetAsync(status_dev, 0, sizeof(int32_t), stream);
  if (e != cudaSuccess) return e;
  const int8_t* C = static_cast<const int8_t*>(p.X);
  int64_t ldc = p.ldx;
  const float* s = p.x_scales;
  if (!s) {
    int8_t* codes = static_cast<int8_t*>(ws);
    float* scales = reinterpret_cast<float*>(codes + (p.T * p.K + 255) / 256 * 256);
    e = quantize_tokens_launch(p.X, p.x_dtype, p.T, p.K, p.ldx, codes, p.K, scales, stream);
    if (e != cudaSuccess) return e;
    C = codes, ldc = p.K, s = scales;
  }
  switch (p.y_dtype) {
    case kF32: product<float>(p, C, ldc, s, stream); break;
    case kF16: product<__half>(p, C, ldc, s, stream); break;
    default: product<__nv_bfloat16>(p, C, ldc, s, stream);
  }
  return cudaGetLastError();
}

}  // namespace bakron
