// layers.h -- the layer operators' launch functions (declared to callers in
// bakron.h, arguments checked in abi_layers.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bakron {

// Element types: the values of BAKRON_F32 / F16 / BF16 in bakron.h.
enum ElemType { kF32 = 0, kF16 = 1, kBF16 = 2 };
inline size_t elem_size(int dtype) { return dtype == kF32 ? 4 : 2; }
inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// int8_matmul.cu
cudaError_t quantize_tokens_launch(const void* X, int dtype, int64_t T, int64_t K, int64_t ldx, int8_t* C, int64_t ldc,
                                   float* s, cudaStream_t stream);
struct Int8Matmul {
  const void* X;      // T x K values of x_dtype, or 8-bit codes with x_scales
  const float* x_scales;  // null: X holds values
  int x_dtype;
  int64_t ldx;
  const int8_t* V;  // N x K codes
  int64_t ldv;
  const float* scales;
  const float* bias;  // or null
  int64_t T, K, N;
  void* Y;
  int y_dtype;
  int64_t ldy;
};
// copies: with room for the weights' codes in aligned rows, which
// int8_matmul_needs_copies() tells the need of.
size_t int8_matmul_workspace_bytes(int64_t T, int64_t K, int64_t N, bool copies);
bool int8_matmul_needs_copies(const Int8Matmul& p);
cudaError_t int8_matmul_launch(const Int8Matmul& p, void* ws, int32_t* status_dev, cudaStream_t stream);

// norm_residual.cu
struct NormResidual {
  const void *X, *H;  // T x D; H may be null (no block output)
  int64_t ldx, ldh;
  const float *post, *post_bias;  // D, or null
  const void* gate;               // groups x D of the element type, or null
  int64_t ldg, groups;
  const float *pre, *pre_bias;  // D, or null (pre null: no norm after the sum)
  float alpha, eps;
  int layer;  // 0: RMS norm, 1: layer norm
  int dtype;
  int64_t T, D;
  void *Y, *Z;   // T x D
  int8_t* C;     // instead of Z: T x D codes
  float* cs;     // and T scales
};
constexpr int64_t kNormMaxD = 32768;
cudaError_t norm_residual_launch(const NormResidual& p, cudaStream_t stream);
struct NormBackward {
  const void *dY, *dZ, *Y, *H;  // dY or dZ may be null (zero); H null: no block output
  int64_t lddy, lddz, ldy, ldh;
  const float *post, *post_bias;
  const void* gate;
  int64_t ldg, groups;
  const float* pre;
  float alpha, eps;
  int layer, dtype;
  int64_t T, D;
  void *dX, *dH;                                        // T x D
  float *dpost, *dpost_bias, *dgate, *dpre, *dpre_bias;  // D (dgate: groups x D), or null
};
size_t norm_backward_workspace_bytes(int64_t T, int64_t D, int64_t groups);
cudaError_t norm_backward_launch(const NormBackward& p, void* ws, cudaStream_t stream);

// cross_entropy.cu
struct CrossEntropy {
  const void *H, *W;  // T x D hidden states, V x D output embedding
  int64_t ldh, ldw;
  int dtype;  // kF16 or kBF16
  const int64_t* target;
  int64_t T, D, V;
  float *loss, *lse;
  const float* coef;  // T, or null: 1 / (number of tokens with a target)
  void *dH, *dW;      // null: loss only
};
// copies: with room for aligned copies of H and W, which
// cross_entropy_needs_copies() tells the need of.
size_t cross_entropy_workspace_bytes(int64_t T, int64_t D, int64_t V, bool grad, bool copies);
bool cross_entropy_needs_copies(const CrossEntropy& p);
cudaError_t cross_entropy_launch(const CrossEntropy& p, void* ws, int32_t* status_dev, cudaStream_t stream);

}  // namespace bakron
