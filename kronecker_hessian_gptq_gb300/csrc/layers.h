// layers.h -- the layer operators' launch functions (declared to callers in
// bakron.h, arguments checked in abi_layers.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "bakron.h"

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

// head_norm.cu
struct HeadSide {  // queries or keys
  const void* x;   // T x heads x D
  int64_t x_token, x_head;  // strides in elements
  const void* dy;  // backward: the result's gradient
  int64_t dy_token, dy_head;
  const float* w;  // D, or null: no norm
  void* y;         // T x heads x D, dense: the result, or the gradient of x
  float* dw;       // D, or null
  int heads;       // 0: not there
};
struct HeadNorm {
  HeadSide side[2];
  const int64_t* positions;  // T
  const double* freqs;       // half
  int half;                  // pairs that are turned
  int neighbours;
  float eps;
  int dtype;
  int64_t T;
  int D;
};
constexpr int kHeadMaxD = 1024;
cudaError_t head_norm_launch(const HeadNorm& p, cudaStream_t stream);
size_t head_norm_backward_workspace_bytes(int64_t T, int64_t D);
cudaError_t head_norm_backward_launch(const HeadNorm& p, void* ws, cudaStream_t stream);

// adamw.cu
struct Adamw {
  bool eight;
  double lr, scale, b1, b2, eps, decay;
  int64_t step;
  const float *lr_dev, *scale_dev;  // null: the numbers above
  const int64_t* step_dev;
  const int32_t* skip;  // or null
  uint64_t seed;
};
size_t adamw_workspace_bytes();
// Whether nothing that is written, parameter, state, scales (of states in 8 bits) or copy, is in the list twice.
bool adamw_all_different(const bakron_adamw_tensor* tensors, int64_t count, bool eight);
cudaError_t adamw_launch(const Adamw& a, const bakron_adamw_tensor* tensors, int64_t count, void* ws, int32_t* status,
                         cudaStream_t stream);

// fp8_quantize.cu
struct Fp8Codes {
  const void* X;  // rows x cols
  int dtype;
  int64_t rows, cols, ldx;
  // Codes with a scale for each 128 of a row, of a column, or 128 x 128; null: not wanted.
  uint8_t *along, *down, *whole;
  int64_t ld_along, ld_down, ld_whole;
  float *along_scales, *down_scales, *whole_scales;
  int64_t along_row, along_col;  // strides of along_scales
  int64_t down_pitch, whole_row;
  float* sums;  // of the columns of each 128 rows, rows of down_pitch; or null
  void* clear;  // words set to 0 by the same launch
  int64_t clear_words;
};
// other: a second matrix of the same type in the same launch, or null.
cudaError_t fp8_codes_launch(const Fp8Codes& q, const Fp8Codes* other, cudaStream_t stream);
cudaError_t fp8_column_sums_launch(const float* parts, int64_t rows, int64_t pitch, int64_t cols, float* out, cudaStream_t stream);

// fp8_matmul.cu
struct Fp8Matmul {
  const void* X;          // T x K values of x_dtype, or e4m3 codes with x_scales
  const float* x_scales;  // T x ceil(K / 128), or null
  int x_dtype;
  int64_t ldx;
  const uint8_t* V;  // N x K codes
  int64_t ldv;
  const float* scales;  // ceil(N / 128) x ceil(K / 128)
  const float* bias;    // N, or null
  int64_t T, K, N;
  void* Y;
  int y_dtype;
};
// fp8_rows.cu: few tokens, without a workspace.
bool fp8_few_tokens(int64_t T, int64_t K, int64_t N);
cudaError_t fp8_rows(const Fp8Matmul& p, int32_t* status_dev, cudaStream_t stream);

size_t fp8_matmul_workspace_bytes(int64_t T, int64_t K, int64_t N, bool copies);
bool fp8_matmul_needs_copies(const Fp8Matmul& p);
cudaError_t fp8_matmul_launch(const Fp8Matmul& p, void* ws, int32_t* status_dev, cudaStream_t stream);
struct Fp8Backward {
  const void *dY, *X;  // T x N, T x K
  int64_t lddy, ldx;
  int dtype;
  const uint8_t* V;
  int64_t ldv;
  const float* scales;
  int64_t T, K, N;
  void *dX, *dW;  // T x K, N x K; or null
  float* dbias;   // N, or null
};
size_t fp8_backward_workspace_bytes(int64_t T, int64_t K, int64_t N, bool dX, bool dW, bool dbias, bool copies);
bool fp8_backward_needs_copies(const Fp8Backward& p);
cudaError_t fp8_backward_launch(const Fp8Backward& p, void* ws, int32_t* status_dev, cudaStream_t stream);

}  // namespace bakron
