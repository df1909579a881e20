// abi_layers.cu -- the extern "C" entry points of the layer operators
// (declared in bakron.h): arguments are checked on the host before anything
// is enqueued.
#include <initializer_list>

#include "bakron.h"
#include "internal.h"
#include "layers.h"

namespace {

using bakron::aligned_to;

int from_cuda(cudaError_t e) { return e == cudaSuccess ? BAKRON_OK : BAKRON_ERR_CUDA; }
bool float_type(int dtype) { return dtype == BAKRON_F32 || dtype == BAKRON_F16 || dtype == BAKRON_BF16; }
bool on_element(const void* p, int dtype) { return aligned_to(p, bakron::elem_size(dtype)); }
// Arrays of 32-bit elements (null: not there).
bool on_words(std::initializer_list<const void*> arrays) {
  for (const void* p : arrays)
    if (!aligned_to(p, 4)) return false;
  return true;
}
bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && aligned_to(ws, bakron::kAlign) && have >= need);
}

constexpr int64_t kMaxRows = (int64_t)1 << 31;  // tokens: one thread block each in x
constexpr int64_t kMaxD = (int64_t)1 << 20, kMaxV = (int64_t)1 << 24;
constexpr int64_t kMaxK = (int64_t)1 << 17;     // 2^14 K stays below 2^31: 32-bit sums are exact

}  // namespace

extern "C" {

int bakron_quantize_tokens(const void* X, int dtype, int64_t T, int64_t K, int64_t ldx, int8_t* codes, float* scales,
                           void* stream) {
  if (!X || !codes || !scales || !float_type(dtype) || T < 1 || T >= kMaxRows || K < 1 || K >= kMaxRows || ldx < K ||
      !on_element(X, dtype) || !aligned_to(scales, 4) || X == (const void*)codes)
    return BAKRON_ERR_INVALID_ARG;
  return from_cuda(bakron::quantize_tokens_launch(X, dtype, T, K, ldx, codes, K, scales, (cudaStream_t)stream));
}

size_t bakron_int8_matmul_workspace_size(int64_t T, int64_t K, int64_t N, int copies) {
  if (T < 1 || T >= kMaxRows || K < 1 || K >= kMaxK || N < 1 || N >= kMaxRows) return 0;
  return bakron::int8_matmul_workspace_bytes(T, K, N, copies != 0);
}

int bakron_int8_matmul(const void* X, int x_dtype, int64_t ldx, const float* x_scales, const int8_t* codes, int64_t ldc,
                       const float* scales, const float* bias, int64_t T, int64_t K, int64_t N, void* Y, int y_dtype,
                       void* ws, size_t ws_bytes, int32_t* status_dev, void* stream) {
  if (!X || !codes || !scales || !Y || !status_dev) return BAKRON_ERR_INVALID_ARG;
  if (T < 1 || T >= kMaxRows || K < 1 || K >= kMaxK || N < 1 || N >= kMaxRows || ldx < K || ldc < K)
    return BAKRON_ERR_INVALID_ARG;
  if (x_dtype == BAKRON_I8 ? !x_scales : (x_scales || !float_type(x_dtype) || !on_element(X, x_dtype)))
    return BAKRON_ERR_INVALID_ARG;
  if (!on_words({x_scales, scales, bias, status_dev})) return BAKRON_ERR_INVALID_ARG;
  if (!float_type(y_dtype) || !on_element(Y, y_dtype) || Y == X || Y == (const void*)codes) return BAKRON_ERR_INVALID_ARG;
  const bakron::Int8Matmul p{X, x_scales, x_dtype, ldx, codes, ldc, scales, bias, T, K, N, Y, y_dtype, N};
  const bool copies = bakron::int8_matmul_needs_copies(p);
  if (!workspace_ok(ws, ws_bytes, bakron::int8_matmul_workspace_bytes(T, K, N, copies))) return BAKRON_ERR_WORKSPACE;
  return from_cuda(bakron::int8_matmul_launch(p, ws, status_dev, (cudaStream_t)stream));
}

int bakron_norm_residual(const void* X, int64_t ldx, const void* H, int64_t ldh, const float* post,
                         const float* post_bias, const void* gate, int64_t ldg, int64_t groups, const float* pre,
                         const float* pre_bias, float alpha, float eps, int kind, int dtype, int64_t T, int64_t D,
                         void* Y, void* Z, int8_t* codes, float* code_scales, void* stream) {
  if (!X || !Y || !float_type(dtype) || T < 1 || T >= kMaxRows || D < 1 || D > bakron::kNormMaxD || ldx < D ||
      (kind != BAKRON_NORM_RMS && kind != BAKRON_NORM_LAYER) || !(eps >= 0.f))
    return BAKRON_ERR_INVALID_ARG;
  if (H ? ldh < D : (post || post_bias || gate)) return BAKRON_ERR_INVALID_ARG;
  if ((post_bias && !post) || (pre_bias && !pre) || (kind == BAKRON_NORM_RMS && (post_bias || pre_bias)))
    return BAKRON_ERR_INVALID_ARG;
  if (gate && (groups < 1 || T % groups || ldg < D)) return BAKRON_ERR_INVALID_ARG;
  if (pre ? ((Z != nullptr) == (codes != nullptr) || (codes != nullptr) != (code_scales != nullptr))
          : (Z || codes || code_scales))
    return BAKRON_ERR_INVALID_ARG;
  if (!on_element(X, dtype) || !on_element(H, dtype) || !on_element(gate, dtype) || !on_element(Y, dtype) ||
      !on_element(Z, dtype) || !on_words({post, post_bias, pre, pre_bias, code_scales}))
    return BAKRON_ERR_INVALID_ARG;
  if (Z == Y || (Z && (Z == X || Z == H)) || (codes && (codes == X || codes == H || codes == Y)))
    return BAKRON_ERR_INVALID_ARG;
  if ((Y == X && ldx != D) || (H && Y == H && ldh != D)) return BAKRON_ERR_INVALID_ARG;
  bakron::NormResidual p{X,   H,     ldx, ldh,  post,  post_bias, gate, ldg, gate ? groups : 1, pre, pre_bias, alpha,
                         eps, kind, dtype, T, D, Y, Z, codes, code_scales};
  return from_cuda(bakron::norm_residual_launch(p, (cudaStream_t)stream));
}

size_t bakron_norm_residual_backward_workspace_size(int64_t T, int64_t D, int64_t groups) {
  if (T < 1 || T >= kMaxRows || D < 1 || D > bakron::kNormMaxD || groups < 0 || (groups && T % groups)) return 0;
  return bakron::norm_backward_workspace_bytes(T, D, groups);
}

int bakron_norm_residual_backward(const void* dY, int64_t lddy, const void* dZ, int64_t lddz, const void* Y, int64_t ldy,
                                  const void* H, int64_t ldh, const float* post, const float* post_bias,
                                  const void* gate, int64_t ldg, int64_t groups, const float* pre, float alpha, float eps,
                                  int kind, int dtype, int64_t T, int64_t D, void* dX, void* dH, float* dpost,
                                  float* dpost_bias, float* dgate, float* dpre, float* dpre_bias, void* ws,
                                  size_t ws_bytes, void* stream) {
  if (!Y || !dX || (!dY && !dZ) || !float_type(dtype) || T < 1 || T >= kMaxRows || D < 1 || D > bakron::kNormMaxD ||
      ldy < D || (dY && lddy < D) || (dZ && lddz < D) || (kind != BAKRON_NORM_RMS && kind != BAKRON_NORM_LAYER) ||
      !(eps >= 0.f))
    return BAKRON_ERR_INVALID_ARG;
  if (H ? (ldh < D || !dH) : (dH || post || post_bias || gate)) return BAKRON_ERR_INVALID_ARG;
  if ((post_bias && (!post || kind == BAKRON_NORM_RMS)) || (dZ && !pre)) return BAKRON_ERR_INVALID_ARG;
  if ((dpost && !post) || (dpre && !pre) || (dgate && !gate)) return BAKRON_ERR_INVALID_ARG;
  // biases are those of layer norms
  if ((dpost_bias && (!post || kind != BAKRON_NORM_LAYER)) || (dpre_bias && (!pre || kind != BAKRON_NORM_LAYER)))
    return BAKRON_ERR_INVALID_ARG;
  if (gate && (groups < 1 || T % groups || ldg < D)) return BAKRON_ERR_INVALID_ARG;
  for (const void* q : {dY, dZ, Y, H, gate, (const void*)dX, (const void*)dH})
    if (!on_element(q, dtype)) return BAKRON_ERR_INVALID_ARG;
  if (!on_words({post, post_bias, pre, dpost, dpost_bias, dgate, dpre, dpre_bias})) return BAKRON_ERR_INVALID_ARG;
  for (const void* q : {Y, H, gate, (const void*)dH})
    if (q && q == dX) return BAKRON_ERR_INVALID_ARG;
  for (const void* q : {dY, dZ, Y, gate})
    if (q && q == dH) return BAKRON_ERR_INVALID_ARG;
  if ((dX == dY && lddy != D) || (dX == dZ && lddz != D) || (H && dH == H && ldh != D)) return BAKRON_ERR_INVALID_ARG;
  const int64_t g = gate ? groups : 0;
  if (!workspace_ok(ws, ws_bytes, bakron::norm_backward_workspace_bytes(T, D, g))) return BAKRON_ERR_WORKSPACE;
  bakron::NormBackward p{dY,  dZ,  Y,    H,     lddy, lddz, ldy, ldh,   post,       post_bias, gate, ldg, g, pre,
                         alpha, eps, kind, dtype, T,    D,    dX,  dH, dpost, dpost_bias, dgate,     dpre, dpre_bias};
  return from_cuda(bakron::norm_backward_launch(p, ws, (cudaStream_t)stream));
}

size_t bakron_linear_cross_entropy_workspace_size(int64_t T, int64_t D, int64_t V, int grad, int copies) {
  if (T < 1 || T >= kMaxRows || D < 1 || D > kMaxD || V < 1 || V > kMaxV) return 0;
  return bakron::cross_entropy_workspace_bytes(T, D, V, grad != 0, copies != 0);
}

static int cross_entropy(const void* H, int64_t ldh, const void* W, int64_t ldw, int dtype, const int64_t* targets,
                         const float* coef, int64_t T, int64_t D, int64_t V, float* loss, float* lse, void* dH, void* dW,
                         void* ws, size_t ws_bytes, int32_t* status_dev, void* stream) {
  if (!H || !W || !targets || !loss || !lse || !status_dev || (dtype != BAKRON_F16 && dtype != BAKRON_BF16))
    return BAKRON_ERR_INVALID_ARG;
  if (T < 1 || T >= kMaxRows || D < 1 || D > kMaxD || V < 1 || V > kMaxV || ldh < D || ldw < D)
    return BAKRON_ERR_INVALID_ARG;
  if (!on_element(H, dtype) || !on_element(W, dtype) || !aligned_to(targets, 8) || loss == lse ||
      !on_words({coef, loss, lse, status_dev}))
    return BAKRON_ERR_INVALID_ARG;
  const bakron::CrossEntropy p{H, W, ldh, ldw, dtype, targets, T, D, V, loss, lse, coef, dH, dW};
  const bool copies = bakron::cross_entropy_needs_copies(p);
  if (!workspace_ok(ws, ws_bytes, bakron::cross_entropy_workspace_bytes(T, D, V, dH != nullptr, copies)))
    return BAKRON_ERR_WORKSPACE;
  return from_cuda(bakron::cross_entropy_launch(p, ws, status_dev, (cudaStream_t)stream));
}

int bakron_linear_cross_entropy(const void* H, int64_t ldh, const void* W, int64_t ldw, int dtype, const int64_t* targets,
                                int64_t T, int64_t D, int64_t V, float* loss, float* lse, void* ws, size_t ws_bytes,
                                int32_t* status_dev, void* stream) {
  return cross_entropy(H, ldh, W, ldw, dtype, targets, nullptr, T, D, V, loss, lse, nullptr, nullptr, ws, ws_bytes,
                       status_dev, stream);
}

int bakron_linear_cross_entropy_grad(const void* H, int64_t ldh, const void* W, int64_t ldw, int dtype,
                                     const int64_t* targets, const float* coef, int64_t T, int64_t D, int64_t V,
                                     float* loss, float* lse, void* dH, void* dW, void* ws, size_t ws_bytes,
                                     int32_t* status_dev, void* stream) {
  if (!dH || !dW || dH == dW || dH == H || dW == W || dH == W || dW == H) return BAKRON_ERR_INVALID_ARG;
  if (!on_element(dH, dtype) || !on_element(dW, dtype)) return BAKRON_ERR_INVALID_ARG;
  return cross_entropy(H, ldh, W, ldw, dtype, targets, coef, T, D, V, loss, lse, dH, dW, ws, ws_bytes, status_dev, stream);
}

}  // extern "C"
