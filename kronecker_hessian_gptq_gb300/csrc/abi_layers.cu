// abi_layers.cu -- the extern "C" entry points of the layer operators
// (declared in bakron.h): arguments are checked on the host before anything
// is enqueued.
#include <initializer_list>

#include "bakron.h"
#include "internal.h"
#include "layers.h"

namespace {

using bakron::aligned_to;

// An error is reported once: what is left of it would be the next launch's.
int from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return BAKRON_OK;
  (void)cudaGetLastError();
  return BAKRON_ERR_CUDA;
}
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
constexpr int64_t kMaxFp8T = (int64_t)1 << 24, kMaxFp8 = (int64_t)1 << 20;
constexpr int64_t kMaxHeads = 65535;
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

int bakron_quantize_blocks(const void* X, int dtype, int64_t T, int64_t K, int64_t ldx, int rows, int cols, uint8_t* codes,
                           int64_t ldc, float* scales, void* stream) {
  if (!X || !codes || !scales || !float_type(dtype) || T < 1 || T >= kMaxRows || K < 1 || K >= kMaxRows || ldx < K || ldc < K ||
      !on_element(X, dtype) || !aligned_to(scales, 4) || X == (const void*)codes)
    return BAKRON_ERR_INVALID_ARG;
  const int64_t across = (K + 127) / 128;
  bakron::Fp8Codes q = {};
  q.X = X, q.dtype = dtype, q.rows = T, q.cols = K, q.ldx = ldx;
  if (rows == 1 && cols == 128)
    q.along = codes, q.ld_along = ldc, q.along_scales = scales, q.along_row = across, q.along_col = 1;
  else if (rows == 128 && cols == 128)
    q.whole = codes, q.ld_whole = ldc, q.whole_scales = scales, q.whole_row = across;
  else if (rows == 128 && cols == 1)
    q.down = codes, q.ld_down = ldc, q.down_scales = scales, q.down_pitch = K;
  else
    return BAKRON_ERR_INVALID_ARG;
  return from_cuda(bakron::fp8_codes_launch(q, nullptr, (cudaStream_t)stream));
}

size_t bakron_fp8_matmul_workspace_size(int64_t T, int64_t K, int64_t N, int x_dtype, int copies) {
  if (T < 1 || T > kMaxFp8T || K < 1 || K > kMaxFp8 || N < 1 || N > kMaxFp8 || (x_dtype != BAKRON_E4M3 && !float_type(x_dtype)))
    return 0;
  return bakron::fp8_matmul_workspace_bytes(T, K, N, copies != 0);
}

int bakron_fp8_matmul(const void* X, int x_dtype, int64_t ldx, const float* x_scales, const uint8_t* codes, int64_t ldc,
                      const float* scales, const float* bias, int64_t T, int64_t K, int64_t N, void* Y, int y_dtype,
                      void* ws, size_t ws_bytes, int32_t* status_dev, void* stream) {
  if (!X || !codes || !scales || !Y || !status_dev) return BAKRON_ERR_INVALID_ARG;
  if (T < 1 || T > kMaxFp8T || K < 1 || K > kMaxFp8 || N < 1 || N > kMaxFp8 || ldx < K || ldc < K) return BAKRON_ERR_INVALID_ARG;
  if (x_dtype == BAKRON_E4M3 ? !x_scales : (x_scales || !float_type(x_dtype) || !on_element(X, x_dtype)))
    return BAKRON_ERR_INVALID_ARG;
  if (!on_words({x_scales, scales, bias, status_dev})) return BAKRON_ERR_INVALID_ARG;
  if (!float_type(y_dtype) || !on_element(Y, y_dtype) || Y == X || Y == (const void*)codes) return BAKRON_ERR_INVALID_ARG;
  const bakron::Fp8Matmul p{X, x_scales, x_dtype, ldx, codes, ldc, scales, bias, T, K, N, Y, y_dtype};
  const bool copies = bakron::fp8_matmul_needs_copies(p);
  if (!workspace_ok(ws, ws_bytes, bakron::fp8_matmul_workspace_bytes(T, K, N, copies))) return BAKRON_ERR_WORKSPACE;
  return from_cuda(bakron::fp8_matmul_launch(p, ws, status_dev, (cudaStream_t)stream));
}

size_t bakron_fp8_matmul_backward_workspace_size(int64_t T, int64_t K, int64_t N, int want, int copies) {
  if (T < 1 || T > kMaxFp8T || K < 1 || K > kMaxFp8 || N < 1 || N > kMaxFp8) return 0;
  return bakron::fp8_backward_workspace_bytes(T, K, N, want & 1, want & 2, want & 4, copies != 0);
}

int bakron_fp8_matmul_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, int dtype, const uint8_t* codes,
                               int64_t ldc, const float* scales, int64_t T, int64_t K, int64_t N, void* dX, void* dW,
                               float* dbias, void* ws, size_t ws_bytes, int32_t* status_dev, void* stream) {
  if (!dY || !status_dev || (!dX && !dW) || !float_type(dtype)) return BAKRON_ERR_INVALID_ARG;
  if (T < 1 || T > kMaxFp8T || K < 1 || K > kMaxFp8 || N < 1 || N > kMaxFp8 || lddy < N) return BAKRON_ERR_INVALID_ARG;
  if ((dW && (!X || ldx < K)) || (dX && (!codes || !scales || ldc < K))) return BAKRON_ERR_INVALID_ARG;
  for (const void* q : {dY, X, (const void*)dX, (const void*)dW})
    if (!on_element(q, dtype)) return BAKRON_ERR_INVALID_ARG;
  if (!on_words({scales, dbias, status_dev})) return BAKRON_ERR_INVALID_ARG;
  for (const void* q : {dY, X, (const void*)codes, (const void*)dW})
    if (q && q == dX) return BAKRON_ERR_INVALID_ARG;
  for (const void* q : {dY, X, (const void*)codes})
    if (q && q == dW) return BAKRON_ERR_INVALID_ARG;
  const bakron::Fp8Backward p{dY, X, lddy, ldx, dtype, codes, ldc, scales, T, K, N, dX, dW, dbias};
  const bool copies = bakron::fp8_backward_needs_copies(p);
  if (!workspace_ok(ws, ws_bytes, bakron::fp8_backward_workspace_bytes(T, K, N, dX, dW, dbias, copies))) return BAKRON_ERR_WORKSPACE;
  return from_cuda(bakron::fp8_backward_launch(p, ws, status_dev, (cudaStream_t)stream));
}

static bool heads_ok(int64_t Hq, int64_t Hk, const int64_t* positions, const double* freqs, int64_t R, int pairs, float eps,
                     int dtype, int64_t T, int64_t D) {
  return Hq >= 0 && Hq <= kMaxHeads && Hk >= 0 && Hk <= kMaxHeads && Hq + Hk > 0 && float_type(dtype) && T >= 1 && T < kMaxRows &&
         D >= 1 && D <= bakron::kHeadMaxD && R >= 0 && R <= D && R % 2 == 0 && (R == 0 || (positions && freqs)) &&
         aligned_to(positions, 8) && aligned_to(freqs, 8) && eps >= 0.f &&
         (pairs == BAKRON_PAIRS_HALVES || pairs == BAKRON_PAIRS_NEIGHBOURS);
}

int bakron_head_norm_rotary(const void* Q, int64_t q_token, int64_t q_head, int64_t Hq, const void* K, int64_t k_token,
                            int64_t k_head, int64_t Hk, const float* q_weight, const float* k_weight,
                            const int64_t* positions, const double* freqs, int64_t R, int pairs, float eps, int dtype,
                            int64_t T, int64_t D, void* YQ, void* YK, void* stream) {
  if (!heads_ok(Hq, Hk, positions, freqs, R, pairs, eps, dtype, T, D)) return BAKRON_ERR_INVALID_ARG;
  if ((Hq && (!Q || !YQ)) || (Hk && (!K || !YK))) return BAKRON_ERR_INVALID_ARG;
  for (const void* q : {Q, K, (const void*)YQ, (const void*)YK})
    if (!on_element(q, dtype)) return BAKRON_ERR_INVALID_ARG;
  if (!on_words({q_weight, k_weight})) return BAKRON_ERR_INVALID_ARG;
  for (const void* y : {YQ, YK})
    if (y && (y == Q || y == K)) return BAKRON_ERR_INVALID_ARG;
  if (YQ && YQ == YK) return BAKRON_ERR_INVALID_ARG;
  bakron::HeadNorm p = {};
  p.side[0] = bakron::HeadSide{Q, q_token, q_head, nullptr, 0, 0, q_weight, YQ, nullptr, (int)Hq};
  p.side[1] = bakron::HeadSide{K, k_token, k_head, nullptr, 0, 0, k_weight, YK, nullptr, (int)Hk};
  p.positions = positions, p.freqs = freqs, p.half = (int)(R / 2), p.neighbours = pairs == BAKRON_PAIRS_NEIGHBOURS;
  p.eps = eps, p.dtype = dtype, p.T = T, p.D = (int)D;
  return from_cuda(bakron::head_norm_launch(p, (cudaStream_t)stream));
}

size_t bakron_head_norm_rotary_backward_workspace_size(int64_t T, int64_t D) {
  if (T < 1 || T >= kMaxRows || D < 1 || D > bakron::kHeadMaxD) return 0;
  return bakron::head_norm_backward_workspace_bytes(T, D);
}

int bakron_head_norm_rotary_backward(const void* dYQ, int64_t dq_token, int64_t dq_head, const void* dYK, int64_t dk_token,
                                     int64_t dk_head, const void* Q, int64_t q_token, int64_t q_head, int64_t Hq,
                                     const void* K, int64_t k_token, int64_t k_head, int64_t Hk, const float* q_weight,
                                     const float* k_weight, const int64_t* positions, const double* freqs, int64_t R,
                                     int pairs, float eps, int dtype, int64_t T, int64_t D, void* dQ, void* dK,
                                     float* dq_weight, float* dk_weight, void* ws, size_t ws_bytes, void* stream) {
  if (!heads_ok(Hq, Hk, positions, freqs, R, pairs, eps, dtype, T, D)) return BAKRON_ERR_INVALID_ARG;
  if ((Hq && (!dYQ || !dQ)) || (Hk && (!dYK || !dK))) return BAKRON_ERR_INVALID_ARG;
  if ((Hq && q_weight && !Q) || (Hk && k_weight && !K) || (dq_weight && !q_weight) || (dk_weight && !k_weight))
    return BAKRON_ERR_INVALID_ARG;
  for (const void* q : {dYQ, dYK, Q, K, (const void*)dQ, (const void*)dK})
    if (!on_element(q, dtype)) return BAKRON_ERR_INVALID_ARG;
  if (!on_words({q_weight, k_weight, dq_weight, dk_weight})) return BAKRON_ERR_INVALID_ARG;
  for (const void* y : {dQ, dK})
    for (const void* q : {dYQ, dYK, Q, K})
      if (y && y == q) return BAKRON_ERR_INVALID_ARG;
  if (dQ && dQ == dK) return BAKRON_ERR_INVALID_ARG;
  if (!workspace_ok(ws, ws_bytes, bakron::head_norm_backward_workspace_bytes(T, D))) return BAKRON_ERR_WORKSPACE;
  bakron::HeadNorm p = {};
  p.side[0] = bakron::HeadSide{Q, q_token, q_head, dYQ, dq_token, dq_head, q_weight, dQ, dq_weight, (int)Hq};
  p.side[1] = bakron::HeadSide{K, k_token, k_head, dYK, dk_token, dk_head, k_weight, dK, dk_weight, (int)Hk};
  p.positions = positions, p.freqs = freqs, p.half = (int)(R / 2), p.neighbours = pairs == BAKRON_PAIRS_NEIGHBOURS;
  p.eps = eps, p.dtype = dtype, p.T = T, p.D = (int)D;
  return from_cuda(bakron::head_norm_backward_launch(p, ws, (cudaStream_t)stream));
}

size_t bakron_adamw_workspace_size(void) { return bakron::adamw_workspace_bytes(); }

int bakron_adamw(const bakron_adamw_tensor* tensors, int64_t count, int bits, double lr, const float* lr_dev, int64_t step,
                 const int64_t* step_dev, double beta1, double beta2, double eps, double weight_decay, double grad_scale,
                 const float* grad_scale_dev, const int32_t* skip, uint64_t seed, void* ws, size_t ws_bytes,
                 int32_t* status_dev, void* stream) {
  if (count < 0 || (count && !tensors) || (bits != 8 && bits != 32) || (!step_dev && step < 1) || !status_dev ||
      !(beta1 >= 0. && beta1 < 1.) || !(beta2 >= 0. && beta2 < 1.) || !(eps >= 0.) || lr != lr || weight_decay != weight_decay ||
      grad_scale != grad_scale || !on_words({lr_dev, grad_scale_dev, skip, status_dev}) || !aligned_to(step_dev, 8))
    return BAKRON_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    const bakron_adamw_tensor& t = tensors[i];
    if (t.n < 0) return BAKRON_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || !float_type(t.param_dtype) || !float_type(t.grad_dtype) ||
        !on_element(t.param, t.param_dtype) || !on_element(t.grad, t.grad_dtype))
      return BAKRON_ERR_INVALID_ARG;
    if (t.copy && ((t.copy_dtype != BAKRON_F16 && t.copy_dtype != BAKRON_BF16) || !on_element(t.copy, t.copy_dtype)))
      return BAKRON_ERR_INVALID_ARG;
    if (bits == 8 ? (!t.m_scales || !t.v_scales || !on_words({t.m_scales, t.v_scales})) : !on_words({t.m, t.v}))
      return BAKRON_ERR_INVALID_ARG;
    if (t.param == t.grad || t.param == t.m || t.param == t.v || t.m == t.v || t.copy == t.param || t.grad == t.m || t.grad == t.v)
      return BAKRON_ERR_INVALID_ARG;
  }
  if (!bakron::adamw_all_different(tensors, count, bits == 8)) return BAKRON_ERR_INVALID_ARG;
  if (!workspace_ok(ws, ws_bytes, bakron::adamw_workspace_bytes())) return BAKRON_ERR_WORKSPACE;
  const bakron::Adamw a{bits == 8, lr, grad_scale, beta1, beta2, eps, weight_decay, step, lr_dev, grad_scale_dev, step_dev, skip, seed};
  return from_cuda(bakron::adamw_launch(a, tensors, count, ws, status_dev, (cudaStream_t)stream));
}

}  // extern "C"
