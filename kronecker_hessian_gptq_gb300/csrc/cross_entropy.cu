// cross_entropy.cu -- softmax cross entropy of a large vocabulary without
// keeping the logits, and its gradients.
//
//     x = H W^T,  lse_t = log sum_v exp(x_tv),  loss_t = lse_t - x_t,y(t),
//     G_tv = c_t (exp(x_tv - lse_t) - [v = y(t)]),  dH = G W,  dW = G^T H
//
// for hidden states H (T x D), output embedding W (V x D) and targets y; a
// token with a negative target has loss 0 and c_t = 0.
#include <algorithm>

#include "bakron.h"
#include "elem.cuh"
#include "layers.h"
#include "tile_product.cuh"

namespace bakron {
namespace {

// c_t of every token, and the status word: one block.
__global__ void __launch_bounds__(1024) coefficients_kernel(const int64_t* target, int64_t T, int64_t V, const float* given,
                                                            float* coef, int32_t* status) {
  __shared__ int with, bad;
  if (threadIdx.x == 0) with = bad = 0;
  __syncthreads();
  int n = 0, wrong = 0;
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    if (target[t] >= V) wrong = 1;
    if (target[t] >= 0 && target[t] < V) ++n;
  }
  if (n) atomicAdd(&with, n);
  if (wrong) atomicOr(&bad, 1);
  __syncthreads();
  if (threadIdx.x == 0) *status = bad ? BAKRON_DEV_BAD_TARGET : 0;
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    const bool has = target[t] >= 0 && target[t] < V;
    coef[t] = has ? (given ? given[t] : 1.f / (float)with) : 0.f;
  }
}

template <class T>
struct Rows {
  const T* p;
  int64_t ld;
  __device__ float operator()(int64_t r, int64_t c) const { return to_f32<T>(p[r * ld + c]); }
};
template <class T>
struct RowsT {
  const T* p;
  int64_t ld;
  __device__ float operator()(int64_t c, int64_t r) const { return to_f32<T>(p[r * ld + c]); }
};
struct Put {
  float* p;
  int64_t ld;
  __device__ void operator()(int64_t r, int64_t c, float v) const { p[r * ld + c] = v; }
};
struct Add {
  float* p;
  int64_t ld;
  __device__ void operator()(int64_t r, int64_t c, float v) const { p[r * ld + c] += v; }
};
template <class T>
struct PutAs {
  T* p;
  int64_t ld;
  __device__ void operator()(int64_t r, int64_t c, float v) const { p[r * ld + c] = from_f32<T>(v); }
};

// One block for each token: lse and loss of its logits, which become G.
__global__ void __launch_bounds__(256) softmax_kernel(float* x, int64_t V, const int64_t* target, const float* coef,
                                                      float* loss, float* lse, bool grad) {
  __shared__ float red[32];
  float* row = x + (int64_t)blockIdx.x * V;
  const int64_t y = target[blockIdx.x];
  const bool has = y >= 0 && y < V;
  float top = -INFINITY;
  for (int64_t v = threadIdx.x; v < V; v += 256) top = fmaxf(top, row[v]);
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = top;
  __syncthreads();
  for (int w = 0; w < 8; ++w) top = fmaxf(top, red[w]);
  float s[1] = {0.f};
  for (int64_t v = threadIdx.x; v < V; v += 256) s[0] += expf(row[v] - top);
  block_reduce<1>(s, red, SumOp());
  const float l = top + logf(s[0]);
  if (threadIdx.x == 0) {
    lse[blockIdx.x] = l;
    loss[blockIdx.x] = has ? l - row[y] : 0.f;
  }
  if (!grad) return;
  __syncthreads();
  const float c = coef[blockIdx.x];
  for (int64_t v = threadIdx.x; v < V; v += 256) row[v] = c * (expf(row[v] - l) - (has && v == y ? 1.f : 0.f));
}

template <class T>
__global__ void convert_kernel(const float* x, T* y, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    y[i] = from_f32<T>(x[i]);
}

constexpr int64_t kPiece = 256;  // tokens whose logits are held at once

size_t up(size_t x) { return (x + 255) / 256 * 256; }

template <class T>
cudaError_t run(const CrossEntropy& p, void* ws, int32_t* status, cudaStream_t stream) {
  char* at = static_cast<char*>(ws);
  float* coef = reinterpret_cast<float*>(at);
  at += up(p.T * 4);
  float* x = reinterpret_cast<float*>(at);
  at += up(std::min(kPiece, p.T) * p.V * 4);
  float* dw = reinterpret_cast<float*>(at);
  const bool grad = p.dH != nullptr;
  coefficients_kernel<<<1, 1024, 0, stream>>>(p.target, p.T, p.V, p.coef, coef, status);
  if (grad) {
    cudaError_t e = cudaMemsetAsync(dw, 0, p.V * p.D * 4, stream);
    if (e != cudaSuccess) return e;
  }
  for (int64_t t = 0; t < p.T; t += kPiece) {
    const int64_t n = std::min(kPiece, p.T - t);
    const T* H = static_cast<const T*>(p.H) + t * p.ldh;
    const T* W = static_cast<const T*>(p.W);
    auto grid = [](int64_t m, int64_t k) { return dim3((unsigned)((k + 63) / 64), (unsigned)((m + 63) / 64)); };
    tile_product_kernel<float><<<grid(n, p.V), 256, 0, stream>>>(n, p.V, p.D, Rows<T>{H, p.ldh}, RowsT<T>{W, p.ldw}, Put{x, p.V});
    softmax_kernel<<<(unsigned)n, 256, 0, stream>>>(x, p.V, p.target + t, coef + t, p.loss + t, p.lse + t, grad);
    if (!grad) continue;
    tile_product_kernel<float><<<grid(n, p.D), 256, 0, stream>>>(n, p.D, p.V, Rows<float>{x, p.V}, Rows<T>{W, p.ldw},
                                                                 PutAs<T>{static_cast<T*>(p.dH) + t * p.D, p.D});
    tile_product_kernel<float><<<grid(p.V, p.D), 256, 0, stream>>>(p.V, p.D, n, RowsT<float>{x, p.V}, Rows<T>{H, p.ldh}, Add{dw, p.D});
  }
  if (grad) convert_kernel<T><<<1024, 256, 0, stream>>>(dw, static_cast<T*>(p.dW), p.V * p.D);
  return cudaGetLastError();
}

}  // namespace

size_t cross_entropy_workspace_bytes(int64_t T, int64_t D, int64_t V, bool grad) {
  return up(T * 4) + up(std::min(kPiece, T) * V * 4) + (grad ? (size_t)V * D * 4 : 0);
}

cudaError_t cross_entropy_launch(const CrossEntropy& p, void* ws, int32_t* status_dev, cudaStream_t stream) {
  return p.dtype == kF16 ? run<__half>(p, ws, status_dev, stream) : run<__nv_bfloat16>(p, ws, status_dev, stream);
}

}  // namespace bakron
