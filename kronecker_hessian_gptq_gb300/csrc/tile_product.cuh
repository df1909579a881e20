// tile_product.cuh -- C = A B over functors, one 64 x 64 tile for each block
// of 256 threads, 4 x 4 entries for each thread.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace bakron {

template <class Acc, class LoadA, class LoadB, class Put>
__global__ void __launch_bounds__(256) tile_product_kernel(int64_t M, int64_t N, int64_t K, LoadA la, LoadB lb, Put put) {
  __shared__ Acc as[16][65], bs[16][65];
  const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  Acc acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int k = i % 16, r = i / 16;
      as[k][r] = (m0 + r < M && k0 + k < K) ? la(m0 + r, k0 + k) : Acc(0);
      bs[k][r] = (n0 + r < N && k0 + k < K) ? lb(k0 + k, n0 + r) : Acc(0);
    }
    __syncthreads();
    for (int k = 0; k < 16; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] += as[k][ty + 16 * i] * bs[k][tx + 16 * j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j)
      if (m0 + ty + 16 * i < M && n0 + tx + 16 * j < N) put(m0 + ty + 16 * i, n0 + tx + 16 * j, acc[i][j]);
}

}  // namespace bakron
