// fp8_rows.cuh -- the product of e4m3 codes for one to four tokens, as fast as
// the weights can be read:
//     Y[t, o] = sum over blocks b of sx[t, b] sw[o / 128, b] sum_{k in b} cx[t, k] cw[o, k] + bias[o].
//
// Every block quantizes the tokens for itself, into shared memory (as fp32
// numbers, which hold codes exactly), while its first weights are on their way:
// one launch in place of two.  A warp takes two outputs at a time, or half, a
// quarter or an eighth of K for them where there are few; a lane 16 codes of every
// 512, all of one block of 128, whose 16 products it sums in fp32 and scales.
// Chunks of 512 codes, with their scales, are on their way four ahead, from one
// pair of outputs into the next.  The sums of lanes and warps are joined in a
// fixed order.
#pragma once

#include <algorithm>
#include <cstdint>

#include "fp8_codes.cuh"
#include "layers.h"

namespace bakron {

constexpr int kRowThreads = 256;
constexpr int kRowOutputs = 2;  // of a warp
constexpr int kRowAhead = 4;    // chunks of 512 codes on their way
constexpr int kRowTokens = 4;
constexpr size_t kRowSmem = 96 * 1024;

constexpr int kRowBlocks = 2 * 152;  // as many as the SMs hold at a time

inline int64_t row_chunks(int64_t K) { return (K + 511) / 512; }
inline size_t row_smem(int64_t T, int64_t K) {
  return (size_t)T * row_chunks(K) * (512 + 4) * 4 + kRowThreads / 32 * kRowOutputs * kRowTokens * 4;
}

// The numbers of 16 codes.
__device__ __forceinline__ void open_codes16(const uint4& u, float (&v)[16]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
// 16 codes of a row from its k-th on, zeros behind its end.
__device__ __forceinline__ uint4 row_codes16(const uint8_t* row, int64_t k, int64_t K, bool vec) {
  if (vec && k + 16 <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
  if (k >= K) return make_uint4(0, 0, 0, 0);
  return load_codes(reinterpret_cast<const int8_t*>(row + k), K - k < 16 ? (int)(K - k) : 16);
}

// TX: the type of X, or uint8_t for codes.  share: warps that share two outputs;
// where it is more than one, no warp has two outputs after another.
template <class TX, class TY, int kT>
__global__ void __launch_bounds__(kRowThreads, 2) fp8_rows_kernel(const Fp8Matmul p, int share, bool vec_x, bool vec, int32_t* status) {
  extern __shared__ __align__(16) float row_smem_raw[];
  const int64_t K = p.K, N = p.N, blocks = (K + 127) / 128;
  const int chunks = (int)((K + 511) / 512);
  float* numbers = row_smem_raw;                 // [token][chunk][quarter of 16][lane][4]
  float* scales = numbers + kT * chunks * 512;   // [token][chunk][4]
  float* red = scales + kT * chunks * 4;         // [warp][output][token]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % share, groups = kRowThreads / 32 / share;
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  const uint8_t* V = static_cast<const uint8_t*>(p.V);
  const int64_t stride = (int64_t)gridDim.x * groups * kRowOutputs;  // from a warp's outputs to its next
  int64_t o = ((int64_t)blockIdx.x * groups + warp / share) * kRowOutputs, next = o;
  int ahead = part;  // the chunk of the outputs `next` that is fetched next
  uint4 w[kRowAhead][kRowOutputs];
  float by[kRowAhead];
  auto fetch = [&](uint4 (&to)[kRowOutputs], float& scale) {
    if (next >= N) return;
#pragma unroll
    for (int r = 0; r < kRowOutputs; ++r)
      to[r] = next + r < N ? row_codes16(V + (next + r) * p.ldv, (int64_t)ahead * 512 + lane * 16, K, vec) : make_uint4(0, 0, 0, 0);
    const int64_t b = (int64_t)ahead * 4 + (lane >> 3);  // both outputs are of the same 128
    scale = b < blocks ? p.scales[(next >> 7) * blocks + b] : 0.f;
    ahead += share;
    if (ahead >= chunks) ahead = part, next += stride;
  };
#pragma unroll
  for (int n = 0; n < kRowAhead; ++n) fetch(w[n], by[n]);
  // 16 values a thread; eight threads next to one another hold a block.
  for (int i = threadIdx.x; i < kT * chunks * 32; i += kRowThreads) {
    const int t = i / (chunks * 32), at = i - t * chunks * 32;
    const int64_t k = (int64_t)at * 16;
    float v[16], scale;
    if constexpr (sizeof(TX) == 1) {
      open_codes16(row_codes16(static_cast<const uint8_t*>(p.X) + t * p.ldx, k, K, vec_x), v);
      scale = k < K ? p.x_scales[t * blocks + (k >> 7)] : 0.f;
    } else {
      const TX* x = static_cast<const TX*>(p.X) + t * p.ldx;
      uint32_t top = 0;
      float inv;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float u[8];
        if (vec_x && k + 8 * h + 8 <= K) {
          load_vec<TX, 8>(x + k + 8 * h, u);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = k + 8 * h + e < K ? to_f32<TX>(x[k + 8 * h + e]) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * h + e] = u[e], top = max(top, magnitude(u[e]));
      }
      // 32 threads of a warp take 32 places of one token: chunks * 32 is a multiple of 32.
#pragma unroll
      for (int o = 4; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      block_scale(top, scale, inv);
      uint4 c;
      float lo[8], hi[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) lo[e] = v[e], hi[e] = v[8 + e];
      const uint2 a = fp8_codes8(lo, inv), b = fp8_codes8(hi, inv);
      c = make_uint4(a.x, a.y, b.x, b.y);
      open_codes16(c, v);
    }
    const int l = at & 31;
    float4* to = reinterpret_cast<float4*>(numbers + (t * chunks + (at >> 5)) * 512) + l;
#pragma unroll
    for (int e = 0; e < 4; ++e) to[32 * e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
    if ((l & 7) == 0) scales[(t * chunks + (at >> 5)) * 4 + (l >> 3)] = scale;
  }
  __syncthreads();
  float acc[kRowOutputs][kT] = {};
  int chunk = part;
  while (o < N) {
#pragma unroll
    for (int n = 0; n < kRowAhead; ++n) {
      if (o >= N) break;
      float v[kRowOutputs][16];
#pragma unroll
      for (int r = 0; r < kRowOutputs; ++r) open_codes16(w[n][r], v[r]);
      const float scale = by[n];
      fetch(w[n], by[n]);
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        const float4* x = reinterpret_cast<const float4*>(numbers + (t * chunks + chunk) * 512) + lane;
        float dot[kRowOutputs] = {};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 f = x[32 * e];
#pragma unroll
          for (int r = 0; r < kRowOutputs; ++r)
            dot[r] = fmaf(f.w, v[r][4 * e + 3], fmaf(f.z, v[r][4 * e + 2], fmaf(f.y, v[r][4 * e + 1], fmaf(f.x, v[r][4 * e], dot[r]))));
        }
        const float both = scales[(t * chunks + chunk) * 4 + (lane >> 3)] * scale;
#pragma unroll
        for (int r = 0; r < kRowOutputs; ++r) acc[r][t] = fmaf(dot[r], both, acc[r][t]);
      }
      chunk += share;
      if (chunk < chunks) continue;
      // The outputs are done, or this warp's part of them.
#pragma unroll
      for (int r = 0; r < kRowOutputs; ++r)
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          const float sum = warp_reduce(acc[r][t], SumOp());
          acc[r][t] = 0.f;
          if (lane == 0 && share > 1)
            red[(warp * kRowOutputs + r) * kT + t] = sum;
          else if (lane == 0 && o + r < N)
            static_cast<TY*>(p.Y)[t * N + o + r] = from_f32<TY>(p.bias ? sum + p.bias[o + r] : sum);
        }
      chunk = part;
      o += stride;
    }
  }
  if (share == 1) return;
  __syncthreads();
  // The parts of K in their order.
  for (int i = threadIdx.x; i < groups * kRowOutputs * kT; i += kRowThreads) {
    const int group = i / (kRowOutputs * kT), r = i / kT % kRowOutputs, t = i % kT;
    const int64_t at = ((int64_t)blockIdx.x * groups + group) * kRowOutputs + r;
    if (at >= N) continue;
    float v = 0.f;
    for (int s = 0; s < share; ++s) v += red[((group * share + s) * kRowOutputs + r) * kT + t];
    static_cast<TY*>(p.Y)[t * N + at] = from_f32<TY>(p.bias ? v + p.bias[at] : v);
  }
}

template <class TX, class TY>
cudaError_t fp8_rows_tokens(const Fp8Matmul& p, int32_t* status, cudaStream_t stream) {
  // Few outputs: as many warps for two of them as the SMs hold, up to eight, each with a chunk of 512.
  int share = 1;
  const int64_t pairs = (p.N + kRowOutputs - 1) / kRowOutputs, warps = (int64_t)kRowBlocks * (kRowThreads / 32);
  while (share < 8 && pairs * share * 2 <= warps && share * 2 <= row_chunks(p.K)) share *= 2;
  const int64_t each = kRowThreads / 32 / share;
  const unsigned grid = (unsigned)std::min<int64_t>((pairs + each - 1) / each, share == 1 ? kRowBlocks : pairs);
  const size_t smem = row_smem(p.T, p.K);
  const bool vec = aligned_to(p.V, 16) && p.ldv % 16 == 0;
  const bool vec_x = aligned_to(p.X, 16) && p.ldx % (16 / (int64_t)sizeof(TX)) == 0;
  auto go = [&](auto kernel) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRowSmem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kRowThreads, smem, stream>>>(p, share, vec_x, vec, status);
    return cudaGetLastError();
  };
  switch (p.T) {
    case 1: return go(fp8_rows_kernel<TX, TY, 1>);
    case 2: return go(fp8_rows_kernel<TX, TY, 2>);
    case 3: return go(fp8_rows_kernel<TX, TY, 3>);
    default: return go(fp8_rows_kernel<TX, TY, 4>);
  }
}
template <class TY>
cudaError_t fp8_rows_launch(const Fp8Matmul& p, int32_t* status, cudaStream_t stream) {
  switch (p.x_dtype) {
    case kF32: return fp8_rows_tokens<float, TY>(p, status, stream);
    case kF16: return fp8_rows_tokens<__half, TY>(p, status, stream);
    case kBF16: return fp8_rows_tokens<__nv_bfloat16, TY>(p, status, stream);
    default: return fp8_rows_tokens<uint8_t, TY>(p, status, stream);
  }
}

}  // namespace bakron
