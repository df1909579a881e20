// fp8_quantize.cu -- codes in e4m3 with a scale for each 128 values of a row,
// 128 of a column, or block of 128 x 128 (see fp8_codes.cuh).
//
// Bound by memory: values are read once, into registers, their maxima taken
// there, and the codes written.  Along rows a warp takes 512 values of a row.
// Otherwise a block takes 128 x 128 values, 4 x 8 a thread; one read of them
// gives the codes along rows, the codes along columns and the columns' sums
// (what the backward pass of a product needs of its output's gradient).
// 4096 x 4096 in bf16: 12.9 us along rows, 15.0 along columns, 14.2 in blocks (3.4
// to 3.9 TB/s); with maxima of single fp32 magnitudes 14.3, 22 and 20.5.
#include <algorithm>
#include <cstring>

#include "fp8_codes.cuh"
#include "layers.h"

namespace bakron {
namespace {

constexpr int kCodeThreads = 256;
constexpr int kTileThreads = 512;

__device__ __forceinline__ void put_codes8(uint8_t* c, int64_t i, int64_t n, bool vec, const uint2& w) {
  if (vec && i + 8 <= n) {
    *reinterpret_cast<uint2*>(c + i) = w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) c[i + k] = (uint8_t)((k < 4 ? w.x : w.y) >> (8 * (k % 4)));
  }
}

// What is cleared beside the codes, for the kernel that follows.
struct Clear {
  uint32_t* word;
  int words;
};
__device__ __forceinline__ void clear_words(const Clear& c) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < c.words; i += (int64_t)gridDim.x * blockDim.x)
    c.word[i] = 0;
}

// Eight values as they lie in registers: four words of two 16-bit ones, or eight.
// Magnitudes of floats order as their bits do, with infinity and then NaN above
// all, so maxima are taken of the bits, two 16-bit ones at a time.
template <class T>
struct Eight {
  static constexpr bool kPairs = sizeof(T) == 2;
  static constexpr int kWords = kPairs ? 4 : 8;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* x, int64_t i, int64_t n, bool vec) {
    if (vec && i + 8 <= n) {
#pragma unroll
      for (int k = 0; k < kWords / 4; ++k) {
        const uint4 u = reinterpret_cast<const uint4*>(x + i)[k];
        w[4 * k] = u.x, w[4 * k + 1] = u.y, w[4 * k + 2] = u.z, w[4 * k + 3] = u.w;
      }
    } else if constexpr (kPairs) {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(x);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = (i + 2 * k < n ? (uint32_t)h[i + 2 * k] : 0u) | (i + 2 * k + 1 < n ? (uint32_t)h[i + 2 * k + 1] << 16 : 0u);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = i + k < n ? __float_as_uint(x[i + k]) : 0u;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = 0;
  }
  static __device__ __forceinline__ uint32_t size_of(uint32_t word) { return word & (kPairs ? 0x7fff7fffu : 0x7fffffffu); }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return kPairs ? __vmaxu2(a, b) : max(a, b); }
  // The fp32 magnitude, in bits, of one 16-bit magnitude or of a word.
  static __device__ __forceinline__ uint32_t as_fp32(uint32_t bits) {
    if constexpr (kPairs) {
      const uint16_t h = (uint16_t)bits;
      T t;
      memcpy(&t, &h, 2);
      return __float_as_uint(to_f32<T>(t));
    } else {
      return bits;
    }
  }
  // ... and of the larger one of a word.
  static __device__ __forceinline__ uint32_t top_of(uint32_t word) { return as_fp32(kPairs ? max(word & 0xffffu, word >> 16) : word); }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = size_of(w[0]);
#pragma unroll
    for (int k = 1; k < kWords; ++k) t = larger(t, size_of(w[k]));
    return t;
  }
  // The values, or zeros where `keep` (bits) is 0: a block without a reciprocal may hold what is not finite.
  __device__ __forceinline__ void open(const uint32_t (&keep)[kWords], float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const uint32_t x = w[k] & keep[k];
      if constexpr (kPairs) {
        T t[2];
        memcpy(t, &x, 4);
        v[2 * k] = to_f32<T>(t[0]), v[2 * k + 1] = to_f32<T>(t[1]);
      } else {
        v[k] = __uint_as_float(x);
      }
    }
  }
  __device__ __forceinline__ void open(bool keep, float (&v)[8]) const {
    uint32_t all[kWords];
#pragma unroll
    for (int k = 0; k < kWords; ++k) all[k] = keep ? 0xffffffffu : 0u;
    open(all, v);
  }
};
__device__ __forceinline__ uint32_t codes2(float a, float b, float inv_a, float inv_b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a * inv_a, b * inv_b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const float (&inv)[8]) {
  return make_uint2(codes2(v[0], v[1], inv[0], inv[1]) | (codes2(v[2], v[3], inv[2], inv[3]) << 16),
                    codes2(v[4], v[5], inv[4], inv[5]) | (codes2(v[6], v[7], inv[6], inv[7]) << 16));
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  return make_uint2(codes2(v[0], v[1], inv, inv) | (codes2(v[2], v[3], inv, inv) << 16),
                    codes2(v[4], v[5], inv, inv) | (codes2(v[6], v[7], inv, inv) << 16));
}

// A warp takes 512 values of a row, 16 a lane: the block's scale, two divisions,
// is then computed for 16 values.  It goes from place to place by adding: a
// division of 64 bits costs as much as the codes.
template <class T>
__global__ void __launch_bounds__(kCodeThreads) row_codes_kernel(const T* X, int64_t rows, int64_t cols, int64_t ldx, bool vec,
                                                                 uint8_t* codes, int64_t ldc, bool vec_codes, float* scales,
                                                                 int64_t scale_row, int64_t scale_col, Clear clear) {
  asm volatile("griddepcontrol.launch_dependents;\n");
  clear_words(clear);
  const int lane = threadIdx.x & 31;
  const int64_t per = (cols + 511) / 512, first = (int64_t)blockIdx.x * (kCodeThreads / 32) + (threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * (kCodeThreads / 32);
  auto over = [&](int64_t x) { return (x | per) >> 32 ? x / per : (int64_t)((uint32_t)x / (uint32_t)per); };
  const int64_t step_rows = over(step), step_cols = step - step_rows * per;
  int64_t row = over(first), col = first - row * per;
  while (row < rows) {
    const int64_t k = col * 512 + lane * 16;
    Eight<T> x[2];
    x[0].load(X + row * ldx, k, cols, vec);
    x[1].load(X + row * ldx, k + 8, cols, vec);
    uint32_t top = Eight<T>::larger(x[0].top(), x[1].top());
#pragma unroll
    for (int o = 4; o; o >>= 1) top = Eight<T>::larger(top, __shfl_xor_sync(0xffffffffu, top, o));
    float scale, inv, v[2][8];
    block_scale(Eight<T>::top_of(top), scale, inv);
    if (k < cols) {
      uint8_t* to = codes + row * ldc;
      x[0].open(inv > 0.f, v[0]);
      x[1].open(inv > 0.f, v[1]);
      const uint2 a = codes8(v[0], inv), b = codes8(v[1], inv);
      if (vec_codes && k + 16 <= cols) {
        *reinterpret_cast<uint4*>(to + k) = make_uint4(a.x, a.y, b.x, b.y);
      } else {
        put_codes8(to, k, cols, false, a);
        put_codes8(to, k + 8, cols, false, b);
      }
      if ((lane & 7) == 0) scales[row * scale_row + (k >> 7) * scale_col] = scale;
    }
    row += step_rows, col += step_cols;
    if (col >= per) ++row, col -= per;
  }
}

// A tile of 128 x 128 for each block: codes along rows, along columns, or one
// scale for all, and the sums of the tile's columns.
struct TileCodes {
  int64_t rows, cols, ldx;
  bool vec;
  uint8_t *along, *down, *whole;  // null: not wanted
  int64_t ld_along, ld_down, ld_whole;
  bool vec_along, vec_down, vec_whole;
  float *along_scales, *down_scales, *whole_scales;
  int64_t along_row, along_col;  // strides of along_scales
  int64_t down_pitch;  // down_scales: a row of this many floats for each 128 rows
  int64_t whole_row;
  float* sums;  // a row of down_pitch floats for each 128 rows
  Clear clear;
};
template <class T>
__global__ void __launch_bounds__(kTileThreads, 2) tile_codes_kernel(const T* X, const __grid_constant__ TileCodes first, const T* second_X,
                                                                      const __grid_constant__ TileCodes second, int64_t split) {
  // The tiles of one matrix, then those of the other.
  const bool other = blockIdx.x >= split;
  const TileCodes& p = other ? second : first;
  if (other) X = second_X;
  using V = Eight<T>;
  constexpr int kWarps = kTileThreads / 32, kRows = 128 / (kTileThreads / 16), kEach = 128 / kRows;  // rows of a thread, kEach apart
  constexpr int kWords = V::kWords;
  __shared__ __align__(16) uint32_t tops[kWarps][16 * kWords];
  __shared__ __align__(16) float sums[kWarps][128];
  __shared__ __align__(16) float down_inv[128];
  asm volatile("griddepcontrol.launch_dependents;\n");
  clear_words(first.clear);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = lane & 15;
  const int64_t tile = (int64_t)blockIdx.x - (other ? split : 0), tiles_n = (p.cols + 127) / 128, tm = tile / tiles_n, tn = tile - tm * tiles_n;
  const int64_t r0 = tm * 128 + (threadIdx.x >> 4), k = tn * 128 + part * 8;  // rows r0, r0 + kEach, ..
  V x[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = r0 + kEach * i;
    if (r < p.rows)
      x[i].load(X + r * p.ldx, k, p.cols, p.vec);
    else
      x[i].zero();
  }
  float v[8], scale, inv;
  uint32_t all = 0;
  if (p.along || p.whole) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      uint32_t top = x[i].top();
      all = V::larger(all, top);
      if (!p.along) continue;
#pragma unroll
      for (int o = 8; o; o >>= 1) top = V::larger(top, __shfl_xor_sync(0xffffffffu, top, o));
      block_scale(V::top_of(top), scale, inv);
      const int64_t r = r0 + kEach * i;
      if (r < p.rows && k < p.cols) {
        x[i].open(inv > 0.f, v);
        put_codes8(p.along + r * p.ld_along, k, p.cols, p.vec_along, codes8(v, inv));
        if (part == 0) p.along_scales[r * p.along_row + tn * p.along_col] = scale;
      }
    }
  }
  if (p.whole) {
    all = __reduce_max_sync(0xffffffffu, V::top_of(all));
    if (lane == 0) tops[0][warp] = all;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all = max(all, tops[0][w]);
    block_scale(all, scale, inv);
    if (threadIdx.x == 0) p.whole_scales[tm * p.whole_row + tn] = scale;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t r = r0 + kEach * i;
      x[i].open(inv > 0.f, v);
      if (r < p.rows && k < p.cols) put_codes8(p.whole + r * p.ld_whole, k, p.cols, p.vec_whole, codes8(v, inv));
    }
    __syncthreads();
  }
  if (!p.down && !p.sums) return;
  uint32_t top[kWords];
#pragma unroll
  for (int e = 0; e < kWords; ++e) {
    top[e] = V::size_of(x[0].w[e]);
#pragma unroll
    for (int i = 1; i < kRows; ++i) top[e] = V::larger(top[e], V::size_of(x[i].w[e]));
    top[e] = V::larger(top[e], __shfl_xor_sync(0xffffffffu, top[e], 16));
  }
  if (lane < 16) {
#pragma unroll
    for (int e = 0; e < kWords; e += 4)
      *reinterpret_cast<uint4*>(&tops[warp][part * kWords + e]) = make_uint4(top[e], top[e + 1], top[e + 2], top[e + 3]);
  }
  if (p.sums) {
    float s[8] = {};
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      x[i].open(true, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += v[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += __shfl_xor_sync(0xffffffffu, s[e], 16);
    if (lane < 16) {
      *reinterpret_cast<float4*>(&sums[warp][part * 8]) = make_float4(s[0], s[1], s[2], s[3]);
      *reinterpret_cast<float4*>(&sums[warp][part * 8 + 4]) = make_float4(s[4], s[5], s[6], s[7]);
    }
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    uint32_t most = 0;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t word = tops[w][V::kPairs ? threadIdx.x / 2 : threadIdx.x];
      most = max(most, V::kPairs ? (threadIdx.x & 1 ? word >> 16 : word & 0xffffu) : word);
      if (p.sums) s += sums[w][threadIdx.x];
    }
    block_scale(V::as_fp32(most), scale, inv);
    down_inv[threadIdx.x] = inv;
    const int64_t c = tn * 128 + threadIdx.x;
    if (c < p.cols) {
      if (p.down) p.down_scales[tm * p.down_pitch + c] = scale;
      if (p.sums) p.sums[tm * p.down_pitch + c] = s;
    }
  }
  if (!p.down) return;
  __syncthreads();
  float each[8];
#pragma unroll
  for (int e = 0; e < 8; e += 4) {
    const float4 f = *reinterpret_cast<const float4*>(&down_inv[part * 8 + e]);
    each[e] = f.x, each[e + 1] = f.y, each[e + 2] = f.z, each[e + 3] = f.w;
  }
  uint32_t keep[kWords];
#pragma unroll
  for (int e = 0; e < kWords; ++e)
    keep[e] = V::kPairs ? (each[2 * e & 7] > 0.f ? 0xffffu : 0u) | (each[(2 * e + 1) & 7] > 0.f ? 0xffff0000u : 0u)
                        : (each[e] > 0.f ? 0xffffffffu : 0u);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = r0 + kEach * i;
    if (r < p.rows && k < p.cols) {
      x[i].open(keep, v);
      put_codes8(p.down + r * p.ld_down, k, p.cols, p.vec_down, codes8(v, each));
    }
  }
}

// The tiles' column sums added up, in their order.
__global__ void __launch_bounds__(256) column_sums_kernel(const float* parts, int64_t rows, int64_t pitch, int64_t cols, float* out) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= cols) return;
  float s = 0.f;
  for (int64_t r = 0; r < rows; ++r) s += parts[r * pitch + c];
  out[c] = s;
}

template <class T>
TileCodes tile_codes(const Fp8Codes& q) {
  auto in8 = [](const void* p, int64_t ld) { return aligned_to(p, 8) && ld % 8 == 0; };
  return TileCodes{q.rows, q.cols, q.ldx, aligned_to(q.X, 16) && q.ldx % (16 / (int64_t)sizeof(T)) == 0, q.along, q.down, q.whole,
                   q.ld_along, q.ld_down, q.ld_whole, in8(q.along, q.ld_along), in8(q.down, q.ld_down), in8(q.whole, q.ld_whole),
                   q.along_scales, q.down_scales, q.whole_scales, q.along_row, q.along_col, q.down_pitch, q.whole_row, q.sums,
                   Clear{static_cast<uint32_t*>(q.clear), (int)q.clear_words}};
}
int64_t tiles_of(const Fp8Codes& q) { return (q.rows + 127) / 128 * ((q.cols + 127) / 128); }
template <class T>
cudaError_t codes_typed(const Fp8Codes& q, const Fp8Codes* other, cudaStream_t stream) {
  const T* X = static_cast<const T*>(q.X);
  if (!other && q.along && !q.down && !q.whole && !q.sums) {
    const int64_t units = q.rows * ((q.cols + 511) / 512);
    const unsigned grid = (unsigned)std::min<int64_t>((units + kCodeThreads / 32 - 1) / (kCodeThreads / 32), 1 << 20);
    row_codes_kernel<T><<<grid, kCodeThreads, 0, stream>>>(
        X, q.rows, q.cols, q.ldx, aligned_to(q.X, 16) && q.ldx % (16 / (int64_t)sizeof(T)) == 0, q.along, q.ld_along,
        aligned_to(q.along, 16) && q.ld_along % 16 == 0, q.along_scales, q.along_row, q.along_col,
        Clear{static_cast<uint32_t*>(q.clear), (int)q.clear_words});
    return cudaGetLastError();
  }
  const int64_t split = tiles_of(q), tiles = split + (other ? tiles_of(*other) : 0);
  tile_codes_kernel<T><<<(unsigned)tiles, kTileThreads, 0, stream>>>(X, tile_codes<T>(q), other ? static_cast<const T*>(other->X) : X,
                                                                     tile_codes<T>(other ? *other : q), split);
  return cudaGetLastError();
}

}  // namespace

cudaError_t fp8_codes_launch(const Fp8Codes& q, const Fp8Codes* other, cudaStream_t stream) {
  switch (q.dtype) {
    case kF32: return codes_typed<float>(q, other, stream);
    case kF16: return codes_typed<__half>(q, other, stream);
    default: return codes_typed<__nv_bfloat16>(q, other, stream);
  }
}

cudaError_t fp8_column_sums_launch(const float* parts, int64_t rows, int64_t pitch, int64_t cols, float* out, cudaStream_t stream) {
  column_sums_kernel<<<(unsigned)((cols + 255) / 256), 256, 0, stream>>>(parts, rows, pitch, cols, out);
  return cudaGetLastError();
}

}  // namespace bakron
