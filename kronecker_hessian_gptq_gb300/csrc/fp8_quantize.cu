// fp8_quantize.cu -- codes in e4m3 with a scale for each 128 values of a row,
// 128 of a column, or block of 128 x 128 (see fp8_codes.cuh).
//
// Bound by memory: values are read once, into registers, their maxima taken
// there, and the codes written.  Along rows a warp takes 512 values of a row.
// Otherwise a block takes 128 x 128 values, 8 x 8 a thread; one read of them
// gives the codes along rows, the codes along columns and the columns' sums
// (what the backward pass of a product needs of its output's gradient).
#include <algorithm>

#include "fp8_codes.cuh"
#include "layers.h"

namespace bakron {
namespace {

constexpr int kCodeThreads = 256;
constexpr int kTileThreads = 512;

// 8 values from x[i] on, those past n as zeros.  Vectors where the rows allow.
template <class T>
__device__ __forceinline__ void values8(const T* x, int64_t i, int64_t n, bool vec, float (&v)[8]) {
  if (vec && i + 8 <= n) {
    load_vec<T, 8>(x + i, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = i + k < n ? to_f32<T>(x[i + k]) : 0.f;
  }
}
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
    float v[2][8];
    values8(X + row * ldx, k, cols, vec, v[0]);
    values8(X + row * ldx, k + 8, cols, vec, v[1]);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, magnitude(v[i / 8][i % 8]));
#pragma unroll
    for (int o = 4; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    float scale, inv;
    block_scale(top, scale, inv);
    if (k < cols) {
      uint8_t* to = codes + row * ldc;
      const uint2 a = fp8_codes8(v[0], inv), b = fp8_codes8(v[1], inv);
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
  constexpr int kWarps = kTileThreads / 32, kRows = 128 / (kTileThreads / 16), kEach = 128 / kRows;  // rows of a thread, kEach apart
  __shared__ uint32_t tops[kWarps][128];
  __shared__ float sums[kWarps][128];
  __shared__ float down_inv[128];
  asm volatile("griddepcontrol.launch_dependents;\n");
  clear_words(first.clear);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = lane & 15;
  const int64_t tile = (int64_t)blockIdx.x - (other ? split : 0), tiles_n = (p.cols + 127) / 128, tm = tile / tiles_n, tn = tile - tm * tiles_n;
  const int64_t r0 = tm * 128 + (threadIdx.x >> 4), k = tn * 128 + part * 8;  // rows r0, r0 + kEach, ..
  float v[kRows][8];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = r0 + kEach * i;
    if (r < p.rows) {
      values8(X + r * p.ldx, k, p.cols, p.vec, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }
  uint32_t all = 0;
  if (p.along || p.whole) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[i][e]));
      all = max(all, top);
      if (!p.along) continue;
#pragma unroll
      for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      float scale, inv;
      block_scale(top, scale, inv);
      const int64_t r = r0 + kEach * i;
      if (r < p.rows && k < p.cols) {
        put_codes8(p.along + r * p.ld_along, k, p.cols, p.vec_along, fp8_codes8(v[i], inv));
        if (part == 0) p.along_scales[r * p.along_row + tn * p.along_col] = scale;
      }
    }
  }
  if (p.whole) {
    all = __reduce_max_sync(0xffffffffu, all);
    if (lane == 0) tops[0][warp] = all;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all = max(all, tops[0][w]);
    float scale, inv;
    block_scale(all, scale, inv);
    if (threadIdx.x == 0) p.whole_scales[tm * p.whole_row + tn] = scale;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t r = r0 + kEach * i;
      if (r < p.rows && k < p.cols) put_codes8(p.whole + r * p.ld_whole, k, p.cols, p.vec_whole, fp8_codes8(v[i], inv));
    }
    __syncthreads();
  }
  if (!p.down && !p.sums) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) top = max(top, magnitude(v[i][e]));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
    if (lane < 16) tops[warp][part * 8 + e] = top;
    if (p.sums) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) s += v[i][e];
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      if (lane < 16) sums[warp][part * 8 + e] = s;
    }
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    uint32_t top = 0;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      top = max(top, tops[w][threadIdx.x]);
      if (p.sums) s += sums[w][threadIdx.x];
    }
    float scale, inv;
    block_scale(top, scale, inv);
    down_inv[threadIdx.x] = inv;
    const int64_t c = tn * 128 + threadIdx.x;
    if (c < p.cols) {
      if (p.down) p.down_scales[tm * p.down_pitch + c] = scale;
      if (p.sums) p.sums[tm * p.down_pitch + c] = s;
    }
  }
  if (!p.down) return;
  __syncthreads();
  float inv[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) inv[e] = down_inv[part * 8 + e];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = r0 + kEach * i;
    if (r < p.rows && k < p.cols)
      put_codes8(p.down + r * p.ld_down, k, p.cols, p.vec_down,
                 make_uint2(fp8_pair(v[i][0], v[i][1], inv[0], inv[1]) | (fp8_pair(v[i][2], v[i][3], inv[2], inv[3]) << 16),
                            fp8_pair(v[i][4], v[i][5], inv[4], inv[5]) | (fp8_pair(v[i][6], v[i][7], inv[6], inv[7]) << 16)));
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
