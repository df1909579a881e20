// fp8_matmul.cu -- the product of activations and weights in e4m3 with a scale
// for each block of 128, and its gradients (fp8_pair.cuh, fp8_codes.cuh):
//     Y  = Q(X) V^T + b     Q: a scale for each 128 of a row of X,
//     dX = Q(dY) V          for each 128 of a row of dY,
//     dW = Q(dY)^T Q(X)     for each 128 tokens of a column of dY and of X.
// V's scales are one for 128 x 128, so that V's blocks serve both directions.
#include <algorithm>

#include "bakron.h"
#include "fp8_pair.cuh"
#include "layers.h"

namespace bakron {
namespace {

// Pairs of SMs that work is planned for: a whole GB300.  With fewer the results
// are the same (no pair waits for another), and some pairs work for two.
constexpr int kPlanPairs = 76;
// Up to so many tokens are the columns of a tile, whose rows are outputs; more
// are the rows, and outputs, which share a scale, the columns.
constexpr int64_t kColumnTokens = 128;

int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }
int64_t blocks_of(int64_t x) { return (x + kF8K - 1) / kF8K; }
bool on_16(const void* p, int64_t ld) { return aligned_to(p, 16) && ld % 16 == 0; }

// Workspace parts one after another, each on 256 bytes.
struct Room {
  size_t at = 0;
  size_t take(size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  }
};

// Tiles of 256 x kN, and parts of K where pairs would be without a tile.
PairWork plan(int64_t rows, int64_t cols, int kN, int64_t K) {
  PairWork w;
  w.tiles_m = (int)((rows + 255) / 256);
  w.tiles_n = (int)((cols + kN - 1) / kN);
  w.group = 16;
  w.ksteps = (int)blocks_of(K);
  const int64_t tiles = (int64_t)w.tiles_m * w.tiles_n;
  w.parts = tiles < kPlanPairs ? (int)std::max<int64_t>(1, std::min<int64_t>(kPlanPairs / tiles, w.ksteps / 2)) : 1;
  return w;
}
// Columns of a tile: 256 halve what is read for a product; with so few tiles that
// K is cut for most pairs, 128 halve the sums that meet in memory.  Microseconds with
// 128 / 256: 512 tokens 4096 -> 4096 17.5 / 23.3, 333 tokens 4096 -> 2048 15.8 / 21.0.
int columns_for(int64_t rows, int64_t cols) {
  const int64_t tiles = (rows + 255) / 256 * ((cols + 255) / 256);
  return 2 * tiles <= kPlanPairs ? 128 : 256;
}
// A slice is what one epilogue warp holds of a tile; the parts' sums are whole tiles.
int64_t slices(const PairWork& w) { return (int64_t)w.tiles_m * w.tiles_n * 2 * kF8Warps; }
size_t join_bytes(const PairWork& w, int kN) {
  return w.parts > 1 ? (size_t)w.parts * w.tiles_m * w.tiles_n * 256 * kN * sizeof(float) : 0;
}
size_t arrived_bytes(const PairWork& w) { return w.parts > 1 ? (size_t)slices(w) * 4 : 0; }

// ------------------------------------------------------------ forward

struct Forward {
  bool columns;  // tokens as columns
  int kN;
  PairWork work;
  int64_t pitch;  // of the tokens' scales, a row for each block of K
  size_t codes, scales, arrived, sums, weights, bytes;
};
Forward forward_plan(int64_t T, int64_t K, int64_t N, bool copies) {
  Forward f = {};
  f.columns = T <= kColumnTokens;
  f.kN = !f.columns ? columns_for(T, N) : T <= 64 ? 64 : 128;
  f.work = f.columns ? plan(N, T, f.kN, K) : plan(T, N, f.kN, K);
  f.pitch = f.columns ? (int64_t)f.work.tiles_n * f.kN : (int64_t)f.work.tiles_m * 256;
  Room room;
  f.codes = room.take(T * up16(K));
  f.scales = room.take(f.pitch * blocks_of(K) * 4);
  f.arrived = room.take(arrived_bytes(f.work));
  f.sums = room.take(join_bytes(f.work, f.kN));
  if (copies) f.weights = room.take(N * up16(K));
  f.bytes = room.at;
  return f;
}

// Rows of codes into rows that start on 16 bytes.
__global__ void __launch_bounds__(256) copy_codes_kernel(const int8_t* from, int64_t ld, int64_t rows, int64_t cols, int8_t* to,
                                                         int64_t ldt) {
  const int64_t per = (cols + 15) / 16, all = rows * per, step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += step) {
    const int64_t r = i / per, k = (i - r * per) * 16, left = cols - k;
    *reinterpret_cast<uint4*>(to + r * ldt + k) = load_codes(from + r * ld + k, left < 16 ? (int)left : 16);
  }
}
void copy_codes(const void* from, int64_t ld, int64_t rows, int64_t cols, void* to, cudaStream_t stream) {
  const int64_t all = rows * ((cols + 15) / 16);
  copy_codes_kernel<<<(unsigned)std::min<int64_t>((all + 255) / 256, 152 * 32), 256, 0, stream>>>(
      static_cast<const int8_t*>(from), ld, rows, cols, static_cast<int8_t*>(to), up16(cols));
}
// Given scales (a row for each token) as a row for each block; clears the join's counters.
__global__ void __launch_bounds__(256) turn_scales_kernel(const float* from, int64_t T, int64_t blocks, float* to, int64_t pitch,
                                                          uint32_t* word, int64_t words) {
  const int64_t step = (int64_t)gridDim.x * 256, first = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int64_t i = first; i < T * blocks; i += step) {
    const int64_t t = i / blocks;
    to[(i - t * blocks) * pitch + t] = from[i];
  }
  for (int64_t i = first; i < words; i += step) word[i] = 0;
}

template <class T>
cudaError_t forward(const Fp8Matmul& p, char* ws, int32_t* status, cudaStream_t stream) {
  const bool values = !p.x_scales, copy = !on_16(p.V, p.ldv);
  const Forward f = forward_plan(p.T, p.K, p.N, copy);
  const int64_t blocks = blocks_of(p.K);
  const void* codes = ws + f.codes;
  int64_t ldc = up16(p.K);
  float* scales = reinterpret_cast<float*>(ws + f.scales);
  uint32_t* arrived = reinterpret_cast<uint32_t*>(ws + f.arrived);
  const int64_t words = (int64_t)arrived_bytes(f.work) / 4;
  const void* V = p.V;
  int64_t ldv = p.ldv;
  if (copy) {
    copy_codes(p.V, p.ldv, p.N, p.K, ws + f.weights, stream);
    V = ws + f.weights, ldv = up16(p.K);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (values) {
    Fp8Codes q = {};
    q.X = p.X, q.dtype = p.x_dtype, q.rows = p.T, q.cols = p.K, q.ldx = p.ldx;
    q.along = reinterpret_cast<uint8_t*>(ws + f.codes), q.ld_along = ldc;
    q.along_scales = scales;
    q.along_row = 1, q.along_col = f.pitch;
    q.clear = arrived, q.clear_words = words;
    e = fp8_codes_launch(q, nullptr, stream);
  } else {
    if (on_16(p.X, p.ldx))
      codes = p.X, ldc = p.ldx;
    else
      copy_codes(p.X, p.ldx, p.T, p.K, ws + f.codes, stream);
    const int64_t all = std::max<int64_t>(p.T * blocks, words);
    turn_scales_kernel<<<(unsigned)std::min<int64_t>((all + 255) / 256, 152 * 8), 256, 0, stream>>>(
        p.x_scales, p.T, blocks, scales, f.pitch, arrived, words);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  const F8Join join{reinterpret_cast<float*>(ws + f.sums), arrived};
  const F8Operand x{codes, p.T, ldc}, v{V, p.N, ldv};
  const bool early = values && !copy;
  if (f.columns) {
    const F8Scales sc{p.scales, scales, 1, f.pitch, blocks, p.N};
    const F8Columns<T> epi{p.N, p.T, p.bias, static_cast<T*>(p.Y)};
    if (f.kN == 64)
      return fp8_pair_launch<false, false, 64, 1>(v, x, p.K, f.work, sc, join, epi, early, status, stream, 0);
    return fp8_pair_launch<false, false, 128, 1>(v, x, p.K, f.work, sc, join, epi, early, status, stream, 0);
  }
  const F8Scales sc{scales, p.scales, f.pitch, 1, blocks, p.N};
  F8Rows<T> epi{{}, p.T, p.N, p.bias, static_cast<T*>(p.Y), false};
  epi.tma = sizeof(T) == 2 && p.N % 8 == 0 && aligned_to(p.Y, 16) && aligned_to(p.bias, 16);
  if (epi.tma)
    e = make_tensor_map(&epi.map, TileMap{p.Y, p.y_dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                          p.T, p.N, p.N, 32, 64, true});
  if (e != cudaSuccess) return e;
  if (f.kN == 128)
    return fp8_pair_launch<false, false, 128, 2>(x, v, p.K, f.work, sc, join, epi, early, status, stream, 0);
  return fp8_pair_launch<false, false, 256, 2>(x, v, p.K, f.work, sc, join, epi, early, status, stream, 0);
}

// ------------------------------------------------------------ backward

struct Backward {
  int dx_kN, dw_kN;
  PairWork dx, dw;
  int64_t pitch_t, pitch_n, pitch_k;  // of scales, a row for each block of what is summed
  size_t along, along_scales, down_y, down_y_scales, down_x, down_x_scales, sums, arrived, arrived_words, join, weights, bytes;
};
Backward backward_plan(int64_t T, int64_t K, int64_t N, bool dX, bool dW, bool dbias, bool copies) {
  Backward b = {};
  b.dx_kN = columns_for(T, K), b.dw_kN = columns_for(N, K);
  b.dx = plan(T, K, b.dx_kN, N);
  b.dw = plan(N, K, b.dw_kN, T);
  b.pitch_t = (T + 255) / 256 * 256, b.pitch_n = (N + 255) / 256 * 256, b.pitch_k = (K + 255) / 256 * 256;
  Room room;
  if (dX) {
    b.along = room.take(T * up16(N));
    b.along_scales = room.take(b.pitch_t * blocks_of(N) * 4);
    if (copies) b.weights = room.take(N * up16(K));
  }
  if (dW) {
    b.down_y = room.take(T * up16(N));
    b.down_x = room.take(T * up16(K));
    b.down_x_scales = room.take(blocks_of(T) * b.pitch_k * 4);
    b.down_y_scales = room.take(blocks_of(T) * b.pitch_n * 4);
  }
  if (dbias) b.sums = room.take(blocks_of(T) * b.pitch_n * 4);
  // The two products follow one another: they share the room of their sums, not the counters.
  b.arrived = room.take((dX ? arrived_bytes(b.dx) : 0) + (dW ? arrived_bytes(b.dw) : 0));
  b.arrived_words = ((dX ? arrived_bytes(b.dx) : 0) + (dW ? arrived_bytes(b.dw) : 0)) / 4;
  b.join = room.take(std::max(dX ? join_bytes(b.dx, b.dx_kN) : 0, dW ? join_bytes(b.dw, b.dw_kN) : 0));
  b.bytes = room.at;
  return b;
}

template <class T>
cudaError_t backward(const Fp8Backward& p, char* ws, int32_t* status, cudaStream_t stream) {
  const bool copy = p.dX && !on_16(p.V, p.ldv);
  const Backward b = backward_plan(p.T, p.K, p.N, p.dX != nullptr, p.dW != nullptr, p.dbias != nullptr, copy);
  const CUtensorMapDataType type = p.dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  auto at = [&](size_t off) { return reinterpret_cast<uint8_t*>(ws + off); };
  auto floats = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  uint32_t* arrived = reinterpret_cast<uint32_t*>(ws + b.arrived);
  Fp8Codes q = {};
  q.X = p.dY, q.dtype = p.dtype, q.rows = p.T, q.cols = p.N, q.ldx = p.lddy;
  if (p.dX) q.along = at(b.along), q.ld_along = up16(p.N), q.along_scales = floats(b.along_scales), q.along_row = 1, q.along_col = b.pitch_t;
  if (p.dW) q.down = at(b.down_y), q.ld_down = up16(p.N), q.down_scales = floats(b.down_y_scales);
  q.down_pitch = b.pitch_n;
  if (p.dbias) q.sums = floats(b.sums);
  q.clear = arrived, q.clear_words = (int64_t)b.arrived_words;
  Fp8Codes x = {};
  x.X = p.X, x.dtype = p.dtype, x.rows = p.T, x.cols = p.K, x.ldx = p.ldx;
  if (p.dW) x.down = at(b.down_x), x.ld_down = up16(p.K), x.down_scales = floats(b.down_x_scales), x.down_pitch = b.pitch_k;
  cudaError_t e = fp8_codes_launch(q, p.dW ? &x : nullptr, stream);
  if (e == cudaSuccess && p.dbias) e = fp8_column_sums_launch(floats(b.sums), blocks_of(p.T), b.pitch_n, p.N, p.dbias, stream);
  auto rows = [&](void* y, int64_t m, int64_t n) {
    F8Rows<T> epi{{}, m, n, nullptr, static_cast<T*>(y), false};
    epi.tma = sizeof(T) == 2 && n % 8 == 0 && aligned_to(y, 16);
    if (epi.tma && e == cudaSuccess) e = make_tensor_map(&epi.map, TileMap{y, type, m, n, n, 32, 64, true});
    return epi;
  };
  if (e == cudaSuccess && p.dX) {
    const void* V = p.V;
    int64_t ldv = p.ldv;
    if (copy) {
      copy_codes(p.V, p.ldv, p.N, p.K, at(b.weights), stream);
      V = at(b.weights), ldv = up16(p.K);
      e = cudaGetLastError();
    }
    const F8Scales sc{q.along_scales, p.scales, b.pitch_t, blocks_of(p.K), 1, p.K};
    const F8Rows<T> epi = rows(p.dX, p.T, p.K);
    const F8Operand y{q.along, p.T, q.ld_along}, v{V, p.K, ldv};
    const F8Join join{floats(b.join), arrived};
    const bool early = !copy && !p.dbias;
    if (e == cudaSuccess)
      e = b.dx_kN == 128 ? fp8_pair_launch<false, true, 128, 2>(y, v, p.N, b.dx, sc, join, epi, early, status, stream, 0)
                         : fp8_pair_launch<false, true, 256, 2>(y, v, p.N, b.dx, sc, join, epi, early, status, stream, 0);
  }
  if (e == cudaSuccess && p.dW) {
    const F8Scales sc{q.down_scales, x.down_scales, b.pitch_n, b.pitch_k, 0, 0};
    const F8Rows<T> epi = rows(p.dW, p.N, p.K);
    if (p.dX) arrived += arrived_bytes(b.dx) / 4;
    const F8Operand y{q.down, p.N, q.ld_down}, v{x.down, p.K, x.ld_down};
    const F8Join join{floats(b.join), arrived};
    const int32_t first = p.dX ? -1 : 0;
    if (e == cudaSuccess)
      e = b.dw_kN == 128 ? fp8_pair_launch<true, true, 128, 0>(y, v, p.T, b.dw, sc, join, epi, true, status, stream, first)
                         : fp8_pair_launch<true, true, 256, 0>(y, v, p.T, b.dw, sc, join, epi, true, status, stream, first);
  }
  return e;
}

}  // namespace

size_t fp8_matmul_workspace_bytes(int64_t T, int64_t K, int64_t N, bool copies) {
  return fp8_few_tokens(T, K, N) ? 256 : forward_plan(T, K, N, copies).bytes;
}
bool fp8_matmul_needs_copies(const Fp8Matmul& p) { return !on_16(p.V, p.ldv); }
cudaError_t fp8_matmul_launch(const Fp8Matmul& p, void* ws, int32_t* status_dev, cudaStream_t stream) {
  if (fp8_few_tokens(p.T, p.K, p.N)) return fp8_rows(p, status_dev, stream);
  char* at = static_cast<char*>(ws);
  switch (p.y_dtype) {
    case kF32: return forward<float>(p, at, status_dev, stream);
    case kF16: return forward<__half>(p, at, status_dev, stream);
    default: return forward<__nv_bfloat16>(p, at, status_dev, stream);
  }
}

size_t fp8_backward_workspace_bytes(int64_t T, int64_t K, int64_t N, bool dX, bool dW, bool dbias, bool copies) {
  return backward_plan(T, K, N, dX, dW, dbias, copies).bytes;
}
bool fp8_backward_needs_copies(const Fp8Backward& p) { return p.dX && !on_16(p.V, p.ldv); }
cudaError_t fp8_backward_launch(const Fp8Backward& p, void* ws, int32_t* status_dev, cudaStream_t stream) {
  char* at = static_cast<char*>(ws);
  switch (p.dtype) {
    case kF32: return backward<float>(p, at, status_dev, stream);
    case kF16: return backward<__half>(p, at, status_dev, stream);
    default: return backward<__nv_bfloat16>(p, at, status_dev, stream);
  }
}

}  // namespace bakron
