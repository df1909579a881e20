// int8_matmul.cu -- the product of quantized activations and quantized weights,
//     Y[t, o] = s_t w_o sum_k c[t, k] v[o, k] + b_o,
// for 8-bit codes c (one scale s_t for each token) and v (one scale w_o for
// each output), and the codes of activations,
//     s_t = fp32(max_k |x_tk| / 127), c_tk = rint(fp32(x_tk / s_t)).
// The integer sums are exact.  Three ways, by the number of tokens:
//
//   up to kRowTokens   a warp takes a row of weights in 16-byte pieces and
//                      multiplies it by every token's codes, which each block
//                      computes for itself while its first weights are on
//                      their way (dp4a): one launch, one read of the weights;
//   up to kPairTokens  int8_pair.cuh: tensor cores, weights converted to fp16
//                      inside, one read of them for 128 tokens;
//   above              the weights converted to fp16 once for the call (3
//                      bytes moved for each), then pair_gemm.cuh, whose
//                      operands come ready from memory.
#include <algorithm>

#include "bakron.h"
#include "elem.cuh"
#include "int8_pair.cuh"
#include "layers.h"
#include "quantize_tokens.cuh"

namespace bakron {
namespace {

// Where the next way becomes the faster one (us on the GPU for 4096 -> 4096,
// 4096 -> 14336 and 14336 -> 4096): 4 tokens by rows 9, 17, 24 and 8 tokens 14,
// 26, 39, where the tensor cores take 12, 19, 22 for either: up to 4 tokens, for
// the first two of the three.  768 tokens without
// the conversion 41, 99, 102, with it 42, 109, 123, and 1024 tokens 45, 125, 131
// against 44, 110, 129.
constexpr int64_t kRowTokens = 4;
constexpr int64_t kPairTokens = 768;
// Pairs of SMs that work is planned for: a whole GB300.  With fewer the results
// are the same (no pair waits for another), and some pairs work for two.
constexpr int kPlanPairs = 76;
constexpr int kRowThreads = 1024;
constexpr int64_t kRowSmem = 200 * 1024;  // codes of the tokens that a block keeps

int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }
int64_t up64(int64_t x) { return (x + 63) / 64 * 64; }
// Tokens that the row kernel is compiled for.
int row_tokens(int64_t T) { return T <= 1 ? 1 : T <= 2 ? 2 : 4; }
bool by_rows(int64_t T, int64_t K) { return T <= kRowTokens && row_tokens(T) * up16(K) <= kRowSmem; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// ------------------------------------------------------------ codes of tokens

constexpr int kPrepareThreads = 512;

// What a product does before its main kernel, in one launch: a block for each
// token takes its scale and its codes, as bytes or as fp16 for the tensor
// cores; the blocks after them rewrite codes that were given (as fp16, or as
// bytes in rows that start on 16 bytes), 16 at a time; all of them clear what
// the main kernel adds to.
struct Rewrite {
  const int8_t* from;
  int64_t ld, rows, cols;
  void* to;  // rows of ldt
  int64_t ldt;
  bool f16;
};
struct Prepare {
  const void* X;  // tokens x K values, or null
  int64_t tokens, K, ldx;
  bool vec;  // rows of X on 16 bytes, rows of the codes on a vector's own
  void* codes;
  int64_t ldc;
  float* scales;
  Rewrite rewrite[2];
  uint4* zero;
  int64_t zeros;
  int32_t* status;
};

// The 16 codes at v, of which `bytes` are there, zeros for the others.  Rows
// may start anywhere: the codes come in the 32-bit words that hold them,
// shifted into place.
__device__ __forceinline__ uint4 load_codes(const int8_t* v, int bytes) {
  const int off = (int)(reinterpret_cast<uintptr_t>(v) & 3);
  const uint32_t* word = reinterpret_cast<const uint32_t*>(v - off);
  uint32_t f[5], e[4];
#pragma unroll
  for (int i = 0; i < 5; ++i) f[i] = 4 * i < off + bytes ? word[i] : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[i] = __funnelshift_r(f[i], f[i + 1], 8 * off);
    const int here = bytes - 4 * i;
    if (here < 4) e[i] = here <= 0 ? 0u : e[i] & ((1u << (8 * here)) - 1u);
  }
  return make_uint4(e[0], e[1], e[2], e[3]);
}
__device__ __forceinline__ void store_codes(void* to, int64_t at, bool f16, const uint4& u) {
  if (f16) {
    uint32_t h[8];
    i8_to_f16(u.x, h[0], h[1]);
    i8_to_f16(u.y, h[2], h[3]);
    i8_to_f16(u.z, h[4], h[5]);
    i8_to_f16(u.w, h[6], h[7]);
    uint4* f = reinterpret_cast<uint4*>(static_cast<__half*>(to) + at);
    f[0] = make_uint4(h[0], h[1], h[2], h[3]);
    f[1] = make_uint4(h[4], h[5], h[6], h[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<int8_t*>(to) + at) = u;
  }
}
__device__ __forceinline__ void rewrite_codes(const Rewrite& w, int64_t at, int64_t step) {
  const int64_t per = (w.cols + 15) / 16, all = w.rows * per;
  if (w.ld == w.cols && w.ldt == w.cols && reinterpret_cast<uintptr_t>(w.from) % 16 == 0 && w.cols % 16 == 0) {
    // Dense on both sides: four loads of a thread on their way at once.
    const uint4* from = reinterpret_cast<const uint4*>(w.from);
    for (; at < all; at += 4 * step) {
      uint4 u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = at + i * step < all ? __ldcs(from + at + i * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i * step < all) store_codes(w.to, (at + i * step) * 16, w.f16, u[i]);
    }
    return;
  }
  for (; at < all; at += step) {
    const int64_t row = at < (1ll << 32) ? (int64_t)((uint32_t)at / (uint32_t)per) : at / per;  // per < 2^13
    const int64_t k = (at - row * per) * 16, left = w.cols - k;
    const int8_t* v = w.from + row * w.ld + k;
    const bool whole = left >= 16 && reinterpret_cast<uintptr_t>(v) % 16 == 0;
    store_codes(w.to, row * w.ldt + k, w.f16, whole ? __ldcs(reinterpret_cast<const uint4*>(v)) : load_codes(v, left < 16 ? (int)left : 16));
  }
}

template <class C>
__device__ __forceinline__ void put8(C* to, const float (&v)[8], float s, float inv) {
  uint32_t w[4];
  if constexpr (sizeof(C) == 1) {
    w[0] = w[1] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 4] |= (uint32_t)(token_code(v[i], s, inv) & 255) << (8 * (i % 4));
    *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<__half>((float)token_code(v[2 * i], s, inv), (float)token_code(v[2 * i + 1], s, inv));
    *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// NV > 0: a thread keeps its NV runs of 8 values in registers (K up to 4096
// NV), so that they are read once; 0: any K, read twice.
template <class T, class C, int NV>
__global__ void __launch_bounds__(kPrepareThreads) prepare_kernel(Prepare p) {
  __shared__ float red[32];
  asm volatile("griddepcontrol.launch_dependents;\n");  // see int8_pair_kernel
  if (p.status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < p.zeros; i += (int64_t)gridDim.x * blockDim.x)
    p.zero[i] = make_uint4(0, 0, 0, 0);
  if ((int64_t)blockIdx.x >= p.tokens) {
    const int64_t at = ((int64_t)blockIdx.x - p.tokens) * blockDim.x + threadIdx.x;
    const int64_t step = ((int64_t)gridDim.x - p.tokens) * blockDim.x;
#pragma unroll 1
    for (int i = 0; i < 2; ++i)
      if (p.rewrite[i].from) rewrite_codes(p.rewrite[i], at, step);
    return;
  }
  const T* x = static_cast<const T*>(p.X) + (int64_t)blockIdx.x * p.ldx;
  C* c = static_cast<C*>(p.codes) + (int64_t)blockIdx.x * p.ldc;
  const int64_t whole = p.vec ? p.K / 8 * 8 : 0;
  const int64_t stride = (int64_t)blockDim.x * 8;
  float v[NV ? NV : 1][8];
  float top[1] = {0.f};
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = threadIdx.x * 8 + i * stride;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      if (k < whole) load_vec<T, 8>(x + k, v[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) top[0] = MaxOp()(fabsf(v[i][e]), top[0]);
  } else {
    for (int64_t k = threadIdx.x * 8; k < whole; k += stride) {
      load_vec<T, 8>(x + k, v[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) top[0] = MaxOp()(fabsf(v[0][e]), top[0]);
    }
  }
  for (int64_t k = whole + threadIdx.x; k < p.K; k += blockDim.x) top[0] = MaxOp()(fabsf(to_f32<T>(x[k])), top[0]);
  block_reduce<1>(top, red, MaxOp());
  const float scale = token_scale(top[0]), inv = token_inv(scale);
  if (threadIdx.x == 0) p.scales[blockIdx.x] = scale;
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = threadIdx.x * 8 + i * stride;
      if (k < whole) put8(c + k, v[i], scale, inv);
    }
  } else {
    for (int64_t k = threadIdx.x * 8; k < whole; k += stride) {
      load_vec<T, 8>(x + k, v[0]);
      put8(c + k, v[0], scale, inv);
    }
  }
  for (int64_t k = whole + threadIdx.x; k < p.K; k += blockDim.x) {
    const int q = token_code(to_f32<T>(x[k]), scale, inv);
    if constexpr (sizeof(C) == 1)
      c[k] = (C)q;
    else
      c[k] = __int2half_rn(q);
  }
}

template <class T, class C>
void prepare_typed(const Prepare& p, unsigned grid, cudaStream_t stream) {
  const unsigned threads = (unsigned)std::min<int64_t>(kPrepareThreads, std::max<int64_t>(1, (p.K + 255) / 256) * 32);
  const int64_t one = (int64_t)threads * 8;
  if (!p.vec || p.K > 4 * one)
    prepare_kernel<T, C, 0><<<grid, threads, 0, stream>>>(p);
  else if (p.K <= one)
    prepare_kernel<T, C, 1><<<grid, threads, 0, stream>>>(p);
  else if (p.K <= 2 * one)
    prepare_kernel<T, C, 2><<<grid, threads, 0, stream>>>(p);
  else
    prepare_kernel<T, C, 4><<<grid, threads, 0, stream>>>(p);
}
template <class C>
cudaError_t prepare_launch(Prepare p, int dtype, cudaStream_t stream) {
  if (!p.X) p.tokens = 0;
  int64_t blocks = 0;  // of the rewriting: 16 codes for each thread, at most what fills the SMs four times
  for (const Rewrite& w : p.rewrite)
    if (w.from) blocks += (w.rows * ((w.cols + 15) / 16) + kPrepareThreads - 1) / kPrepareThreads;
  blocks = std::min<int64_t>(blocks, 2 * pair_count() * 16);
  const unsigned grid = (unsigned)std::max<int64_t>(1, p.tokens + blocks);
  p.vec = aligned_to(p.X, 16) && p.ldx % (16 / (int64_t)elem_size(dtype)) == 0 && p.ldc % 8 == 0 &&
          aligned_to(p.codes, 8 * sizeof(C));
  if (!p.X) p.K = kPrepareThreads * 8;  // whole blocks for the rewriting
  switch (dtype) {
    case kF32: prepare_typed<float, C>(p, grid, stream); break;
    case kF16: prepare_typed<__half, C>(p, grid, stream); break;
    default: prepare_typed<__nv_bfloat16, C>(p, grid, stream);
  }
  return cudaGetLastError();
}

// ------------------------------------------------------------ a few tokens

__device__ __forceinline__ void store_value(void* p, int dtype, int64_t i, float v) {
  if (dtype == kF32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == kF16)
    static_cast<__half*>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Codes of TT tokens (those past T are zeros) into shared memory, rows of
// `pitch` bytes with zeros from K on; 32 / TT warps for each token.  Every
// block does this for itself: it is a read of the tokens from the L2 cache.
// The maximum of magnitudes is taken on their bits, which order alike, with
// NaN above infinity.
template <int TT, class T>
__device__ __forceinline__ void tokens_to_shared(const Int8Matmul& p, int8_t* codes, int pitch, float* scales, uint32_t* top) {
  constexpr int VEC = 16 / sizeof(T), kPer = kRowThreads / TT;
  const int t = (threadIdx.x >> 5) % TT, id = (threadIdx.x >> 5) / TT * 32 + (threadIdx.x & 31);
  const int K = (int)p.K;
  const bool live = t < p.T;
  const T* x = static_cast<const T*>(p.X) + (live ? t : 0) * p.ldx;
  const int whole = reinterpret_cast<uintptr_t>(p.X) % 16 == 0 && p.ldx % VEC == 0 ? K / VEC * VEC : 0;
  if (threadIdx.x < TT) top[threadIdx.x] = 0;
  __syncthreads();
  if (live) {
    float m = 0.f;
    for (int k = id * VEC; k < whole; k += kPer * VEC) {
      float v[VEC];
      load_vec<T, VEC>(x + k, v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) m = MaxOp()(fabsf(v[i]), m);
    }
    for (int k = whole + id; k < K; k += kPer) m = MaxOp()(fabsf(to_f32<T>(x[k])), m);
    m = warp_reduce(m, MaxOp());
    if ((threadIdx.x & 31) == 0) atomicMax(top + t, __float_as_uint(m) & 0x7fffffffu);
  }
  __syncthreads();
  int8_t* c = codes + t * pitch;
  for (int k = (live ? K : 0) + id; k < pitch; k += kPer) c[k] = 0;
  if (!live) return;
  const float s = token_scale(__uint_as_float(top[t])), inv = token_inv(s);
  if (id == 0) scales[t] = s;
  for (int k = id * VEC; k < whole; k += kPer * VEC) {
    float v[VEC];
    load_vec<T, VEC>(x + k, v);
#pragma unroll
    for (int q = 0; q < VEC; q += 4) {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) w |= (uint32_t)(token_code(v[q + i], s, inv) & 255) << (8 * i);
      *reinterpret_cast<uint32_t*>(c + k + q) = w;
    }
  }
  for (int k = whole + id; k < K; k += kPer) c[k] = (int8_t)token_code(to_f32<T>(x[k]), s, inv);
}

// A row of weights for each `split` warps of a block (1, or where there are
// fewer rows than warps a power of two, which share a row and join through
// shared memory).  kVec: rows start on 16 bytes.
template <int TT, bool kVec>
__global__ void __launch_bounds__(kRowThreads) int8_rows_kernel(Int8Matmul p, int pitch, int split, int32_t* status) {
  extern __shared__ __align__(16) unsigned char rows_smem[];
  int8_t* codes = reinterpret_cast<int8_t*>(rows_smem);
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  __shared__ float scales[TT];
  __shared__ uint32_t top[TT];
  __shared__ int joined[32][TT];
  constexpr int kAhead = TT <= 2 ? 8 : 4;  // 16-byte pieces of a lane in flight, 512 bytes of a row each
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int K = (int)p.K, groups = (kRowThreads / 32) / split, part = warp % split;
  const int64_t stride = (int64_t)gridDim.x * groups;
  const int whole = K / 16 * 16;
  // this warp's pieces of a row: 512 bytes at lo + 512 i
  const int pieces = (whole + 511) / 512, lo = (int)((int64_t)pieces * part / split), hi = (int)((int64_t)pieces * (part + 1) / split);
  int64_t row = (int64_t)blockIdx.x * groups + warp / split;
  uint4 w[kAhead];
  auto fetch = [&](int64_t r, int first) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = (first + i) * 512 + lane * 16;
      w[i] = make_uint4(0, 0, 0, 0);
      if (r < p.N && first + i < hi && k < whole) w[i] = __ldcs(reinterpret_cast<const uint4*>(p.V + r * p.ldv + k));
    }
  };
  if (kVec) fetch(row, lo);  // on its way while the tokens are quantized
  if (p.x_scales) {
    const int live = (int)p.T;
    for (int t = 0; t < TT; ++t) {
      const int8_t* x = static_cast<const int8_t*>(p.X) + t * p.ldx;
      for (int k = threadIdx.x; k < pitch; k += kRowThreads) codes[t * pitch + k] = t < live && k < K ? x[k] : (int8_t)0;
      if (threadIdx.x == 0 && t < live) scales[t] = p.x_scales[t];
    }
  } else if (p.x_dtype == kF32) {
    tokens_to_shared<TT, float>(p, codes, pitch, scales, top);
  } else if (p.x_dtype == kF16) {
    tokens_to_shared<TT, __half>(p, codes, pitch, scales, top);
  } else {
    tokens_to_shared<TT, __nv_bfloat16>(p, codes, pitch, scales, top);
  }
  __syncthreads();
  for (; row < p.N || split > 1; row += stride) {
    int acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0;
    if (kVec) {
      for (int first = lo; first < hi; first += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int k = (first + i) * 512 + lane * 16;
          if (first + i >= hi || k >= whole) continue;
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const uint4 c = *reinterpret_cast<const uint4*>(codes + t * pitch + k);
            acc[t] = __dp4a((int)w[i].x, (int)c.x, acc[t]);
            acc[t] = __dp4a((int)w[i].y, (int)c.y, acc[t]);
            acc[t] = __dp4a((int)w[i].z, (int)c.z, acc[t]);
            acc[t] = __dp4a((int)w[i].w, (int)c.w, acc[t]);
          }
        }
        if (first + kAhead < hi) fetch(row, first + kAhead);
      }
      if (part == split - 1 && whole + lane < K && row < p.N) {
        const int v = p.V[row * p.ldv + whole + lane];
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[t] += v * codes[t * pitch + whole + lane];
      }
      if (split == 1) fetch(row + stride, lo);
    } else if (row < p.N) {
      const int8_t* v = p.V + row * p.ldv;
      for (int k = part * 32 + lane; k < K; k += split * 32) {
        const int x = v[k];
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[t] += x * codes[t * pitch + k];
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = __reduce_add_sync(0xffffffffu, acc[t]);
    if (split > 1) {  // one row for each group of warps, and no more
      if (lane == 0) {
#pragma unroll
        for (int t = 0; t < TT; ++t) joined[warp][t] = acc[t];
      }
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
          for (int q = 1; q < split; ++q) acc[t] += joined[warp + q][t];
      }
    }
    if (row < p.N && part == 0 && lane == 0) {
      const float ws = p.scales[row], bias = p.bias ? p.bias[row] : 0.f;
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (t < p.T) store_value(p.Y, p.y_dtype, t * p.ldy + row, fmaf((float)acc[t] * scales[t], ws, bias));
    }
    if (split > 1) break;
  }
}

template <int TT>
cudaError_t rows_launch(const Int8Matmul& p, int32_t* status, cudaStream_t stream) {
  const int pitch = (int)up16(p.K), sms = 2 * pair_count();
  const bool vec = aligned_to(p.V, 16) && p.ldv % 16 == 0;
  const int64_t warps = (int64_t)sms * (kRowThreads / 32);
  int split = 1;
  while (split < 32 && p.N * split * 2 <= warps && p.K >= 1024 * split) split *= 2;
  const int64_t groups = kRowThreads / 32 / split;
  const unsigned grid = (unsigned)std::min<int64_t>(sms, (p.N + groups - 1) / groups);
  const int smem = TT * pitch;
  auto kernel = vec ? int8_rows_kernel<TT, true> : int8_rows_kernel<TT, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRowSmem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kRowThreads, smem, stream>>>(p, pitch, split, status);
  return cudaGetLastError();
}

// ------------------------------------------------------------ many tokens

// Scales a tile's exact sums and sends them out in whole lines: 16-bit results
// whose rows start on 16 bytes by TMA, others row by row.
template <class T>
struct ScaledEpilogue {
  static constexpr bool kAhead = false;
  using Sum = int;
  CUtensorMap map;
  int64_t tokens, outputs;
  const float *x_scales, *w_scales, *bias;
  T* y;
  bool tma;  // then outputs is a multiple of 8 and the vectors start on 16 bytes
  __device__ __forceinline__ void operator()(const PairUnit&, int64_t row0, int64_t col, int64_t, const int (&acc)[64],
                                             const PairBox& box) const {
    if (row0 >= tokens || col >= outputs) return;
    const int here = (int)(tokens - row0 < 32 ? tokens - row0 : 32);
    const float s = box.lane < here ? x_scales[row0 + box.lane] : 0.f;
    if constexpr (sizeof(T) == 2) {
      if (tma) {
        box.open();
#pragma unroll
        for (int c = 0; c < 64; c += 8) {
          float w[8], b[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = b[i] = 0.f;
          if (col + c < outputs) {
            load_vec<float, 8>(w_scales + col + c, w);
            if (bias) load_vec<float, 8>(bias + col + c, b);
          }
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = fmaf((float)acc[c + i] * s, w[i], b[i]);
          box.put(c / 8, pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
        }
        box.send(&map, (int)col, (int)row0);
        return;
      }
    }
#pragma unroll
    for (int c = 0; c < 64; c += 32) {
      if (col + c >= outputs) break;
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = (float)acc[c + i] * s;
      const int64_t o = col + c + box.lane;
      const bool in = o < outputs;
      const float w = in ? w_scales[o] : 0.f, b = in && bias ? bias[o] : 0.f;
      T* to = y + row0 * outputs + o;
      box.by_row(v, here, in, [&](int r, float x) { to[r * outputs] = from_f32<T>(fmaf(x, w, b)); });
    }
  }
};

struct Layout {
  size_t codes, scales, zeros, arrived, sums, weights, end_zeros, bytes;
  I8Work work;
};

// copies: with room for the weights in aligned rows.
Layout layout(int64_t T, int64_t K, int64_t N, bool copies) {
  Layout l = {};
  if (by_rows(T, K)) return l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up256(bytes);
    return here;
  };
  l.codes = take(T * up64(K) * 2);
  l.scales = take(T * 4);
  if (T <= kPairTokens) {
    l.work = i8_work(T, K, N, kPlanPairs);
    l.zeros = at;
    l.arrived = take(i8_slices(l.work) * 4);
    l.sums = take(l.work.shared ? T * N * 4 : 0);
    l.end_zeros = l.work.shared ? at : l.zeros;
    if (copies) l.weights = take(N * up16(K));
  } else {
    l.weights = take(N * up64(K) * 2);
  }
  l.bytes = at;
  return l;
}

bool tma_codes(const Int8Matmul& p) { return aligned_to(p.V, 16) && p.ldv % 16 == 0; }

template <class T>
cudaError_t batch(const Int8Matmul& p, const Layout& l, char* ws, int32_t* status, cudaStream_t stream) {
  __half* codes = reinterpret_cast<__half*>(ws + l.codes);
  float* own_scales = reinterpret_cast<float*>(ws + l.scales);
  const float* s = p.x_scales ? p.x_scales : own_scales;
  const int64_t ldc = up64(p.K);
  const bool pairs = p.T <= kPairTokens, copy = !tma_codes(p);
  Prepare a = {};
  a.K = p.K;
  a.status = status;
  a.zero = reinterpret_cast<uint4*>(ws + l.zeros), a.zeros = (int64_t)(l.end_zeros - l.zeros) / 16;
  if (p.x_scales) {
    a.rewrite[0] = Rewrite{static_cast<const int8_t*>(p.X), p.ldx, p.T, p.K, codes, ldc, true};
  } else {
    a.X = p.X, a.tokens = p.T, a.ldx = p.ldx, a.codes = codes, a.ldc = ldc, a.scales = own_scales;
  }
  if (!pairs)
    a.rewrite[1] = Rewrite{p.V, p.ldv, p.N, p.K, ws + l.weights, ldc, true};
  else if (copy)
    a.rewrite[1] = Rewrite{p.V, p.ldv, p.N, p.K, ws + l.weights, up16(p.K), false};
  cudaError_t e = prepare_launch<__half>(a, p.x_scales ? kF32 : p.x_dtype, stream);
  if (e != cudaSuccess) return e;
  if (pairs) {
    const I8Out<T> out{p.T, p.N, s, p.scales, p.bias, static_cast<T*>(p.Y), reinterpret_cast<int32_t*>(ws + l.sums),
                       reinterpret_cast<uint32_t*>(ws + l.arrived)};
    return int8_pair_launch<T>(copy ? reinterpret_cast<int8_t*>(ws + l.weights) : p.V, copy ? up16(p.K) : p.ldv, codes, ldc,
                               p.K, l.work, out, !copy, status, stream);
  }
  const PairWork work{(int)((p.T + 255) / 256), (int)((p.N + 255) / 256), 16, (int)((p.K + kPairK - 1) / kPairK), 1};
  const PairOperand pc{codes, p.T, ldc}, pw{ws + l.weights, p.N, ldc};
  ScaledEpilogue<T> epi{{}, p.T, p.N, s, p.scales, p.bias, static_cast<T*>(p.Y), false};
  epi.tma = sizeof(T) == 2 && p.N % 8 == 0 && aligned_to(p.Y, 16) && aligned_to(p.scales, 16) && aligned_to(p.bias, 16);
  if (epi.tma)
    e = make_tensor_map(&epi.map, TileMap{p.Y, p.y_dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                          p.T, p.N, p.N, 32, 64, true});
  if (e != cudaSuccess) return e;
  return pair_gemm_launch<false, false, 4, 1024 / kPairK>(pc, pw, p.K, false, work, epi, status, stream);
}

}  // namespace

cudaError_t quantize_tokens_launch(const void* X, int dtype, int64_t T, int64_t K, int64_t ldx, int8_t* C, int64_t ldc,
                                   float* s, cudaStream_t stream) {
  Prepare a = {};
  a.X = X, a.tokens = T, a.K = K, a.ldx = ldx, a.codes = C, a.ldc = ldc, a.scales = s;
  return prepare_launch<int8_t>(a, dtype, stream);
}

size_t int8_matmul_workspace_bytes(int64_t T, int64_t K, int64_t N, bool copies) { return layout(T, K, N, copies).bytes; }
bool int8_matmul_needs_copies(const Int8Matmul& p) { return !tma_codes(p); }

cudaError_t int8_matmul_launch(const Int8Matmul& p, void* ws, int32_t* status_dev, cudaStream_t stream) {
  if (by_rows(p.T, p.K)) {
    switch (row_tokens(p.T)) {
      case 1: return rows_launch<1>(p, status_dev, stream);
      case 2: return rows_launch<2>(p, status_dev, stream);
      default: return rows_launch<4>(p, status_dev, stream);
    }
  }
  const Layout l = layout(p.T, p.K, p.N, !tma_codes(p));
  char* at = static_cast<char*>(ws);
  switch (p.y_dtype) {
    case kF32: return batch<float>(p, l, at, status_dev, stream);
    case kF16: return batch<__half>(p, l, at, status_dev, stream);
    default: return batch<__nv_bfloat16>(p, l, at, status_dev, stream);
  }
}

}  // namespace bakron
