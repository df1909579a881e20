// elem.cuh -- element types of the layer operators (fp32, fp16, bf16):
// conversions from and to fp32, vector loads and stores, and reductions over
// a team of threads.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace bakron {

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two values in the 16-bit type, the first in the low half.
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}

// Two fp32 values that go through the pipe together (the packed fp32
// instructions of sm_100 and later): half the instructions of kernels that
// are bound by issuing them.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split(F2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ float sum(F2 x) {
  float a, b;
  split(x, a, b);
  return a + b;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// Eight consecutive values of a thread, as 16 or 32 bytes and as pairs.
template <class T>
struct Raw8 {
  uint32_t w[2 * sizeof(T)];
};
template <class T>
__device__ __forceinline__ void open8(const Raw8<T>& raw, F2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = f2(__uint_as_float(raw.w[2 * i]), __uint_as_float(raw.w[2 * i + 1]));
    } else {
      T e[2];
      memcpy(e, &raw.w[i], 4);
      v[i] = f2(to_f32<T>(e[0]), to_f32<T>(e[1]));
    }
  }
}
template <class T>
__device__ __forceinline__ void close8(const F2 (&v)[4], Raw8<T>& raw) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    split(v[i], a, b);
    if constexpr (sizeof(T) == 4)
      raw.w[2 * i] = __float_as_uint(a), raw.w[2 * i + 1] = __float_as_uint(b);
    else
      raw.w[i] = pack2<T>(a, b);
  }
}

// VEC consecutive elements in one access of VEC * sizeof(T) bytes (at most
// 16 at a time); p must be aligned to that size.
template <class T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
  constexpr int kBytes = VEC * (int)sizeof(T);
  if constexpr (kBytes % 16 == 0) {
#pragma unroll
    for (int q = 0; q < kBytes / 16; ++q) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[q];
      T e[16 / sizeof(T)];
      memcpy(e, &u, 16);
#pragma unroll
      for (int i = 0; i < (int)(16 / sizeof(T)); ++i) v[q * (16 / sizeof(T)) + i] = to_f32<T>(e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = to_f32<T>(p[i]);
  }
}
template <class T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  constexpr int kBytes = VEC * (int)sizeof(T);
  if constexpr (kBytes % 16 == 0) {
#pragma unroll
    for (int q = 0; q < kBytes / 16; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4)
          w[i] = __float_as_uint(v[4 * q + i]);
        else
          w[i] = pack2<T>(v[8 * q + 2 * i], v[8 * q + 2 * i + 1]);
      }
      reinterpret_cast<uint4*>(p)[q] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = from_f32<T>(v[i]);
  }
}

// Sums and maxima over the threads of a block (any multiple of 32, at most
// 1024): N values at once; `red` holds 32 N floats.
struct SumOp {
  static constexpr float kIdentity = 0.f;
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// A NaN on either side stays: the maximum of a row with a NaN is NaN.
struct MaxOp {  // of magnitudes
  static constexpr float kIdentity = 0.f;
  __device__ __forceinline__ float operator()(float a, float b) const { return a > b || isnan(a) ? a : b; }
};
template <class Op>
__device__ __forceinline__ float warp_reduce(float v, Op op) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int N, class Op>
__device__ __forceinline__ void block_reduce(float (&v)[N], float* red, Op op) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_reduce(v[k], op);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();  // `red` may still be read by an earlier use
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) red[k * 32 + warp] = v[k];
  }
  __syncthreads();
  // every warp reduces the warps' values itself, in the same order
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_reduce(lane < nw ? red[k * 32 + lane] : Op::kIdentity, op);
}

// One value over a block of at most 32 warps with one barrier; `red`: two
// buffers of 64 floats that successive uses take turns with, so that one is
// written again only after a barrier that every reader of it has passed.
template <class Op>
__device__ __forceinline__ float block_one(float v, float* red, int& turn, Op op) {
  const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  v = warp_reduce(v, op);
  float* to = red + 64 * turn;
  turn ^= 1;
  if (lane == 0) to[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_reduce(lane < nw ? to[lane] : Op::kIdentity, op);
}

// Sums of four values over a warp in six exchanges: at each of the first two
// steps a lane hands on half of its values.  Lane 8 i has the i-th sum.
__device__ __forceinline__ float warp_sums4(const float (&v)[4]) {
  const int lane = threadIdx.x & 31;
  const bool high = lane & 16, odd = lane & 8;
  float a = (high ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, high ? v[0] : v[2], 16);
  float b = (high ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, high ? v[1] : v[3], 16);
  float s = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
  for (int o = 4; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Sums of eight values over a warp in nine exchanges; lane 4 i has the i-th sum.
__device__ __forceinline__ float warp_sums8(const float (&v)[8]) {
  const int lane = threadIdx.x & 31;
  const bool high = lane & 16, mid = lane & 8, odd = lane & 4;
  float a[4], b[2];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    a[k] = (high ? v[k + 4] : v[k]) + __shfl_xor_sync(0xffffffffu, high ? v[k] : v[k + 4], 16);
#pragma unroll
  for (int k = 0; k < 2; ++k) b[k] = (mid ? a[k + 2] : a[k]) + __shfl_xor_sync(0xffffffffu, mid ? a[k] : a[k + 2], 8);
  float s = (odd ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, odd ? b[0] : b[1], 4);
#pragma unroll
  for (int o = 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Sums of up to eight values over a block of at most 32 warps with one
// barrier.  `red`: two buffers of 256 floats, zero at first, which successive
// uses take turns with (`turn`), so that a buffer is written again only after
// a barrier that every reader of it has passed.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* red, int& turn) {
  static_assert(N <= 8, "");
  constexpr int kEach = N <= 4 ? 8 : 4;  // lanes that share a value
  const int lane = threadIdx.x & 31;
  float* to = red + 256 * turn;
  turn ^= 1;
  float w[32 / kEach], s;
#pragma unroll
  for (int k = 0; k < 32 / kEach; ++k) w[k] = k < N ? v[k] : 0.f;
  if constexpr (N <= 4)
    s = warp_sums4(w);
  else
    s = warp_sums8(w);
  if (lane % kEach == 0) to[lane / kEach * 32 + (threadIdx.x >> 5)] = s;
  __syncthreads();
  // value lane / kEach of 32 / kEach warps
  float t = 0.f;
#pragma unroll
  for (int k = 0; k < 8 / kEach; ++k) {
    const float4 f = *reinterpret_cast<const float4*>(to + lane / kEach * 32 + (k * kEach + lane % kEach) * 4);
    t += (f.x + f.y) + (f.z + f.w);
  }
#pragma unroll
  for (int o = kEach / 2; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = __shfl_sync(0xffffffffu, t, kEach * k);
}

// The 16 codes of a byte each at v, of which `bytes` are there, zeros for the
// others.  Rows may start anywhere: the codes come in the 32-bit words that hold them,
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

}  // namespace bakron
