// adamw.cu -- an AdamW step over many tensors in one launch.  With g = c grad:
//     m' = b1 m + (1 - b1) g,   v' = b2 v + (1 - b2) g^2,
//     p' = (1 - lr wd) p - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps).
// States are fp32, or e4m3 codes of m and of sqrt(v) with a scale for each 256
// values (scale = max / 448).  The codes are rounded at random, up with the
// probability of what is cut off: v changes by a thousandth a step, which
// rounding to nearest (half a step of e4m3 is up to 6%) would always lose.
//
// Bound by memory: parameters and states are read and written once, gradients
// read once (28 bytes a value in fp32; 16 with 8-bit states, 16-bit gradients
// and 16-bit copies).  A thread takes 8 values, a warp the 256 that share a
// scale; blocks walk over units of 2048 values of all tensors, whose addresses
// come in the kernel's parameters, so that a launch takes up to 128 tensors
// and a captured one keeps them.  Statistics, sums and the update are fp32.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "bakron.h"
#include "elem.cuh"
#include "layers.h"

namespace bakron {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamUnit = kAdamThreads * 8;
constexpr int kAdamList = 128;  // tensors of a launch

struct AdamConstants {
  float b1, c1, b2, c2, eps, root, rate, decay, grad;
  uint32_t key;  // of the seed and the step
};
struct AdamEntry {
  void* p;
  const void* g;
  void *m, *v;
  float *ms, *vs;
  void* copy;
  int64_t n;
  uint8_t p_type, g_type, copy_type, vec;
  uint32_t place;  // in the call's list
};
struct AdamList {
  AdamEntry e[kAdamList];
  int64_t first[kAdamList + 1];  // units before each tensor
  int count;
};

// 8 values from the i-th on, or fewer: up to n, then zeros.
template <class T>
__device__ __forceinline__ void get8(const T* p, int64_t i, int64_t n, bool vec, F2 (&v)[4]) {
  Raw8<T> raw;
  if (vec && i + 8 <= n) {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p + i) + k);
      raw.w[4 * k] = u.x, raw.w[4 * k + 1] = u.y, raw.w[4 * k + 2] = u.z, raw.w[4 * k + 3] = u.w;
    }
    open8<T>(raw, v);
  } else {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = i + k < n ? to_f32<T>(p[i + k]) : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = f2(f[2 * k], f[2 * k + 1]);
  }
}
template <class T>
__device__ __forceinline__ void put8(T* p, int64_t i, int64_t n, bool vec, const F2 (&v)[4]) {
  if (vec && i + 8 <= n) {
    Raw8<T> raw;
    close8<T>(v, raw);
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k)
      __stcs(reinterpret_cast<uint4*>(p + i) + k, make_uint4(raw.w[4 * k], raw.w[4 * k + 1], raw.w[4 * k + 2], raw.w[4 * k + 3]));
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a, b;
      split(v[k], a, b);
      if (i + 2 * k < n) p[i + 2 * k] = from_f32<T>(a);
      if (i + 2 * k + 1 < n) p[i + 2 * k + 1] = from_f32<T>(b);
    }
  }
}
__device__ __forceinline__ void get8(const void* p, int type, int64_t i, int64_t n, bool vec, F2 (&v)[4]) {
  if (type == kF32)
    get8(static_cast<const float*>(p), i, n, vec, v);
  else if (type == kF16)
    get8(static_cast<const __half*>(p), i, n, vec, v);
  else
    get8(static_cast<const __nv_bfloat16*>(p), i, n, vec, v);
}
__device__ __forceinline__ void put8(void* p, int type, int64_t i, int64_t n, bool vec, const F2 (&v)[4]) {
  if (type == kF32)
    put8(static_cast<float*>(p), i, n, vec, v);
  else if (type == kF16)
    put8(static_cast<__half*>(p), i, n, vec, v);
  else
    put8(static_cast<__nv_bfloat16*>(p), i, n, vec, v);
}
// 8 codes as bytes.
__device__ __forceinline__ uint2 get_codes(const void* p, int64_t i, int64_t n, bool vec) {
  const uint8_t* c = static_cast<const uint8_t*>(p) + i;
  if (vec && i + 8 <= n) return __ldcs(reinterpret_cast<const uint2*>(c));
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (i + k < n) w[k / 4] |= (uint32_t)c[k] << (8 * (k % 4));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void put_codes(void* p, int64_t i, int64_t n, bool vec, const uint32_t (&w)[2]) {
  uint8_t* c = static_cast<uint8_t*>(p) + i;
  if (vec && i + 8 <= n) {
    __stcs(reinterpret_cast<uint2*>(c), make_uint2(w[0], w[1]));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) c[k] = (uint8_t)(w[k / 4] >> (8 * (k % 4)));
  }
}
__device__ __forceinline__ void open_codes(const uint2& u, float scale, F2 (&v)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w = k < 2 ? u.x : u.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (k & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[k] = f2(f.x, f.y) * f2(scale);
  }
}

// 32 random bits for the i-th value of a tensor: a product with 2^32 over the
// golden ratio, then two rounds of a shift and a product with an odd number
// (the fractions of the roots of 2 and 3).
constexpr uint32_t kMixA = 0x9E3779B1u, kMixB = 0x6A09E667u, kMixC = 0xBB67AE85u;
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * kMixB;
  x = (x ^ (x >> 15)) * kMixC;
  return x ^ (x >> 16);
}

// 0 <= q <= 448 on the numbers of e4m3 at or below q plus `bits` / 2^16 of a
// step: q + step + bits step / 2^16 is cut to whole steps by adding a power of
// two whose own last place is a step, towards zero; then that power and the
// one step are taken off again.
__device__ __forceinline__ float cut_at_random(float q, uint32_t bits) {
  const uint32_t e = max(__float_as_uint(q) & 0x7f800000u, 121u << 23);  // at least 2^-6
  const float step = __uint_as_float(e - (3u << 23)), big = __uint_as_float(e + (20u << 23));
  const float t = fmaf(__uint_as_float(0x3f800000u | (bits << 7)), step, q);
  return __fadd_rz(t, big) - (big + step);
}
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// scale = max / 448 of the warp's values and its reciprocal; 0 and 0 where the reciprocal would overflow.
__device__ __forceinline__ void group_scale(float top, float& scale, float& inv) {
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // not negative: ordered as their bits
  scale = __fdiv_rn(top, 448.f);
  inv = scale >= 1.17549435e-38f ? __fdiv_rn(1.f, scale) : 0.f;
  if (inv == 0.f) scale = 0.f;
}

template <bool k8>
__global__ void __launch_bounds__(kAdamThreads, k8 ? 4 : 3)
    adamw_kernel(const __grid_constant__ AdamList list, const __grid_constant__ AdamConstants given, const AdamConstants* made,
                 const int32_t* skip, int32_t* status) {
  if (skip && *skip) return;
  const AdamConstants c = made ? *made : given;
  const int lane = threadIdx.x & 31;
  bool bad = false;
  int at = 0;
  const int64_t units = list.first[list.count];
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    if (u >= list.first[at + 1]) {  // the last tensor that begins at or before u
      int lo = at + 1, hi = list.count - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (list.first[mid] <= u)
          lo = mid;
        else
          hi = mid - 1;
      }
      at = lo;
    }
    const AdamEntry& e = list.e[at];
    const int64_t n = e.n, i = (u - list.first[at]) * kAdamUnit + threadIdx.x * 8;
    const bool vec = e.vec;
    if (i - lane * 8 >= n) continue;  // the whole warp's
    F2 p[4], g[4], m[4], v[4];
    float ms = 0.f, vs = 0.f;
    if constexpr (k8) {
      const uint2 mc = get_codes(e.m, i, n, vec), vc = get_codes(e.v, i, n, vec);
      ms = e.ms[i >> 8], vs = e.vs[i >> 8];
      get8(e.p, e.p_type, i, n, vec, p);
      get8(e.g, e.g_type, i, n, vec, g);
      open_codes(mc, ms, m);
      open_codes(vc, vs, v);  // the root
    } else {
      get8(static_cast<const float*>(e.m), i, n, vec, m);
      get8(static_cast<const float*>(e.v), i, n, vec, v);
      get8(e.p, e.p_type, i, n, vec, p);
      get8(e.g, e.g_type, i, n, vec, g);
    }
    float mt = 0.f, rt = 0.f;
    F2 root[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const F2 gk = g[k] * f2(c.grad);
      const F2 m0 = m[k], v0 = k8 ? v[k] * v[k] : v[k];
      const F2 m1 = fma2(gk, f2(c.c1), m0 * f2(c.b1)), v1 = fma2(gk * gk, f2(c.c2), v0 * f2(c.b2));
      float x[2], y[2], q[2], r[2], old[2], mo[2], vo[2];
      split(m1, x[0], x[1]);
      split(v1, y[0], y[1]);
      split(p[k], q[0], q[1]);
      split(m0, mo[0], mo[1]);
      split(v0, vo[0], vo[1]);
      if (k8) split(v[k], old[0], old[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        asm("sqrt.approx.f32 %0, %1;\n" : "=f"(r[h]) : "f"(y[h]));
        float d = fmaf(r[h], c.root, c.eps), over;
        asm("rcp.approx.f32 %0, %1;\n" : "=f"(over) : "f"(d));
        const float step = x[h] == 0.f ? 0.f : x[h] * over * c.rate;
        // A value whose gradient (or its square) is not finite stays what it is.
        const bool fine = fabsf(x[h]) < INFINITY && y[h] < INFINITY;
        const float moved = fmaf(q[h], c.decay, -step);
        if (fine) {
          q[h] = moved;
        } else {
          bad = true;
          x[h] = mo[h], y[h] = vo[h];
          if (k8) {
            x[h] = fabsf(x[h]) < INFINITY ? x[h] : 0.f;
            r[h] = fabsf(old[h]) < INFINITY ? old[h] : 0.f;
          }
        }
        if (k8) mt = fmaxf(mt, fabsf(x[h])), rt = fmaxf(rt, r[h]);
      }
      p[k] = f2(q[0], q[1]);
      m[k] = f2(x[0], x[1]);
      v[k] = f2(y[0], y[1]);
      root[k] = f2(r[0], r[1]);
    }
    put8(e.p, e.p_type, i, n, vec, p);
    if (e.copy) {
      if (e.copy_type == kF16)
        put8(static_cast<__half*>(e.copy), i, n, vec, p);
      else
        put8(static_cast<__nv_bfloat16*>(e.copy), i, n, vec, p);
    }
    if constexpr (k8) {
      float mi, vi;
      group_scale(mt, ms, mi);
      group_scale(rt, vs, vi);
      if (lane == 0) e.ms[i >> 8] = ms, e.vs[i >> 8] = vs;
      const uint32_t key = c.key + e.place * kMixC + (uint32_t)i * kMixA + (uint32_t)(i >> 32) * kMixC;
      uint32_t mc[2], vc[2];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x[2], r[2];
        split(m[k], x[0], x[1]);
        split(root[k], r[0], r[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t bits = mix(key + (uint32_t)(2 * k + h) * kMixA);
          x[h] = copysignf(cut_at_random(fabsf(x[h]) * mi, bits >> 16), x[h]);
          const float q = r[h] * vi, z = cut_at_random(q, bits & 0xffffu);
          // A root that is there stays there: nothing is divided by a lost one.
          r[h] = q > 0.f ? fmaxf(z, 0.001953125f) : 0.f;
        }
        const uint32_t a = e4m3_pair(x[0], x[1]), b = e4m3_pair(r[0], r[1]);
        mc[k >> 1] = k & 1 ? mc[k >> 1] | (a << 16) : a;
        vc[k >> 1] = k & 1 ? vc[k >> 1] | (b << 16) : b;
      }
      put_codes(e.m, i, n, vec, mc);
      put_codes(e.v, i, n, vec, vc);
    } else {
      put8(static_cast<float*>(e.m), i, n, vec, m);
      put8(static_cast<float*>(e.v), i, n, vec, v);
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(status, BAKRON_DEV_NONFINITE_GRAD);
}

__host__ __device__ inline AdamConstants constants(double lr, double step, double scale, double b1, double b2, double eps,
                                                   double decay, uint64_t seed) {
  AdamConstants c;
  c.b1 = (float)b1, c.c1 = (float)(1 - b1), c.b2 = (float)b2, c.c2 = (float)(1 - b2);
  c.eps = (float)eps;
  c.root = (float)(1 / sqrt(1 - pow(b2, step)));
  c.rate = (float)(lr / (1 - pow(b1, step)));
  c.decay = (float)(1 - lr * decay);
  c.grad = (float)scale;
  c.key = (uint32_t)seed * kMixA + (uint32_t)(uint64_t)step * kMixB;
  return c;
}
// Where the step or a factor is on the device.
__global__ void adamw_constants_kernel(Adamw a, AdamConstants* out) {
  *out = constants(a.lr_dev ? (double)*a.lr_dev : a.lr, a.step_dev ? (double)*a.step_dev : (double)a.step,
                   a.scale_dev ? (double)*a.scale_dev : a.scale, a.b1, a.b2, a.eps, a.decay, a.seed);
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 1;
  return std::max(1, sms);
}

}  // namespace

size_t adamw_workspace_bytes() { return 256; }

cudaError_t adamw_launch(const Adamw& a, const bakron_adamw_tensor* tensors, int64_t count, void* ws, int32_t* status,
                         cudaStream_t stream) {
  cudaError_t e = cudaMemsetAsync(status, 0, 4, stream);
  AdamConstants* made = nullptr;
  AdamConstants given = {};
  if (a.lr_dev || a.step_dev || a.scale_dev) {
    made = static_cast<AdamConstants*>(ws);
    if (e == cudaSuccess) adamw_constants_kernel<<<1, 1, 0, stream>>>(a, made);
  } else {
    given = constants(a.lr, (double)a.step, a.scale, a.b1, a.b2, a.eps, a.decay, a.seed);
  }
  const int64_t most = (int64_t)sm_count() * (a.eight ? 4 : 3);
  for (int64_t from = 0; from < count && e == cudaSuccess;) {
    AdamList list;
    list.count = 0;
    list.first[0] = 0;
    for (; from < count && list.count < kAdamList; ++from) {
      const bakron_adamw_tensor& t = tensors[from];
      if (t.n == 0) continue;
      bool vec = true;
      for (const void* q : {(const void*)t.param, t.grad, (const void*)t.m, (const void*)t.v, (const void*)t.copy}) vec = vec && aligned_to(q, 16);
      list.e[list.count] = AdamEntry{t.param, t.grad, t.m, t.v, t.m_scales, t.v_scales, t.copy, t.n, (uint8_t)t.param_dtype,
                                     (uint8_t)t.grad_dtype, (uint8_t)t.copy_dtype, (uint8_t)vec, (uint32_t)from};
      list.first[list.count + 1] = list.first[list.count] + (t.n + kAdamUnit - 1) / kAdamUnit;
      ++list.count;
    }
    if (list.count == 0) break;
    const unsigned grid = (unsigned)std::min<int64_t>(list.first[list.count], most);
    if (a.eight)
      adamw_kernel<true><<<grid, kAdamThreads, 0, stream>>>(list, given, made, a.skip, status);
    else
      adamw_kernel<false><<<grid, kAdamThreads, 0, stream>>>(list, given, made, a.skip, status);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace bakron
