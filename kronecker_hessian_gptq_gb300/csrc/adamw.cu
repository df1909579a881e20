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
// come in the kernel's parameters, so that a launch takes up to 384 tensors
// and a captured one keeps them.  Statistics, sums and the update are fp32.
// 235 million values: 1054 us in fp32 (6.2 TB/s), 696 us with 8-bit states, fp32
// masters, bf16 gradients and copies (5.4 TB/s), which issues 82 instructions a
// value, 70% of the time: a value's hash takes 9, two codes cut at random 16,
// products, sums and the root each rounded by themselves 10 (without that 660 us,
// but codes that fall elsewhere).  Sums and products go in pairs, conditions that
// hardly ever hold are tested for eight values at once, and all loads are under
// way before the first is converted (815 us before that, at 104 instructions).
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>

#include "bakron.h"
#include "elem.cuh"
#include "layers.h"

namespace bakron {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamUnit = kAdamThreads * 8;
// Tensors of a launch: a short list, or as many as a kernel's parameters have room for.
constexpr int kAdamShort = 24, kAdamLong = 384;

// Squares are kept 2^48 times as large where states have 8 bits: none is then
// subnormal, which the approximate square root would take for 0, and those that
// overflow go the way of values that are not finite.
constexpr float kLarger = 281474976710656.f, kRootLarger = 16777216.f;

struct AdamConstants {
  float b1, c1, b2, c2, eps, root, rate, decay, grad;
  uint32_t key;  // of the seed and the step
  // The same in pairs for 8-bit states, with squares kLarger times as large.
  F2 pb1, pc1, pb2, pc2, peps, proot, prate, pdecay, pgrad, one;
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
template <int kMost>
struct AdamList {
  AdamEntry e[kMost];
  int64_t first[kMost + 1];  // units before each tensor
  int count;
};

// 8 values of 16 or 32 bits from the i-th on as they lie in memory, or fewer: up
// to n, then zeros.  What they are is looked at after all loads are under way:
// a conversion waits for its values.
struct Raw {
  uint4 a, b;
};
__device__ __forceinline__ Raw get_raw(const void* p, bool wide, int64_t i, int64_t n, bool vec) {
  Raw r = {};
  if (vec && i + 8 <= n) {
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + (wide ? 4 * i : 2 * i));
    r.a = __ldcs(from);
    if (wide) r.b = __ldcs(from + 1);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      w[k] = 0;
      if (i + k < n) w[k] = wide ? static_cast<const uint32_t*>(p)[i + k] : static_cast<const uint16_t*>(p)[i + k];
    }
    if (wide)
      r.a = make_uint4(w[0], w[1], w[2], w[3]), r.b = make_uint4(w[4], w[5], w[6], w[7]);
    else
      r.a = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
  return r;
}
__device__ __forceinline__ void open_raw(const Raw& r, int type, F2 (&v)[4]) {
  if (type == kF32)
    open8<float>(Raw8<float>{{r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w}}, v);
  else if (type == kF16)
    open8<__half>(Raw8<__half>{{r.a.x, r.a.y, r.a.z, r.a.w}}, v);
  else
    open8<__nv_bfloat16>(Raw8<__nv_bfloat16>{{r.a.x, r.a.y, r.a.z, r.a.w}}, v);
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
// (the fractions of the roots of 2 and 3).  A seed's upper half goes through the
// same rounds before it is added to the lower one's.
constexpr uint32_t kMixA = 0x9E3779B1u, kMixB = 0x6A09E667u, kMixC = 0xBB67AE85u;
// The last step, x ^ x >> 16, is left to those who take the halves r of it, as
// (1 + r) / 8.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * kMixB;
  return (x ^ (x >> 15)) * kMixC;
}
__device__ __forceinline__ float more_of_upper(uint32_t x) { return __uint_as_float(((x >> 9) & 0x7fff80u) | 0x3e000000u); }
__device__ __forceinline__ float more_of_lower(uint32_t x) {
  return __uint_as_float((((x << 7) ^ (x >> 9)) & 0x7fff80u) | 0x3e000000u);
}

__device__ __forceinline__ F2 fma2_rz(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rz.f32x2 %0, %1, %2, %3;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// The roots of two numbers that are 0 or at least 2^-101: the approximate
// reciprocal root and one step of Newton's method with the exact residual y - s^2,
// which leaves the nearest number but for one in 10^5.  No number for an infinity.
__device__ __forceinline__ F2 roots(F2 y) {
  float a[2], r[2];
  split(y, a[0], a[1]);
#pragma unroll
  for (int h = 0; h < 2; ++h) asm("rsqrt.approx.ftz.f32 %0, %1;\n" : "=f"(r[h]) : "f"(fmaxf(a[h], 3.9443045e-31f)));
  const F2 over = f2(r[0], r[1]), s = y * over;
  return fma2(fma2(s, s, y * f2(-1.f)), over * f2(-0.5f), s);
}
// Two values |q| <= 448 on the numbers of e4m3 at or below |q| + r step, r the
// random 16 bits as a fraction, with q's sign.  With e the power of two below q,
// at least 2^-6, a step is e / 8: q + (1 + r) step is cut to whole steps by adding
// e 2^20, whose last place is a step, towards zero (both sums: what is cut twice
// is cut once); then that and the one step are taken off again.  more: (1 + r) / 8.
template <bool kSigned>
__device__ __forceinline__ F2 cut_at_random(F2 q, F2 more) {
  float x[2], e[2];
  split(q, x[0], x[1]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t u = __float_as_uint(x[h]), least = max(u & 0x7f800000u, 0x3c800000u);
    e[h] = __uint_as_float(kSigned ? least | (u & 0x80000000u) : least);
  }
  const F2 each = f2(e[0], e[1]), s = fma2_rz(each, f2(1048576.f), fma2_rz(each, more, q));
  return fma2(each, f2(-1048576.125f), s);
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

// New moment, square and parameter of one value.  One whose gradient or its
// square is not finite stays what it is (false).
__device__ __forceinline__ bool step_of(const AdamConstants& c, float g, float& p, float& m, float& v, float& root) {
  g *= c.grad;
  const float x = fmaf(g, c.c1, m * c.b1), y = fmaf(g * g, c.c2, v * c.b2);
  if (!(fabsf(x) < INFINITY && y < INFINITY)) return false;
  float over;
  asm("sqrt.approx.f32 %0, %1;\n" : "=f"(root) : "f"(y));
  asm("rcp.approx.f32 %0, %1;\n" : "=f"(over) : "f"(fmaf(root, c.root, c.eps)));
  p = fmaf(x * over, -c.rate, p * c.decay);
  m = x, v = y;
  return true;
}
// New moments and roots of two values, the roots kRootLarger times as large.  Each
// product and sum is rounded by itself (a sum as x one + y, which the compiler
// leaves alone), so that what a code is cut from is what the formula in elementary
// fp32 operations gives: a code that is cut the other way, over one unit in the
// last place, is off by a whole step of e4m3.
__device__ __forceinline__ void moments(const AdamConstants& c, F2 g, F2& m, F2& root) {
  m = fma2(m * c.pb1, c.one, g * c.pc1);
  root = roots(fma2(root * root * c.pb2, c.one, g * g * c.pc2));
}
// The codes of a thread's eight values of the warp's group, and lane 0 the scales.
// mt, rt: the largest |m| and root (kRootLarger times as large) of the thread.
__device__ __forceinline__ void put_states(const AdamConstants& c, const AdamEntry& e, int64_t i, float mt, float rt, const F2 (&m)[4],
                                           const F2 (&root)[4]) {
  constexpr float kLeast = 0.001953125f;  // of e4m3
  float ms, vs, mi, vi, least = 1.f;
  group_scale(mt, ms, mi);
  group_scale(rt * (1 / kRootLarger), vs, vi);
  vi *= 1 / kRootLarger;
  if ((threadIdx.x & 31) == 0) e.ms[i >> 8] = ms, e.vs[i >> 8] = vs;
  const uint32_t key = c.key + e.place * kMixC + (uint32_t)i * kMixA + (uint32_t)(i >> 32) * kMixC;
  uint32_t mw[2], vw[2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t h0 = mix(key + (uint32_t)(2 * k) * kMixA), h1 = mix(key + (uint32_t)(2 * k + 1) * kMixA);
    float z[2], q[2], r[2];
    split(cut_at_random<true>(m[k] * f2(mi), f2(more_of_upper(h0), more_of_upper(h1))), z[0], z[1]);
    // A root that is there stays there: nothing is divided by a lost one.
    split(root[k] * f2(vi), q[0], q[1]);
    least = fminf(least, fminf(q[0], q[1]));
    split(cut_at_random<false>(f2(fmaxf(q[0], kLeast), fmaxf(q[1], kLeast)), f2(more_of_lower(h0), more_of_lower(h1))), r[0], r[1]);
    const uint32_t a = e4m3_pair(z[0], z[1]), b = e4m3_pair(r[0], r[1]);
    mw[k >> 1] = k & 1 ? mw[k >> 1] | (a << 16) : a;
    vw[k >> 1] = k & 1 ? vw[k >> 1] | (b << 16) : b;
  }
  if (least == 0.f) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float r[2];
      split(root[k], r[0], r[1]);
      if (r[0] * vi == 0.f) vw[k >> 1] &= ~(0xffu << (16 * (k & 1)));
      if (r[1] * vi == 0.f) vw[k >> 1] &= ~(0xff00u << (16 * (k & 1)));
    }
  }
  put_codes(e.m, i, e.n, e.vec, mw);
  put_codes(e.v, i, e.n, e.vec, vw);
}
__device__ __forceinline__ void put_params(const AdamEntry& e, int64_t i, const F2 (&p)[4]) {
  put8(e.p, e.p_type, i, e.n, e.vec, p);
  if (!e.copy) return;
  if (e.copy_type == kF16)
    put8(static_cast<__half*>(e.copy), i, e.n, e.vec, p);
  else
    put8(static_cast<__nv_bfloat16*>(e.copy), i, e.n, e.vec, p);
}
// A warp's 256 values with 8-bit states, of which some are not finite or their
// squares too large for the fast way.  Returns whether a gradient is not finite.
__device__ __noinline__ bool step_of_group(const AdamConstants& c, const AdamEntry& e, int64_t i) {
  const int64_t n = e.n;
  const bool vec = e.vec;
  F2 p[4], g[4], m[4], root[4];
  open_codes(get_codes(e.m, i, n, vec), e.ms[i >> 8], m);
  open_codes(get_codes(e.v, i, n, vec), e.vs[i >> 8], root);
  open_raw(get_raw(e.p, e.p_type == kF32, i, n, vec), e.p_type, p);
  open_raw(get_raw(e.g, e.g_type == kF32, i, n, vec), e.g_type, g);
  __syncwarp();  // the scales are written below
  bool bad = false;
  float mt = 0.f, rt = 0.f;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const F2 gk = g[k] * c.pgrad;
    F2 m1 = m[k], r1 = root[k];
    moments(c, gk, m1, r1);
    float gs[2], ps[2], ms[2], rs[2], mn[2], rn[2];
    split(gk, gs[0], gs[1]);
    split(p[k], ps[0], ps[1]);
    split(m[k], ms[0], ms[1]);
    split(root[k], rs[0], rs[1]);
    split(m1, mn[0], mn[1]);
    split(r1, rn[0], rn[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // Squares that only the larger ones cannot hold: the root of the others.
      const float y = __fadd_rn(__fmul_rn(__fmul_rn(rs[h], rs[h]), c.b2), __fmul_rn(__fmul_rn(gs[h], gs[h]), c.c2));
      if (!(rn[h] < INFINITY)) rn[h] = sqrtf(y) * kRootLarger;
      float d, over, n0, p0, p1, other;
      split(fma2(f2(rn[h]), c.proot, c.peps), d, other);
      asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(over) : "f"(d));
      split(c.prate, n0, other);
      split(c.pdecay, p0, other);
      p1 = fmaf(mn[h] * over, n0, ps[h] * p0);
      if (fabsf(mn[h]) < INFINITY && y < INFINITY) {
        ps[h] = p1, ms[h] = mn[h], rs[h] = rn[h];
      } else {  // it stays what it is
        bad = true;
        if (!(fabsf(ms[h]) < INFINITY)) ms[h] = 0.f;
        rs[h] = rs[h] < INFINITY ? rs[h] * kRootLarger : 0.f;
      }
      mt = fmaxf(mt, fabsf(ms[h])), rt = fmaxf(rt, rs[h]);
    }
    p[k] = f2(ps[0], ps[1]), m[k] = f2(ms[0], ms[1]), root[k] = f2(rs[0], rs[1]);
  }
  put_params(e, i, p);
  put_states(c, e, i, mt, rt, m, root);
  return bad;
}

// kMade: the constants come from device memory.
template <bool k8, bool kMade, int kMost>
__global__ void __launch_bounds__(kAdamThreads, k8 ? 4 : 3)
    adamw_kernel(const __grid_constant__ AdamList<kMost> list, const __grid_constant__ AdamConstants given, const AdamConstants* made,
                 const int32_t* skip, int32_t* status) {
  if (skip && *skip) return;
  const AdamConstants c = kMade ? *made : given;
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
    F2 p[4], g[4];
    if constexpr (!k8) {
      F2 m[4], v[4];
      const Raw mr = get_raw(e.m, true, i, n, vec), vr = get_raw(e.v, true, i, n, vec);
      const Raw pr = get_raw(e.p, e.p_type == kF32, i, n, vec), gr = get_raw(e.g, e.g_type == kF32, i, n, vec);
      open_raw(mr, kF32, m);
      open_raw(vr, kF32, v);
      open_raw(pr, e.p_type, p);
      open_raw(gr, e.g_type, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float gs[2], ps[2], ms[2], vs[2], root;
        split(g[k], gs[0], gs[1]);
        split(p[k], ps[0], ps[1]);
        split(m[k], ms[0], ms[1]);
        split(v[k], vs[0], vs[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) bad |= !step_of(c, gs[h], ps[h], ms[h], vs[h], root);
        p[k] = f2(ps[0], ps[1]), m[k] = f2(ms[0], ms[1]), v[k] = f2(vs[0], vs[1]);
      }
      put8(static_cast<float*>(e.m), i, n, vec, m);
      put8(static_cast<float*>(e.v), i, n, vec, v);
      put_params(e, i, p);
    } else {
      const uint2 mc = get_codes(e.m, i, n, vec), vc = get_codes(e.v, i, n, vec);
      const float ms = e.ms[i >> 8], vs = e.vs[i >> 8];
      const Raw pr = get_raw(e.p, e.p_type == kF32, i, n, vec), gr = get_raw(e.g, e.g_type == kF32, i, n, vec);
      open_raw(pr, e.p_type, p);
      open_raw(gr, e.g_type, g);
      F2 m[4], root[4], odd = f2(0.f);
      open_codes(mc, ms, m);
      open_codes(vc, vs, root);
      float mt = 0.f, rt = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const F2 gk = g[k] * c.pgrad;
        moments(c, gk, m[k], root[k]);
        float r[2], d[2], o[2], x[2];
        split(root[k], r[0], r[1]);
        split(fma2(root[k], c.proot, c.peps), d[0], d[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(o[h]) : "f"(d[h]));
        p[k] = fma2(m[k] * f2(o[0], o[1]), c.prate, p[k] * c.pdecay);
        odd = fma2(m[k], f2(0.f), fma2(root[k], f2(0.f), odd));  // not 0 where one is not finite
        split(m[k], x[0], x[1]);
        mt = fmaxf(mt, fmaxf(fabsf(x[0]), fabsf(x[1])));
        rt = fmaxf(rt, fmaxf(r[0], r[1]));
      }
      if (__any_sync(0xffffffffu, sum(odd) != 0.f)) {
        bad |= step_of_group(c, e, i);
      } else {
        put_params(e, i, p);
        put_states(c, e, i, mt, rt, m, root);
      }
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(status, BAKRON_DEV_NONFINITE_GRAD);
}

__host__ __device__ inline F2 both(float x) {
  uint32_t u;
  memcpy(&u, &x, 4);
  return F2{(unsigned long long)u << 32 | u};
}
__host__ __device__ inline AdamConstants constants(double lr, double step, double scale, double b1, double b2, double eps,
                                                   double decay, uint64_t seed) {
  AdamConstants c;
  c.b1 = (float)b1, c.c1 = (float)(1 - b1), c.b2 = (float)b2, c.c2 = (float)(1 - b2);
  // At least the smallest normal number, too small to change a sum with any root
  // that is not 0: what is divided by is never 0.
  c.eps = eps > 1.1754943508222875e-38 ? (float)eps : 1.17549435e-38f;
  c.root = (float)(1 / sqrt(1 - pow(b2, step)));
  c.rate = (float)(lr / (1 - pow(b1, step)));
  c.decay = (float)(1 - lr * decay);
  c.grad = (float)scale;
  c.key = (uint32_t)seed * kMixA + mix((uint32_t)(seed >> 32) * kMixA) + (uint32_t)(uint64_t)step * kMixB;
  c.pb1 = both(c.b1), c.pc1 = both(c.c1), c.pb2 = both(c.b2 * kLarger), c.pc2 = both(c.c2 * kLarger), c.peps = both(c.eps);
  c.proot = both(c.root / kRootLarger), c.prate = both(-c.rate), c.pdecay = both(c.decay), c.pgrad = both(c.grad);
  c.one = both(1.f);
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

bool adamw_all_different(const bakron_adamw_tensor* tensors, int64_t count, bool eight) {
  // A table of at least twice as many places as addresses (six of a tensor); an address goes to the next free one.
  uint64_t size = 64;
  while (size < (uint64_t)count * 12) size *= 2;
  std::unique_ptr<const void*[]> seen(new (std::nothrow) const void*[size]());
  if (!seen) return false;
  auto fresh = [&](const void* p) {
    if (!p) return true;
    uint64_t i = (reinterpret_cast<uintptr_t>(p) >> 4) * 0x9E3779B97F4A7C15ull >> 20 & (size - 1);
    for (; seen[i]; i = (i + 1) & (size - 1))
      if (seen[i] == p) return false;
    seen[i] = p;
    return true;
  };
  for (int64_t i = 0; i < count; ++i) {
    const bakron_adamw_tensor& t = tensors[i];
    if (t.n && !(fresh(t.param) && fresh(t.m) && fresh(t.v) && fresh(t.copy) && (!eight || (fresh(t.m_scales) && fresh(t.v_scales)))))
      return false;
  }
  return true;
}

namespace {

template <int kMost>
cudaError_t launch_lists(const Adamw& a, const bakron_adamw_tensor* tensors, int64_t count, const AdamConstants& given,
                         const AdamConstants* made, int32_t* status, cudaStream_t stream) {
  const int64_t most = (int64_t)sm_count() * (a.eight ? 4 : 3);
  auto kernel = a.eight ? (made ? adamw_kernel<true, true, kMost> : adamw_kernel<true, false, kMost>)
                        : (made ? adamw_kernel<false, true, kMost> : adamw_kernel<false, false, kMost>);
  for (int64_t from = 0; from < count;) {
    AdamList<kMost> list;
    list.count = 0;
    list.first[0] = 0;
    for (; from < count && list.count < kMost; ++from) {
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
    // The launch's own error, not one that is left from before: a step that was made is never reported as failed.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid), cfg.blockDim = dim3(kAdamThreads), cfg.stream = stream;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, list, given, made, a.skip, status);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t adamw_launch(const Adamw& a, const bakron_adamw_tensor* tensors, int64_t count, void* ws, int32_t* status,
                         cudaStream_t stream) {
  cudaError_t e = cudaMemsetAsync(status, 0, 4, stream);
  if (e != cudaSuccess) return e;
  AdamConstants* made = nullptr;
  AdamConstants given = {};
  if (a.lr_dev || a.step_dev || a.scale_dev) {
    made = static_cast<AdamConstants*>(ws);
    adamw_constants_kernel<<<1, 1, 0, stream>>>(a, made);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  } else {
    given = constants(a.lr, (double)a.step, a.scale, a.b1, a.b2, a.eps, a.decay, a.seed);
  }
  return count <= kAdamShort ? launch_lists<kAdamShort>(a, tensors, count, given, made, status, stream)
                             : launch_lists<kAdamLong>(a, tensors, count, given, made, status, stream);
}

}  // namespace bakron
