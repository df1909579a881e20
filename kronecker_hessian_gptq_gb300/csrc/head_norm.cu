// head_norm.cu -- the norms of queries and keys for each head with the
// position rotation, forward and backward.  For a head x of D values at the
// position p, with n = x / sqrt(mean(x^2) + eps) * w (or n = x),
//     y[a] = n[a] cos(p f_i) - n[b] sin(p f_i),
//     y[b] = n[b] cos(p f_i) + n[a] sin(p f_i)
// for the pairs (a, b) = (i, i + R / 2) or (2 i, 2 i + 1) of the first R
// values, and y = n for the others.  Backward: dn is dy turned back, and with
// u = x / sqrt(..) and g = dn w
//     dx = (g - u mean(g u)) / sqrt(..),   dw = sum over tokens and heads of dn u.
//
// Bound by memory: each value is read once (dy and x backward) and written
// once.  A team of D / 16 lanes (rounded up to a power of two) holds a head,
// 16 values a lane in two runs of 8, so that both values of a pair are the
// same lane's, and a head's sums take three exchanges for D = 128.  A block
// takes a tile of up to eight tokens with all their heads: the angles of a
// token are computed once, into shared memory, for its 40 or so heads.
//
// An angle is kept as a share of a turn in 64-bit fixed point: p f / 2 pi
// modulo 1 is then one integer product, exact to |p f| 2^-54 turns for any
// position, where fp32 would be off by a tenth of a turn from 10^6 on and fp64
// runs at 1/64 of the fp32 rate.
#include <algorithm>

#include "elem.cuh"
#include "layers.h"

namespace bakron {
namespace {

constexpr int kHeadThreads = 256;
constexpr int kHeadTile = 8;  // tokens of a tile at most, a power of two
constexpr int kHeadBlocks = 4 * 152;  // of the backward pass: four on each SM

// The frequency f as a share of a turn for each position, 2^-64 of it.
__device__ __forceinline__ uint64_t turn_of(double f) {
  const double t = fabs(f) * 0.15915494309189533577;  // 1 / 2 pi
  const double part = t - floor(t);                   // exact
  const uint64_t share = part < 1.0 ? (uint64_t)(part * 18446744073709551616.0) : 0ull;  // 0 for a NaN
  return f < 0.0 ? 0ull - share : share;
}
// cos and sin of 2 pi times the share: the nearest quarter turn is taken off
// in integers, so that what is converted to fp32 is at most an eighth of a turn.
__device__ __forceinline__ void cos_sin(uint64_t share, float& c, float& s) {
  const uint32_t v = (uint32_t)(share >> 32);
  const uint32_t quarter = (v + 0x20000000u) >> 30;
  const int rest = (int)(v - (quarter << 30));
  float a, b;
  sincospif((float)rest * 4.656612873077393e-10f, &b, &a);  // 2^-31: in half turns
  c = quarter & 1 ? (quarter & 2 ? b : -b) : (quarter & 2 ? -a : a);
  s = quarter & 1 ? (quarter & 2 ? -a : a) : (quarter & 2 ? -b : b);
}

// Shared memory of a block: the turns of each frequency, and cos and sin for
// each token of a tile (rows of `pitch` floats).
struct Angles {
  uint64_t* turn;
  float *cos, *sin;
  int pitch;
  static __host__ __device__ int pitch_of(int half) { return (half + 7) / 8 * 8; }
  static __host__ __device__ size_t bytes(int half) { return (size_t)pitch_of(half) * (8 + 2 * 4 * kHeadTile); }
  __device__ explicit Angles(unsigned char* smem, int half) : pitch(pitch_of(half)) {
    turn = reinterpret_cast<uint64_t*>(smem);
    cos = reinterpret_cast<float*>(smem + 8 * pitch);
    sin = cos + pitch * kHeadTile;
  }
};
// A frequency that is not finite turns nothing into numbers.
__device__ __forceinline__ void fill_turns(const HeadNorm& p, const Angles& a) {
  for (int i = threadIdx.x; i < p.half; i += kHeadThreads) a.turn[i] = turn_of(p.freqs[i]);
}
__device__ __forceinline__ void fill_angles(const HeadNorm& p, const Angles& a, int64_t t0, int tokens) {
  for (int i = threadIdx.x; i < tokens * p.half; i += kHeadThreads) {
    const int t = i / p.half, k = i - t * p.half;
    float c, s;
    cos_sin((uint64_t)p.positions[t0 + t] * a.turn[k], c, s);
    if (!isfinite(p.freqs[k])) c = s = __int_as_float(0x7fffffff);
    a.cos[t * a.pitch + k] = c;
    a.sin[t * a.pitch + k] = s;
  }
}

template <class T>
__device__ __forceinline__ void load8(const T* p, Raw8<T>& raw) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    raw.w[4 * i] = u.x, raw.w[4 * i + 1] = u.y, raw.w[4 * i + 2] = u.z, raw.w[4 * i + 3] = u.w;
  }
}
template <class T>
__device__ __forceinline__ void store8(T* p, const F2 (&v)[4]) {
  Raw8<T> raw;
  close8<T>(v, raw);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    reinterpret_cast<uint4*>(p)[i] = make_uint4(raw.w[4 * i], raw.w[4 * i + 1], raw.w[4 * i + 2], raw.w[4 * i + 3]);
}
__device__ __forceinline__ void load_f2(const float* p, F2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 f = reinterpret_cast<const float4*>(p)[i];
    v[2 * i] = f2(f.x, f.y), v[2 * i + 1] = f2(f.z, f.w);
  }
}

// A lane's 16 values: two runs of 8, from lo and from hi on.
struct Place {
  int lo, hi;
  int angle;  // of lo's first pair
};
template <bool kNeighbours>
__device__ __forceinline__ Place place_of(int j, int rotated) {
  if (kNeighbours) return Place{16 * j, 16 * j + 8, 8 * j};
  if (16 * j < rotated) return Place{8 * j, rotated / 2 + 8 * j, 8 * j};
  return Place{16 * j, 16 * j + 8, 8 * j};
}

// Turns a lane's pairs by their angles, or back (kBack).
template <bool kNeighbours, bool kBack>
__device__ __forceinline__ void turn_pairs(F2 (&a)[4], F2 (&b)[4], const float* cos, const float* sin, int angle, int half) {
  if (!kNeighbours) {
    if (angle >= half) return;
    F2 c[4], s[4];
    load_f2(cos + angle, c);
    load_f2(sin + angle, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 minus = f2(-1.f) * s[i];
      const F2 x = a[i], y = b[i];
      a[i] = fma2(y, kBack ? s[i] : minus, x * c[i]);
      b[i] = fma2(x, kBack ? minus : s[i], y * c[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (angle + i >= half) break;
      const float c = cos[angle + i], s = kBack ? -sin[angle + i] : sin[angle + i];
      F2& v = i < 4 ? a[i & 3] : b[i & 3];
      float x, y;
      split(v, x, y);
      v = f2(fmaf(-y, s, x * c), fmaf(x, s, y * c));
    }
  }
}

__device__ __forceinline__ float team_sum(float v, int lanes) {
  for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float squares(const F2 (&a)[4], const F2 (&b)[4]) {
  F2 q = a[0] * a[0];
#pragma unroll
  for (int i = 1; i < 4; ++i) q = fma2(a[i], a[i], q);
#pragma unroll
  for (int i = 0; i < 4; ++i) q = fma2(b[i], b[i], q);
  return sum(q);
}

// Two heads of a team are on their way at a time.
template <class T, bool kNeighbours>
__global__ void __launch_bounds__(kHeadThreads) head_norm_kernel(const __grid_constant__ HeadNorm p, int tile, int lanes) {
  extern __shared__ __align__(16) unsigned char head_smem[];
  const Angles angles(head_smem, p.half);
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  const int tokens = (int)(p.T - t0 < tile ? p.T - t0 : tile);
  const int j = threadIdx.x & (lanes - 1), team = threadIdx.x / lanes, teams = kHeadThreads / lanes;
  const bool mine = 16 * j < p.D;
  const Place at = place_of<kNeighbours>(j, 2 * p.half);
  const float each = 1.f / (float)p.D;
  const int units = (p.side[0].heads + p.side[1].heads) * tile, step = teams * gridDim.y;
  Raw8<T> lo[2], hi[2];
  auto side_of = [&](int u, int& h) {
    h = u / tile;  // a power of two
    const int k = h >= p.side[0].heads;
    if (k) h -= p.side[0].heads;
    return k;
  };
  auto fetch = [&](int u, int n) {
    const int t = u & (tile - 1);
    if (u < units && t < tokens && mine) {
      int h;
      const int k = side_of(u, h);
      const HeadSide& s = p.side[k];
      const T* x = static_cast<const T*>(s.x) + (t0 + t) * s.x_token + h * s.x_head;
      load8(x + at.lo, lo[n]);
      load8(x + at.hi, hi[n]);
    } else {
#pragma unroll
      for (int i = 0; i < 2 * (int)sizeof(T); ++i) lo[n].w[i] = hi[n].w[i] = 0;
    }
  };
  int u = (int)blockIdx.y * teams + team;
  fetch(u, 0);
  fetch(u + step, 1);
  if (p.half) {
    fill_turns(p, angles);
    __syncthreads();
    fill_angles(p, angles, t0, tokens);
    __syncthreads();
  }
  // All teams take the same number of turns: the exchanges are the whole warp's.
  for (int base = (int)blockIdx.y * teams; base < units; base += 2 * step, u += 2 * step) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int v = u + n * step;
      F2 a[4], b[4];
      open8<T>(lo[n], a);
      open8<T>(hi[n], b);
      fetch(v + 2 * step, n);
      const int t = v & (tile - 1);
      int h;
      const int k = side_of(v, h);
      const HeadSide& s = p.side[k];
      const float r = __frsqrt_rn(fmaf(team_sum(squares(a, b), lanes), each, p.eps));
      if (v >= units || t >= tokens || !mine) continue;
      if (s.w) {
        F2 w[4];
        load_f2(s.w + at.lo, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = a[i] * f2(r) * w[i];
        load_f2(s.w + at.hi, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = b[i] * f2(r) * w[i];
      }
      turn_pairs<kNeighbours, false>(a, b, angles.cos + t * angles.pitch, angles.sin + t * angles.pitch, at.angle, p.half);
      T* y = static_cast<T*>(s.y) + ((t0 + t) * s.heads + h) * p.D;
      store8(y + at.lo, a);
      store8(y + at.hi, b);
    }
  }
}

// Any sizes, strides and alignment: a warp for each head, which reads it
// twice.  Pair i of the head (i < half), then its single values.
__device__ __forceinline__ void pair_at(const HeadNorm& p, int i, int& a, int& b) {
  if (i >= p.half) {
    a = b = p.half + i;
  } else if (p.neighbours) {
    a = 2 * i, b = a + 1;
  } else {
    a = i, b = i + p.half;
  }
}

template <class T>
__global__ void __launch_bounds__(kHeadThreads) head_norm_any_kernel(const __grid_constant__ HeadNorm p, int tile) {
  extern __shared__ __align__(16) unsigned char head_smem[];
  const Angles angles(head_smem, p.half);
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  const int tokens = (int)(p.T - t0 < tile ? p.T - t0 : tile);
  if (p.half) {
    fill_turns(p, angles);
    __syncthreads();
    fill_angles(p, angles, t0, tokens);
    __syncthreads();
  }
  const int lane = threadIdx.x & 31, heads = p.side[0].heads + p.side[1].heads, D = p.D, pairs = D - p.half;
  const int warps = kHeadThreads / 32;
  for (int u = (int)blockIdx.y * warps + (threadIdx.x >> 5); u < heads * tile; u += warps * gridDim.y) {
    const int t = u & (tile - 1);
    int h = u / tile;
    if (t >= tokens) continue;
    const int k = h >= p.side[0].heads;
    if (k) h -= p.side[0].heads;
    const HeadSide& s = p.side[k];
    const T* x = static_cast<const T*>(s.x) + (t0 + t) * s.x_token + h * s.x_head;
    T* y = static_cast<T*>(s.y) + ((t0 + t) * s.heads + h) * D;
    float r = 1.f;
    if (s.w) {
      float q = 0.f;
      for (int i = lane; i < D; i += 32) {
        const float v = to_f32<T>(x[i]);
        q = fmaf(v, v, q);
      }
      r = __frsqrt_rn(fmaf(warp_reduce(q, SumOp()), 1.f / (float)D, p.eps));
    }
    for (int i = lane; i < pairs; i += 32) {
      int a, b;
      pair_at(p, i, a, b);
      float va = to_f32<T>(x[a]), vb = to_f32<T>(x[b]);
      if (s.w) va = va * r * s.w[a], vb = vb * r * s.w[b];
      if (i < p.half) {
        const float c = angles.cos[t * angles.pitch + i], z = angles.sin[t * angles.pitch + i];
        y[a] = from_f32<T>(fmaf(-vb, z, va * c));
        y[b] = from_f32<T>(fmaf(va, z, vb * c));
      } else {
        y[a] = from_f32<T>(va);
      }
    }
  }
}

// ------------------------------------------------------------ backward

// Weight gradients of a block: D floats for queries, D for keys, in `parts`.
template <class T, bool kNeighbours>
__global__ void __launch_bounds__(kHeadThreads) head_norm_backward_kernel(const __grid_constant__ HeadNorm p, int tile, int lanes,
                                                                          int64_t tiles, float* parts) {
  extern __shared__ __align__(16) unsigned char head_smem[];
  const Angles angles(head_smem, p.half);
  const int j = threadIdx.x & (lanes - 1), team = threadIdx.x / lanes, teams = kHeadThreads / lanes;
  const bool mine = 16 * j < p.D;
  const Place at = place_of<kNeighbours>(j, 2 * p.half);
  const float each = 1.f / (float)p.D;
  F2 dw[2][8];
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i >> 3][i & 7] = f2(0.f);
  if (p.half) fill_turns(p, angles);
  for (int64_t q = blockIdx.x; q < tiles; q += gridDim.x) {
    const int64_t t0 = q * tile;
    const int tokens = (int)(p.T - t0 < tile ? p.T - t0 : tile);
    if (p.half) {
      __syncthreads();
      fill_angles(p, angles, t0, tokens);
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const HeadSide& s = p.side[k];
      const int units = s.heads * tile;
      for (int base = 0; base < units; base += teams) {
        const int u = base + team, t = u & (tile - 1), h = u / tile;
        const bool live = u < units && t < tokens && mine;
        F2 g[8], x[8];
        F2(&ga)[4] = *reinterpret_cast<F2(*)[4]>(g), (&gb)[4] = *reinterpret_cast<F2(*)[4]>(g + 4);
        F2(&xa)[4] = *reinterpret_cast<F2(*)[4]>(x), (&xb)[4] = *reinterpret_cast<F2(*)[4]>(x + 4);
        if (live) {
          const T* d = static_cast<const T*>(s.dy) + (t0 + t) * s.dy_token + h * s.dy_head;
          Raw8<T> raw[4];
          load8(d + at.lo, raw[0]);
          load8(d + at.hi, raw[1]);
          if (s.w) {
            const T* v = static_cast<const T*>(s.x) + (t0 + t) * s.x_token + h * s.x_head;
            load8(v + at.lo, raw[2]);
            load8(v + at.hi, raw[3]);
            open8<T>(raw[2], xa);
            open8<T>(raw[3], xb);
          }
          open8<T>(raw[0], ga);
          open8<T>(raw[1], gb);
          turn_pairs<kNeighbours, true>(ga, gb, angles.cos + t * angles.pitch, angles.sin + t * angles.pitch, at.angle, p.half);
        }
        if (!live || !s.w) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = f2(0.f);
            if (!live) g[i] = f2(0.f);
          }
        }
        if (s.w) {
          const float r = __frsqrt_rn(fmaf(team_sum(squares(xa, xb), lanes), each, p.eps));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = x[i] * f2(r);
            dw[k][i] = fma2(g[i], x[i], dw[k][i]);
          }
          F2 dot = f2(0.f);
          if (mine) {
            F2 w[4];
            load_f2(s.w + at.lo, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = g[i] * w[i];
            load_f2(s.w + at.hi, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) g[4 + i] = g[4 + i] * w[i];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) dot = fma2(g[i], x[i], dot);
          const float c = -team_sum(sum(dot), lanes) * each;
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = fma2(x[i], f2(c), g[i]) * f2(r);
        }
        if (live) {
          T* y = static_cast<T*>(s.y) + ((t0 + t) * s.heads + h) * p.D;
          store8(y + at.lo, ga);
          store8(y + at.hi, gb);
        }
      }
    }
  }
  if (!parts) return;
  // The teams' sums one after another, in their order.
  __syncthreads();
  float* all = reinterpret_cast<float*>(head_smem);  // teams x D
  for (int k = 0; k < 2; ++k) {
    if (mine) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float a, b;
        split(k ? dw[1][i] : dw[0][i], a, b);
        const int e = (i < 4 ? at.lo : at.hi) + 2 * (i & 3);
        all[team * p.D + e] = a;
        all[team * p.D + e + 1] = b;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.D; e += kHeadThreads) {
      float v = 0.f;
      for (int i = 0; i < teams; ++i) v += all[i * p.D + e];
      parts[((int64_t)blockIdx.x * 2 + k) * p.D + e] = v;
    }
    __syncthreads();
  }
}

template <class T>
__global__ void __launch_bounds__(kHeadThreads) head_norm_backward_any_kernel(const __grid_constant__ HeadNorm p, int tile,
                                                                              int64_t tiles, float* parts) {
  extern __shared__ __align__(16) unsigned char head_smem[];
  const Angles angles(head_smem, p.half);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kHeadThreads / 32, D = p.D, pairs = D - p.half;
  // each warp's sums: 2 D floats
  float* own = reinterpret_cast<float*>(head_smem + Angles::bytes(p.half)) + warp * 2 * D;
  for (int i = lane; i < 2 * D; i += 32) own[i] = 0.f;
  if (p.half) fill_turns(p, angles);
  for (int64_t q = blockIdx.x; q < tiles; q += gridDim.x) {
    const int64_t t0 = q * tile;
    const int tokens = (int)(p.T - t0 < tile ? p.T - t0 : tile);
    if (p.half) {
      __syncthreads();
      fill_angles(p, angles, t0, tokens);
      __syncthreads();
    }
    for (int u = warp; u < (p.side[0].heads + p.side[1].heads) * tile; u += warps) {
      const int t = u & (tile - 1);
      int h = u / tile;
      if (t >= tokens) continue;
      const int k = h >= p.side[0].heads;
      if (k) h -= p.side[0].heads;
      const HeadSide& s = p.side[k];
      const T* x = static_cast<const T*>(s.x) + (t0 + t) * s.x_token + h * s.x_head;
      const T* d = static_cast<const T*>(s.dy) + (t0 + t) * s.dy_token + h * s.dy_head;
      T* y = static_cast<T*>(s.y) + ((t0 + t) * s.heads + h) * D;
      const float *cos = angles.cos + t * angles.pitch, *sin = angles.sin + t * angles.pitch;
      auto turned = [&](int i, int a, int b, float& ga, float& gb) {
        ga = to_f32<T>(d[a]), gb = to_f32<T>(d[b]);
        if (i < p.half) {
          const float da = ga, c = cos[i], z = sin[i];
          ga = fmaf(gb, z, da * c);
          gb = fmaf(-da, z, gb * c);
        }
      };
      float r = 1.f, mean = 0.f;
      if (s.w) {
        float sq = 0.f, dot = 0.f;
        for (int i = lane; i < pairs; i += 32) {
          int a, b;
          pair_at(p, i, a, b);
          float ga, gb;
          turned(i, a, b, ga, gb);
          const float xa = to_f32<T>(x[a]), xb = i < p.half ? to_f32<T>(x[b]) : 0.f;
          sq = fmaf(xa, xa, fmaf(xb, xb, sq));
          dot = fmaf(ga * s.w[a], xa, fmaf(gb * s.w[b], xb, dot));
        }
        r = __frsqrt_rn(fmaf(warp_reduce(sq, SumOp()), 1.f / (float)D, p.eps));
        mean = warp_reduce(dot, SumOp()) * r * (1.f / (float)D);
      }
      for (int i = lane; i < pairs; i += 32) {
        int a, b;
        pair_at(p, i, a, b);
        float ga, gb;
        turned(i, a, b, ga, gb);
        if (s.w) {
          const float ua = to_f32<T>(x[a]) * r, ub = to_f32<T>(x[b]) * r;
          own[k * D + a] += ga * ua;
          if (i < p.half) own[k * D + b] += gb * ub;
          ga = (ga * s.w[a] - ua * mean) * r;
          gb = (gb * s.w[b] - ub * mean) * r;
        }
        y[a] = from_f32<T>(ga);
        if (i < p.half) y[b] = from_f32<T>(gb);
      }
    }
  }
  if (!parts) return;
  __syncthreads();
  own -= warp * 2 * D;
  for (int i = threadIdx.x; i < 2 * D; i += kHeadThreads) {
    float v = 0.f;
    for (int w = 0; w < warps; ++w) v += own[w * 2 * D + i];
    parts[(int64_t)blockIdx.x * 2 * D + i] = v;
  }
}

// The blocks' sums joined: 32 columns for each block, its warps each a share
// of the rows in order, then the warps in order.
__global__ void __launch_bounds__(1024) head_norm_join_kernel(const float* parts, int rows, int D, float* dq, float* dk) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (col < 2 * D)
    for (int r = warp; r < rows; r += 32) v += parts[(int64_t)r * 2 * D + col];
  red[warp][lane] = v;
  __syncthreads();
  v = warp_reduce(red[lane][warp], SumOp());
  const int out = blockIdx.x * 32 + warp;
  if (lane == 0 && out < 2 * D) {
    float* to = out < D ? dq : dk;
    if (to) to[out < D ? out : out - D] = v;
  }
}

bool on_16(const void* p, int64_t token, int64_t head, int dtype) {
  const int64_t per = 16 / (int64_t)elem_size(dtype);
  return aligned_to(p, 16) && token % per == 0 && head % per == 0;
}
// Runs of 8 values of both values of each pair, on 16 bytes everywhere.
bool in_runs(const HeadNorm& p) {
  if (p.D % 16 || p.D > 512 || (!p.neighbours && (2 * p.half) % 16)) return false;
  for (const HeadSide& s : p.side)
    if (s.heads && (!on_16(s.x, s.x_token, s.x_head, p.dtype) || !on_16(s.dy, s.dy_token, s.dy_head, p.dtype) ||
                    !aligned_to(s.y, 16) || !aligned_to(s.w, 16)))
      return false;
  return true;
}
int lanes_of(int D) {
  int l = 1;
  while (16 * l < D) l *= 2;
  return l;
}
// Tokens of a tile: eight where that leaves a tile for each of `blocks`, else fewer.
int tile_of(int64_t T, int64_t blocks) {
  int tile = kHeadTile;
  while (tile > 1 && (T + tile - 1) / tile < blocks) tile /= 2;
  return tile;
}

template <class T>
cudaError_t forward_typed(const HeadNorm& p, cudaStream_t stream) {
  const int tile = tile_of(p.T, kHeadBlocks), heads = p.side[0].heads + p.side[1].heads;
  const int64_t tiles = (p.T + tile - 1) / tile;
  const bool runs = in_runs(p);
  const int lanes = runs ? lanes_of(p.D) : 32, teams = kHeadThreads / lanes;
  // Few tokens: their heads over several blocks, which each compute the angles.
  const int64_t rounds = ((int64_t)heads * tile + teams - 1) / teams;
  const int parts = (int)std::max<int64_t>(1, std::min<int64_t>(rounds, kHeadBlocks / tiles));
  const dim3 grid((unsigned)tiles, (unsigned)parts);
  const size_t smem = Angles::bytes(p.half);
  if (!runs)
    head_norm_any_kernel<T><<<grid, kHeadThreads, smem, stream>>>(p, tile);
  else if (p.neighbours)
    head_norm_kernel<T, true><<<grid, kHeadThreads, smem, stream>>>(p, tile, lanes);
  else
    head_norm_kernel<T, false><<<grid, kHeadThreads, smem, stream>>>(p, tile, lanes);
  return cudaGetLastError();
}

template <class K>
cudaError_t room(K kernel, size_t smem) {
  return smem > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) : cudaSuccess;
}

template <class T>
cudaError_t backward_typed(const HeadNorm& p, float* parts, cudaStream_t stream) {
  const int tile = tile_of(p.T, kHeadBlocks);
  const int64_t tiles = (p.T + tile - 1) / tile;
  const unsigned grid = (unsigned)std::min<int64_t>(tiles, kHeadBlocks);
  float* sums = p.side[0].dw || p.side[1].dw ? parts : nullptr;
  cudaError_t e = cudaSuccess;
  if (!in_runs(p)) {
    const size_t smem = Angles::bytes(p.half) + (size_t)(kHeadThreads / 32) * 2 * p.D * 4;
    e = room(head_norm_backward_any_kernel<T>, smem);
    if (e == cudaSuccess) head_norm_backward_any_kernel<T><<<grid, kHeadThreads, smem, stream>>>(p, tile, tiles, sums);
  } else {
    const int lanes = lanes_of(p.D);
    const size_t smem = std::max(Angles::bytes(p.half), (size_t)(kHeadThreads / lanes) * p.D * 4);
    if (p.neighbours)
      head_norm_backward_kernel<T, true><<<grid, kHeadThreads, smem, stream>>>(p, tile, lanes, tiles, sums);
    else
      head_norm_backward_kernel<T, false><<<grid, kHeadThreads, smem, stream>>>(p, tile, lanes, tiles, sums);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess || !sums) return e;
  head_norm_join_kernel<<<(2 * p.D + 31) / 32, 1024, 0, stream>>>(parts, (int)grid, p.D, p.side[0].dw, p.side[1].dw);
  return cudaGetLastError();
}

}  // namespace

size_t head_norm_backward_workspace_bytes(int64_t T, int64_t D) {
  const int tile = tile_of(T, kHeadBlocks);
  return (size_t)std::min<int64_t>((T + tile - 1) / tile, kHeadBlocks) * 2 * D * 4;
}

cudaError_t head_norm_launch(const HeadNorm& p, cudaStream_t stream) {
  switch (p.dtype) {
    case kF32: return forward_typed<float>(p, stream);
    case kF16: return forward_typed<__half>(p, stream);
    default: return forward_typed<__nv_bfloat16>(p, stream);
  }
}

cudaError_t head_norm_backward_launch(const HeadNorm& p, void* ws, cudaStream_t stream) {
  float* parts = static_cast<float*>(ws);
  switch (p.dtype) {
    case kF32: return backward_typed<float>(p, parts, stream);
    case kF16: return backward_typed<__half>(p, parts, stream);
    default: return backward_typed<__nv_bfloat16>(p, parts, stream);
  }
}

}  // namespace bakron
