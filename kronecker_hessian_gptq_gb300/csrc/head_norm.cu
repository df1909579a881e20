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
// 16 values a lane in two runs of 8 (or half as many in runs of 4), so that both values of a pair are the
// same lane's, and a head's sums take three exchanges for D = 128.  A block
// takes a tile of tokens: their angles are computed once, into shared memory, for
// the 40 or so heads, and a team keeps to one token and goes from head to head.
// The next heads' values are on their way meanwhile.  bf16, 32 and 8 heads of 128:
// 16384 tokens take 63 us (5.3 TB/s), backward 105 us (4.8 TB/s; with three blocks on
// an SM in place of two, and so 80 registers and spills, 20 us more).  What
// is not in such runs, or not on 16 bytes, takes a warp a head.
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
constexpr int kHeadBlocks = 4 * 152;  // forward: four on each SM
constexpr int kBackBlocks = 4 * 152;  // backward: at most
constexpr int kBackTile = 32;
// Dynamic shared memory that a block of any kernel here may take.  The most is that
// of the backward pass for any sizes, with 1024 values, all turned, in tiles of a
// token a warp: 512 turns, 8 rows of 512 angles, and each warp's 1024 sums, 68 KB.
constexpr size_t kHeadSmem = 68 * 1024;

// The frequency f as a share of a turn for each position, 2^-64 of it.
__device__ __forceinline__ uint64_t turn_of(double f) {
  const double t = fabs(f) * 0.15915494309189533577;  // 1 / 2 pi
  const double part = t - floor(t);                   // exact
  const uint64_t share = part < 1.0 ? (uint64_t)(part * 18446744073709551616.0) : 0ull;  // 0 for a NaN
  return f < 0.0 ? 0ull - share : share;
}
// cos and sin of 2 pi times the share: the nearest quarter turn is taken off
// in integers, and for the at most an eighth of a turn that is left, x, Taylor's
// series to x^10, whose next terms are below 2^-29.
__device__ __forceinline__ void cos_sin(uint64_t share, float& c, float& s) {
  const uint32_t v = (uint32_t)(share >> 32), quarter = (v + 0x20000000u) >> 30;
  const float x = (float)(int)(v - (quarter << 30)) * 1.4629180792671596e-9f, y = x * x;  // 2 pi 2^-32
  const float b = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
  const float a = fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
  const uint32_t cos = __float_as_uint(quarter & 1 ? b : a), sin = __float_as_uint(quarter & 1 ? a : b);
  c = __uint_as_float(cos ^ ((quarter + 1 & 2) << 30));
  s = __uint_as_float(sin ^ ((quarter & 2) << 30));
}

// Shared memory of a block: the turns of each frequency, and cos and sin for
// each token of a tile (rows of `pitch` floats).
struct Angles {
  uint64_t* turn;
  float *cos, *sin;
  int pitch;
  static __host__ __device__ int pitch_of(int half) { return (half + 7) / 8 * 8; }
  static __host__ __device__ size_t bytes(int half, int tile) { return (size_t)pitch_of(half) * (8 + 2 * 4 * tile); }
  bool eights;
  // Where the angle of frequency k lies in its row: for lanes that read eight, the
  // first four of each eight, then the last four of each, so that neighbouring
  // lanes' 16 bytes are neighbours.
  __device__ __forceinline__ int place(int k) const { return eights ? (k >> 2 & 1) * (pitch / 2) + (k >> 3) * 4 + (k & 3) : k; }
  __device__ Angles(unsigned char* smem, int half, int tile, bool eights) : pitch(pitch_of(half)), eights(eights) {
    turn = reinterpret_cast<uint64_t*>(smem);
    cos = reinterpret_cast<float*>(smem + 8 * pitch);
    sin = cos + pitch * tile;
  }
};
// A frequency that is not finite turns nothing into numbers.  A thread keeps to
// one frequency, or a few, and walks over the tokens.
__device__ __forceinline__ void fill_turns(const HeadNorm& p, const Angles& a) {
  for (int i = threadIdx.x; i < p.half; i += kHeadThreads) a.turn[i] = turn_of(p.freqs[i]);
}
// The angles of so many tokens into the rows from `to` on.
__device__ __forceinline__ void fill_angles(const HeadNorm& p, const Angles& a, const int64_t* positions, int tokens, int to = 0) {
  const int wide = p.half < kHeadThreads ? p.half : kHeadThreads, rows = kHeadThreads / wide;
  const int row = threadIdx.x / wide, col = threadIdx.x - row * wide;
  if (row >= rows) return;
  for (int k = col; k < p.half; k += wide) {
    const uint64_t turn = a.turn[k];
    const bool finite = isfinite(p.freqs[k]);
    for (int t = row; t < tokens; t += rows) {
      float c, s;
      cos_sin((uint64_t)positions[t] * turn, c, s);
      a.cos[(to + t) * a.pitch + a.place(k)] = finite ? c : __int_as_float(0x7fffffff);
      a.sin[(to + t) * a.pitch + a.place(k)] = finite ? s : __int_as_float(0x7fffffff);
    }
  }
}

// kRun consecutive values of a lane as they lie in memory: 8, 16 or 32 bytes.
template <class T, int kRun>
struct Run {
  static constexpr int kWords = kRun * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 2) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x, w[1] = u.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[i / 4];
        w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void open(F2 (&v)[kRun / 2]) const {
#pragma unroll
    for (int i = 0; i < kRun / 2; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
      } else {
        T e[2];
        memcpy(e, &w[i], 4);
        v[i] = f2(to_f32<T>(e[0]), to_f32<T>(e[1]));
      }
    }
  }
};
template <class T, int kPairs>
__device__ __forceinline__ void store_run(T* p, const F2 (&v)[kPairs]) {
  constexpr int kWords = kPairs * (int)sizeof(T) / 2;
  uint32_t w[kWords];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    float a, b;
    split(v[i], a, b);
    if constexpr (sizeof(T) == 4)
      w[2 * i] = __float_as_uint(a), w[2 * i + 1] = __float_as_uint(b);
    else
      w[i] = pack2<T>(a, b);
  }
  if constexpr (kWords == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < kWords; i += 4) reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}
template <int kPairs>
__device__ __forceinline__ void load_f2(const float* p, F2 (&v)[kPairs]) {
#pragma unroll
  for (int i = 0; i < kPairs; i += 2) {
    const float4 f = reinterpret_cast<const float4*>(p)[i / 2];
    v[i] = f2(f.x, f.y), v[i + 1] = f2(f.z, f.w);
  }
}

// A lane's values: two runs, from lo and from hi on.
struct Place {
  int lo, hi;
  int angle;  // of lo's first pair
};
template <bool kNeighbours, int kRun>
__device__ __forceinline__ Place place_of(int j, int rotated) {
  if (!kNeighbours && 2 * kRun * j < rotated) return Place{kRun * j, rotated / 2 + kRun * j, kRun * j};
  return Place{2 * kRun * j, 2 * kRun * j + kRun, kRun * j};
}

// kRun angles' cosines or sines from a row of Angles, from the first of such a run on.
template <int kRun>
__device__ __forceinline__ void load_angles(const float* row, int angle, int pitch, float (&v)[kRun]) {
#pragma unroll
  for (int i = 0; i < kRun; i += 4) {
    const float4 f = *reinterpret_cast<const float4*>(row + (kRun == 8 ? angle / 2 + i / 4 * (pitch / 2) : angle));
    v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
  }
}
// Turns a lane's pairs by their angles, or back (kBack).
template <bool kNeighbours, bool kBack, int kPairs>
__device__ __forceinline__ void turn_pairs(F2 (&a)[kPairs], F2 (&b)[kPairs], const float* cos, const float* sin, int angle, int half,
                                           int pitch) {
  constexpr int kRun = 2 * kPairs;
  if (angle >= half) return;
  float c[kRun], s[kRun];
  load_angles<kRun>(cos, angle, pitch, c);
  load_angles<kRun>(sin, angle, pitch, s);
  if (!kNeighbours) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const F2 cc = f2(c[2 * i], c[2 * i + 1]), ss = f2(s[2 * i], s[2 * i + 1]), minus = f2(-s[2 * i], -s[2 * i + 1]);
      const F2 x = a[i], y = b[i];
      a[i] = fma2(y, kBack ? ss : minus, x * cc);
      b[i] = fma2(x, kBack ? minus : ss, y * cc);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (angle + i >= half) break;
      F2& v = i < kPairs ? a[i % kPairs] : b[i % kPairs];
      float x, y;
      split(v, x, y);
      v = kBack ? f2(fmaf(y, s[i], x * c[i]), fmaf(-x, s[i], y * c[i])) : f2(fmaf(-y, s[i], x * c[i]), fmaf(x, s[i], y * c[i]));
    }
  }
}

__device__ __forceinline__ float team_sum(float v, int lanes) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    if (o >= lanes) break;
    v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}
template <int kPairs>
__device__ __forceinline__ float squares(const F2 (&a)[kPairs], const F2 (&b)[kPairs]) {
  F2 q = a[0] * a[0];
#pragma unroll
  for (int i = 1; i < kPairs; ++i) q = fma2(a[i], a[i], q);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) q = fma2(b[i], b[i], q);
  return sum(q);
}

// Blocks of a variant that an SM holds at a time.
template <class T, int kRun>
__host__ __device__ constexpr int forward_on_sm() { return kRun == 4 ? (sizeof(T) == 2 ? 5 : 4) : sizeof(T) == 2 ? 4 : 3; }
template <class T, int kRun>
__host__ __device__ constexpr int backward_on_sm() { return kRun == 4 ? (sizeof(T) == 2 ? 4 : 3) : 2; }

// A team takes one token of a tile and every `step`-th of its heads; two heads are
// on their way at a time, from one tile into the next, and so are the next tile's
// angles.
template <class T, bool kNeighbours, int kRun>
__global__ void __launch_bounds__(kHeadThreads, forward_on_sm<T, kRun>())
    head_norm_kernel(const __grid_constant__ HeadNorm p, int tile_log, int lanes, int tiles) {
  extern __shared__ __align__(16) unsigned char head_smem[];
  const int tile = 1 << tile_log;
  const Angles angles(head_smem, p.half, 2 * tile, kRun == 8);  // of two tiles in turn
  const int j = threadIdx.x & (lanes - 1), team = threadIdx.x / lanes, each = (kHeadThreads / lanes) >> tile_log;
  const int t = team & (tile - 1), slot = team >> tile_log, first = (int)blockIdx.y * each, step = each * gridDim.y;
  const bool mine = 2 * kRun * j < p.D;
  const Place at = place_of<kNeighbours, kRun>(j, 2 * p.half);
  const float share = 1.f / (float)p.D;
  const int queries = p.side[0].heads, heads = queries + p.side[1].heads;
  Run<T, kRun> lo[2] = {}, hi[2] = {};
  int ahead_q = blockIdx.x, ahead = first;  // what is fetched next
  auto fetch = [&](int n) {
    const int64_t token = ((int64_t)ahead_q << tile_log) + t;
    const int h = ahead + slot;
    if (mine && token < p.T && h < heads) {  // else what is there is not used, or zeros behind a head's end
      const HeadSide& s = p.side[h >= queries];
      const T* x = static_cast<const T*>(s.x) + token * s.x_token + (h < queries ? h : h - queries) * s.x_head;
      lo[n].load(x + at.lo);
      hi[n].load(x + at.hi);
    }
    ahead += step;
    if (ahead >= heads) ahead = first, ahead_q += gridDim.x;
  };
  auto fill = [&](int q, int buf) {
    if (!p.half || q >= tiles) return;
    const int64_t t0 = (int64_t)q << tile_log;
    const int tokens = (int)(p.T - t0 < tile ? p.T - t0 : tile);
    fill_angles(p, angles, p.positions + t0, tokens, buf * tile);
  };
  int q = blockIdx.x, base = first, buf = 0;
  fetch(0);
  if (ahead_q < tiles) fetch(1);
  if (p.half) {
    fill_turns(p, angles);
    __syncthreads();
    fill(q, 0);
  }
  // All teams take the same number of turns: the exchanges are the whole warp's.
  while (q < tiles) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      if (q >= tiles) break;
      if (base == first && p.half) {
        __syncthreads();  // this tile's angles are there, the one's before are read
        fill(q + gridDim.x, buf ^ 1);
      }
      F2 a[kRun / 2], b[kRun / 2];
      lo[n].open(a);
      hi[n].open(b);
      if (ahead_q < tiles) fetch(n);
      const int64_t token = ((int64_t)q << tile_log) + t;
      const int h = base + slot;
      const HeadSide& s = p.side[h >= queries];
      const float r = rsqrtf(fmaf(team_sum(squares(a, b), lanes), share, p.eps));
      if (mine && token < p.T && h < heads) {
        if (s.w) {
          F2 w[kRun / 2];
          load_f2(s.w + at.lo, w);
#pragma unroll
          for (int i = 0; i < kRun / 2; ++i) a[i] = a[i] * f2(r) * w[i];
          load_f2(s.w + at.hi, w);
#pragma unroll
          for (int i = 0; i < kRun / 2; ++i) b[i] = b[i] * f2(r) * w[i];
        }
        const int row = (buf * tile + t) * angles.pitch;
        turn_pairs<kNeighbours, false>(a, b, angles.cos + row, angles.sin + row, at.angle, p.half, angles.pitch);
        T* y = static_cast<T*>(s.y) + (token * s.heads + (h < queries ? h : h - queries)) * p.D;
        store_run(y + at.lo, a);
        store_run(y + at.hi, b);
      }
      base += step;
      if (base >= heads) base = first, q += gridDim.x, buf ^= 1;
    }
  }
}

// Any sizes, strides and alignment: a warp for each head.  Pair i of the head
// (i < half), then its single values.
__device__ __forceinline__ void pair_at(const HeadNorm& p, int i, int& a, int& b) {
  if (i >= p.half) {
    a = b = p.half + i;
  } else if (p.neighbours) {
    a = 2 * i, b = a + 1;
  } else {
    a = i, b = i + p.half;
  }
}

// kN: a lane holds its kN pairs (there are 32 kN at most), and the next head's
// are on their way; 0: it reads them again.
template <class T, int kN>
__global__ void __launch_bounds__(kHeadThreads) head_norm_any_kernel(const __grid_constant__ HeadNorm p, int tile_log) {
  extern __shared__ __align__(16) unsigned char head_smem[];
  const int tile = 1 << tile_log;
  const Angles angles(head_smem, p.half, tile, false);
  const int64_t t0 = (int64_t)blockIdx.x << tile_log;
  const int tokens = (int)(p.T - t0 < tile ? p.T - t0 : tile);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, queries = p.side[0].heads, heads = queries + p.side[1].heads;
  const int t = warp & (tile - 1), each = (kHeadThreads / 32) >> tile_log, step = each * gridDim.y, D = p.D, pairs = D - p.half;
  auto input = [&](int h) {
    const HeadSide& s = p.side[h >= queries];
    return static_cast<const T*>(s.x) + (t0 + t) * s.x_token + (h < queries ? h : h - queries) * s.x_head;
  };
  constexpr int kRoom = kN ? kN : 1;
  T na[kRoom], nb[kRoom];
  auto fetch = [&](int h) {
    if (t >= tokens || h >= heads) return;
    const T* x = input(h);
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int i = lane + 32 * n;
      int a, b;
      pair_at(p, i, a, b);
      na[n] = i < pairs ? x[a] : from_f32<T>(0.f);
      nb[n] = i < p.half ? x[b] : from_f32<T>(0.f);
    }
  };
  int h = (int)blockIdx.y * each + (warp >> tile_log);
  if (kN) fetch(h);
  if (p.half) {
    fill_turns(p, angles);
    __syncthreads();
    fill_angles(p, angles, p.positions + t0, tokens);
    __syncthreads();
  }
  if (t >= tokens) return;
  const float *cos = angles.cos + t * angles.pitch, *sin = angles.sin + t * angles.pitch;
  auto write = [&](T* y, int i, float va, float vb, float r, const float* w) {
    int a, b;
    pair_at(p, i, a, b);
    if (w) va = va * r * w[a], vb = vb * r * w[b];
    if (i < p.half) {
      const float c = cos[angles.place(i)], z = sin[angles.place(i)];
      y[a] = from_f32<T>(fmaf(-vb, z, va * c));
      y[b] = from_f32<T>(fmaf(va, z, vb * c));
    } else {
      y[a] = from_f32<T>(va);
    }
  };
  for (; h < heads; h += step) {
    const HeadSide& s = p.side[h >= queries];
    T* y = static_cast<T*>(s.y) + ((t0 + t) * s.heads + (h < queries ? h : h - queries)) * D;
    float r = 1.f, q = 0.f;
    if constexpr (kN > 0) {
      float va[kN], vb[kN];
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        va[n] = to_f32<T>(na[n]), vb[n] = to_f32<T>(nb[n]);
        q = fmaf(va[n], va[n], fmaf(vb[n], vb[n], q));
      }
      fetch(h + step);
      if (s.w) r = rsqrtf(fmaf(warp_reduce(q, SumOp()), 1.f / (float)D, p.eps));
#pragma unroll
      for (int n = 0; n < kN; ++n)
        if (lane + 32 * n < pairs) write(y, lane + 32 * n, va[n], vb[n], r, s.w);
    } else {
      const T* x = input(h);
      if (s.w) {
        for (int i = lane; i < D; i += 32) {
          const float v = to_f32<T>(x[i]);
          q = fmaf(v, v, q);
        }
        r = rsqrtf(fmaf(warp_reduce(q, SumOp()), 1.f / (float)D, p.eps));
      }
      for (int i = lane; i < pairs; i += 32) {
        int a, b;
        pair_at(p, i, a, b);
        write(y, i, to_f32<T>(x[a]), to_f32<T>(x[b]), r, s.w);
      }
    }
  }
}

// ------------------------------------------------------------ backward

// The blocks are shared out between queries and keys: the first blocks[0] walk
// over the queries' tiles, the others over the keys', which have tiles of their
// own.  So a block sums one weight's gradient, in registers, and leaves D
// floats in `parts`.  In runs the next tile's angles are computed behind this one's heads.
struct HeadPlan {
  int tile_log[2], blocks[2];
  int64_t tiles[2];
};

template <class T, bool kNeighbours, int kRun>
__global__ void __launch_bounds__(kHeadThreads, backward_on_sm<T, kRun>())
    head_norm_backward_kernel(const __grid_constant__ HeadNorm p, const __grid_constant__ HeadPlan plan, int lanes, float* parts) {
  extern __shared__ __align__(16) unsigned char head_smem[];
  const int k = (int)blockIdx.x >= plan.blocks[0], tile_log = plan.tile_log[k], tile = 1 << tile_log;
  const HeadSide& s = p.side[k];
  const Angles angles(head_smem, p.half, 2 * tile, kRun == 8);  // of two tiles in turn
  const int j = threadIdx.x & (lanes - 1), team = threadIdx.x / lanes, step = (kHeadThreads / lanes) >> tile_log;
  const int t = team & (tile - 1), slot = team >> tile_log, heads = s.heads;
  const bool mine = 2 * kRun * j < p.D, normed = s.w;
  const Place at = place_of<kNeighbours, kRun>(j, 2 * p.half);
  const float share = 1.f / (float)p.D;
  const int64_t tiles = plan.tiles[k];
  const int stride = plan.blocks[k];
  int64_t q = k ? (int)blockIdx.x - plan.blocks[0] : (int)blockIdx.x;
  const T *dy = static_cast<const T*>(s.dy), *xs = static_cast<const T*>(s.x);
  Run<T, kRun> raw[4] = {};
  auto fetch = [&](int64_t q, int h) {
    const int64_t token = (q << tile_log) + t;
    if (!mine || token >= p.T || h >= heads) return;  // what is there is not used, or zeros behind a head's end
    const T* d = dy + token * s.dy_token + h * s.dy_head;
    raw[0].load(d + at.lo);
    raw[1].load(d + at.hi);
    if (normed) {
      const T* v = xs + token * s.x_token + h * s.x_head;
      raw[2].load(v + at.lo);
      raw[3].load(v + at.hi);
    }
  };
  F2 dw[kRun];
#pragma unroll
  for (int i = 0; i < kRun; ++i) dw[i] = f2(0.f);
  auto tokens_of = [&](int64_t q) { return (int)(p.T - (q << tile_log) < tile ? p.T - (q << tile_log) : tile); };
  fetch(q, slot);
  // Positions are read a tile before their angles are computed.
  __shared__ int64_t positions[2][kBackTile];
  auto position = [&](int64_t q) {
    const int64_t token = (q << tile_log) + threadIdx.x;
    return p.half && (int)threadIdx.x < tile && token < p.T ? p.positions[token] : 0;
  };
  if (p.half) {
    if ((int)threadIdx.x < tile) positions[0][threadIdx.x] = position(q), positions[1][threadIdx.x] = position(q + stride);
    fill_turns(p, angles);
    __syncthreads();
    if (q < tiles) fill_angles(p, angles, positions[0], tokens_of(q));
  }
  for (int buf = 0; q < tiles; q += stride, buf ^= 1) {
    const int64_t t0 = q << tile_log;
    const int tokens = tokens_of(q);
    if (p.half) {
      __syncthreads();  // this tile's angles are there, the one's before are read
      if (q + stride < tiles) fill_angles(p, angles, positions[buf ^ 1], tokens_of(q + stride), (buf ^ 1) * tile);
    }
    const int64_t later = position(q + 2 * stride);
    const float *cos = angles.cos + (buf * tile + t) * angles.pitch, *sin = angles.sin + (buf * tile + t) * angles.pitch;
    T* out = static_cast<T*>(s.y) + (t0 + t) * heads * p.D;
    for (int base = 0; base < heads; base += step) {
      const int h = base + slot;
      const bool live = t < tokens && h < heads;
      F2 g[kRun], x[kRun];
      constexpr int kPairs = kRun / 2;
      F2(&ga)[kPairs] = *reinterpret_cast<F2(*)[kPairs]>(g), (&gb)[kPairs] = *reinterpret_cast<F2(*)[kPairs]>(g + kPairs);
      F2(&xa)[kPairs] = *reinterpret_cast<F2(*)[kPairs]>(x), (&xb)[kPairs] = *reinterpret_cast<F2(*)[kPairs]>(x + kPairs);
      raw[0].open(ga);
      raw[1].open(gb);
      raw[2].open(xa);
      raw[3].open(xb);
      if (base + step < heads)
        fetch(q, h + step);
      else
        fetch(q + stride, slot);
      if (mine) turn_pairs<kNeighbours, true>(ga, gb, cos, sin, at.angle, p.half, angles.pitch);
      if (normed) {
        const float r = rsqrtf(fmaf(team_sum(squares(xa, xb), lanes), share, p.eps));
        F2 dot = f2(0.f);
        if (mine) {
          F2 w[kRun];
          load_f2(s.w + at.lo, *reinterpret_cast<F2(*)[kPairs]>(w));
          load_f2(s.w + at.hi, *reinterpret_cast<F2(*)[kPairs]>(w + kPairs));
#pragma unroll
          for (int i = 0; i < kRun; ++i) {
            x[i] = x[i] * f2(r);
            if (live) dw[i] = fma2(g[i], x[i], dw[i]);
            g[i] = g[i] * w[i];
            dot = fma2(g[i], x[i], dot);
          }
        }
        const float c = -team_sum(sum(dot), lanes) * share;
#pragma unroll
        for (int i = 0; i < kRun; ++i) g[i] = fma2(x[i], f2(c), g[i]) * f2(r);
      }
      if (live && mine) {
        T* y = out + h * p.D;
        store_run(y + at.lo, ga);
        store_run(y + at.hi, gb);
      }
    }
    // (All have read this tile's: its angles were computed before the barrier above.)
    if (p.half && (int)threadIdx.x < tile) positions[buf][threadIdx.x] = later;
  }
  asm volatile("griddepcontrol.launch_dependents;\n");
  if (!parts) return;
  // The teams' sums one after another, in their order.
  __syncthreads();
  float* all = reinterpret_cast<float*>(head_smem);  // teams x D
  if (mine) {
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      float a, b;
      split(dw[i], a, b);
      const int e = (i < kRun / 2 ? at.lo : at.hi) + 2 * (i % (kRun / 2));
      all[team * p.D + e] = a;
      all[team * p.D + e + 1] = b;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.D; e += kHeadThreads) {
    float v = 0.f;
    for (int i = 0; i < kHeadThreads / lanes; ++i) v += all[i * p.D + e];
    parts[(int64_t)blockIdx.x * p.D + e] = v;
  }
}

// As forward: a lane holds its kN pairs, with the next head's on their way, or
// (0) reads them again and keeps the weight's gradient in shared memory.
template <class T, int kN>
__global__ void __launch_bounds__(kHeadThreads) head_norm_backward_any_kernel(const __grid_constant__ HeadNorm p,
                                                                              const __grid_constant__ HeadPlan plan, float* parts) {
  extern __shared__ __align__(16) unsigned char head_smem[];
  const int k = (int)blockIdx.x >= plan.blocks[0], tile_log = plan.tile_log[k], tile = 1 << tile_log;
  const HeadSide& s = p.side[k];
  const Angles angles(head_smem, p.half, tile, false);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kHeadThreads / 32, D = p.D, pairs = D - p.half;
  const int t = warp & (tile - 1), slot = warp >> tile_log, step = warps >> tile_log, heads = s.heads;
  // each warp's sums: D floats
  float* own = reinterpret_cast<float*>(head_smem + Angles::bytes(p.half, tile)) + warp * D;
  for (int i = lane; i < D; i += 32) own[i] = 0.f;
  constexpr int kRoom = kN ? kN : 1;
  T da[kRoom], db[kRoom], xa[kRoom], xb[kRoom];
  float wa[kRoom], wb[kRoom];
#pragma unroll
  for (int n = 0; n < kRoom; ++n) wa[n] = wb[n] = 0.f;
  const int64_t tiles = plan.tiles[k];
  const int stride = plan.blocks[k];
  int64_t q = k ? (int)blockIdx.x - plan.blocks[0] : (int)blockIdx.x;
  auto gradient = [&](int64_t token, int h) { return static_cast<const T*>(s.dy) + token * s.dy_token + h * s.dy_head; };
  auto input = [&](int64_t token, int h) { return static_cast<const T*>(s.x) + token * s.x_token + h * s.x_head; };
  auto fetch = [&](int64_t q, int h) {
    const int64_t token = (q << tile_log) + t;
    if (token >= p.T || h >= heads) return;
    const T *d = gradient(token, h), *x = s.w ? input(token, h) : d;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int i = lane + 32 * n;
      int a, b;
      pair_at(p, i, a, b);
      const bool in = i < pairs, two = i < p.half;
      da[n] = in ? d[a] : from_f32<T>(0.f), db[n] = two ? d[b] : from_f32<T>(0.f);
      xa[n] = in ? x[a] : from_f32<T>(0.f), xb[n] = two ? x[b] : from_f32<T>(0.f);
    }
  };
  if (kN) fetch(q, slot);
  if (p.half) fill_turns(p, angles);
  const float *cos = angles.cos + t * angles.pitch, *sin = angles.sin + t * angles.pitch;
  auto back = [&](int i, float& ga, float& gb) {
    if (i >= p.half) return;
    const float d = ga, c = cos[angles.place(i)], z = sin[angles.place(i)];
    ga = fmaf(gb, z, d * c);
    gb = fmaf(-d, z, gb * c);
  };
  for (; q < tiles; q += stride) {
    const int64_t t0 = q << tile_log;
    const int tokens = (int)(p.T - t0 < tile ? p.T - t0 : tile);
    if (p.half) {
      __syncthreads();
      fill_angles(p, angles, p.positions + t0, tokens);
      __syncthreads();
    }
    for (int h = slot; h < heads; h += step) {
      T* y = static_cast<T*>(s.y) + ((t0 + t) * heads + h) * D;
      if constexpr (kN > 0) {
        float ga[kN], gb[kN], ua[kN], ub[kN], sq = 0.f, dot = 0.f;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          ga[n] = to_f32<T>(da[n]), gb[n] = to_f32<T>(db[n]);
          ua[n] = to_f32<T>(xa[n]), ub[n] = to_f32<T>(xb[n]);
        }
        if (h + step < heads)
          fetch(q, h + step);
        else
          fetch(q + stride, slot);
        if (t >= tokens) continue;
        float r = 1.f, mean = 0.f;
        if (s.w) {
#pragma unroll
          for (int n = 0; n < kN; ++n) sq = fmaf(ua[n], ua[n], fmaf(ub[n], ub[n], sq));
          r = rsqrtf(fmaf(warp_reduce(sq, SumOp()), 1.f / (float)D, p.eps));
        }
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          const int i = lane + 32 * n;
          if (i >= pairs) break;
          back(i, ga[n], gb[n]);
          if (!s.w) continue;
          int a, b;
          pair_at(p, i, a, b);
          ua[n] *= r, ub[n] *= r;
          wa[n] = fmaf(ga[n], ua[n], wa[n]), wb[n] = fmaf(gb[n], ub[n], wb[n]);
          ga[n] *= s.w[a], gb[n] *= s.w[b];
          dot = fmaf(ga[n], ua[n], fmaf(gb[n], ub[n], dot));
        }
        if (s.w) mean = warp_reduce(dot, SumOp()) * (1.f / (float)D);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          const int i = lane + 32 * n;
          if (i >= pairs) break;
          int a, b;
          pair_at(p, i, a, b);
          y[a] = from_f32<T>(s.w ? (ga[n] - ua[n] * mean) * r : ga[n]);
          if (i < p.half) y[b] = from_f32<T>(s.w ? (gb[n] - ub[n] * mean) * r : gb[n]);
        }
      } else {
        if (t >= tokens) continue;
        const T *d = gradient(t0 + t, h), *x = s.w ? input(t0 + t, h) : d;
        float r = 1.f, mean = 0.f;
        if (s.w) {
          float sq = 0.f, dot = 0.f;
          for (int i = lane; i < pairs; i += 32) {
            int a, b;
            pair_at(p, i, a, b);
            float ga = to_f32<T>(d[a]), gb = to_f32<T>(d[b]);
            back(i, ga, gb);
            const float va = to_f32<T>(x[a]), vb = i < p.half ? to_f32<T>(x[b]) : 0.f;
            sq = fmaf(va, va, fmaf(vb, vb, sq));
            dot = fmaf(ga * s.w[a], va, fmaf(gb * s.w[b], vb, dot));
          }
          r = rsqrtf(fmaf(warp_reduce(sq, SumOp()), 1.f / (float)D, p.eps));
          mean = warp_reduce(dot, SumOp()) * r * (1.f / (float)D);
        }
        for (int i = lane; i < pairs; i += 32) {
          int a, b;
          pair_at(p, i, a, b);
          float ga = to_f32<T>(d[a]), gb = to_f32<T>(d[b]);
          back(i, ga, gb);
          if (s.w) {
            const float va = to_f32<T>(x[a]) * r, vb = to_f32<T>(x[b]) * r;
            own[a] += ga * va;
            if (i < p.half) own[b] += gb * vb;
            ga = (ga * s.w[a] - va * mean) * r;
            gb = (gb * s.w[b] - vb * mean) * r;
          }
          y[a] = from_f32<T>(ga);
          if (i < p.half) y[b] = from_f32<T>(gb);
        }
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;\n");
  if (!parts) return;
  if constexpr (kN > 0) {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int i = lane + 32 * n;
      if (i >= pairs) break;
      int a, b;
      pair_at(p, i, a, b);
      own[a] = wa[n];
      if (i < p.half) own[b] = wb[n];
    }
  }
  __syncthreads();
  own -= warp * D;
  for (int i = threadIdx.x; i < D; i += kHeadThreads) {
    float v = 0.f;
    for (int w = 0; w < warps; ++w) v += own[w * D + i];
    parts[(int64_t)blockIdx.x * D + i] = v;
  }
}

// The blocks' sums joined: 32 columns of a side for each block, its warps each a
// share of the rows in order, then the warps in order.
__global__ void __launch_bounds__(1024) head_norm_join_kernel(const float* parts, int queries, int keys, int D, float* dq, float* dk) {
  __shared__ float red[32][33];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  const int rows = blockIdx.y ? keys : queries;
  const float* from = parts + (blockIdx.y ? (int64_t)queries * D : 0);
  float v = 0.f;
  if (col < D) {
#pragma unroll 8
    for (int r = warp; r < rows; r += 32) v += from[(int64_t)r * D + col];
  }
  red[warp][lane] = v;
  __syncthreads();
  v = warp_reduce(red[lane][warp], SumOp());
  const int out = blockIdx.x * 32 + warp;
  float* to = blockIdx.y ? dk : dq;
  if (lane == 0 && out < D && to) to[out] = v;
}

bool on_run(const void* p, int64_t token, int64_t head, int dtype, int run) {
  const int64_t bytes = std::min<int64_t>(16, run * (int64_t)elem_size(dtype)), per = bytes / (int64_t)elem_size(dtype);
  return aligned_to(p, bytes) && token % per == 0 && head % per == 0;
}
// Runs of so many values of both values of each pair, at addresses that allow them.
bool in_runs(const HeadNorm& p, int run) {
  if (p.D % (2 * run) || p.D > 64 * run || (!p.neighbours && p.half % run)) return false;
  for (const HeadSide& s : p.side)
    if (s.heads && (!on_run(s.x, s.x_token, s.x_head, p.dtype, run) || !on_run(s.dy, s.dy_token, s.dy_head, p.dtype, run) ||
                    !on_run(s.y, 0, 0, p.dtype, run) || !aligned_to(s.w, 16)))
      return false;
  return true;
}
// Runs of 8 or 4 values, or 0: none.  In 16 bits 8 where they fit, 16 bytes a lane (with 4 the heads of 8192 tokens take 61 us
// for 34, their gradients 85 for 56); in fp32 4 are 16 bytes (4096 tokens, 12 heads of 256: 21.6 us for 24.8, gradients 31.7 for 32.7).
int run_of(const HeadNorm& p) {
  const int first = p.dtype == kF32 ? 4 : 8;
  return in_runs(p, first) ? first : in_runs(p, 12 - first) ? 12 - first : 0;
}
int lanes_of(int D, int run) {
  int l = 1;
  while (2 * run * l < D) l *= 2;
  return l;
}
int log_of(int n) {
  int l = 0;
  while ((1 << (l + 1)) <= n) ++l;
  return l;
}
// Tokens of a tile: eight where that leaves a tile for each of `blocks`, else fewer.
int tile_log_of(int64_t T, int64_t blocks) {
  int l = log_of(kHeadTile);
  while (l && (T + (1 << l) - 1) >> l < blocks) --l;
  return l;
}
int pairs_of(const HeadNorm& p) { return p.D - p.half; }

template <class T>
cudaError_t forward_typed(const HeadNorm& p, cudaStream_t stream) {
  const int run = run_of(p);
  const bool runs = run != 0;
  // In runs half as many tiles as blocks fit are enough: a block's start takes as long as a tile (1024 tokens, 40 heads
  // of 128: 7.2 us, with a tile for each 8.5; any sizes, 4096 tokens, 16 heads of 77: 20.7 and 18.3).
  const int tile_log = tile_log_of(p.T, runs ? kHeadBlocks / 2 : kHeadBlocks), heads = p.side[0].heads + p.side[1].heads;
  const int64_t tiles = (p.T + (1 << tile_log) - 1) >> tile_log;
  const int lanes = runs ? lanes_of(p.D, run) : 32, each = (kHeadThreads / lanes) >> tile_log;
  // Few tokens: their heads over several blocks, which each compute the angles.
  const int parts = (int)std::max<int64_t>(1, std::min<int64_t>((heads + each - 1) / each, kHeadBlocks / tiles));
  const dim3 grid((unsigned)tiles, (unsigned)parts);
  const size_t smem = Angles::bytes(p.half, 1 << tile_log);
  // In runs, with fewer than eight heads for a team: no more blocks than the SMs hold at a time, each with as many
  // tiles as any other or one less, so that one's start is behind another's heads (16384 tokens, 2 heads of 64: 9.4 us,
  // else 11.5).  With more a tile is a block, and the SMs share them out (16384 tokens, 40 heads of 128: 64 us, else 75).
  const bool few = runs && heads < 8 * each;
  const int64_t most = few ? 152 * (run == 4 ? forward_on_sm<T, 4>() : forward_on_sm<T, 8>()) : tiles, rounds = (tiles + most - 1) / most;
  const dim3 walk((unsigned)((tiles + rounds - 1) / rounds), (unsigned)parts);
  const size_t both = Angles::bytes(p.half, 2 << tile_log);
  const int pairs = pairs_of(p);
  auto go = [&](auto kernel) { kernel<<<walk, kHeadThreads, both, stream>>>(p, tile_log, lanes, (int)tiles); };
  if (run == 8)
    p.neighbours ? go(head_norm_kernel<T, true, 8>) : go(head_norm_kernel<T, false, 8>);
  else if (run == 4)
    p.neighbours ? go(head_norm_kernel<T, true, 4>) : go(head_norm_kernel<T, false, 4>);
  else if (pairs <= 32)
    head_norm_any_kernel<T, 1><<<grid, kHeadThreads, smem, stream>>>(p, tile_log);
  else if (pairs <= 64)
    head_norm_any_kernel<T, 2><<<grid, kHeadThreads, smem, stream>>>(p, tile_log);
  else if (pairs <= 128)
    head_norm_any_kernel<T, 4><<<grid, kHeadThreads, smem, stream>>>(p, tile_log);
  else
    head_norm_any_kernel<T, 0><<<grid, kHeadThreads, smem, stream>>>(p, tile_log);
  return cudaGetLastError();
}

// A side's tiles: of so many tokens that a team, of which a block has `teams`, has four heads
// of one between two barriers, and fewer where there would be less than a tile for a third of its blocks.  A
// block takes as many tiles as any other, or one less.
void plan_side(HeadPlan& plan, int k, int64_t T, int heads, int teams, int blocks) {
  if (heads == 0 || blocks == 0) return;
  int l = 0;
  while ((2 << l) <= std::min(teams, kBackTile) && ((int64_t)heads << (l + 1)) <= 4 * teams) ++l;
  while (l && (T + (1 << l) - 1) >> l < (blocks + 2) / 3) --l;
  plan.tile_log[k] = l;
  plan.tiles[k] = (T + (1 << l) - 1) >> l;
  const int64_t rounds = (plan.tiles[k] + blocks - 1) / blocks;
  plan.blocks[k] = (int)((plan.tiles[k] + rounds - 1) / rounds);
}
HeadPlan backward_plan(const HeadNorm& p, int teams, int blocks, bool runs) {
  HeadPlan plan = {};
  // A token's angles cost a side about as much as two of its heads.
  const int64_t hq = p.side[0].heads, hk = p.side[1].heads, more = p.half && runs ? 2 : 0;
  const int64_t share = (blocks * (hq + more) + (hq + hk) / 2 + more) / (hq + hk + 2 * more);
  const int queries = hk == 0 ? blocks : hq == 0 ? 0 : (int)std::min<int64_t>(blocks - 1, std::max<int64_t>(1, share));
  plan_side(plan, 0, p.T, (int)hq, teams, queries);
  plan_side(plan, 1, p.T, (int)hk, teams, blocks - queries);
  return plan;
}

template <class T>
cudaError_t backward_typed(const HeadNorm& p, float* parts, cudaStream_t stream) {
  const int run = run_of(p);
  const bool runs = run != 0;
  const int lanes = runs ? lanes_of(p.D, run) : 32, teams = kHeadThreads / lanes;
  const int pairs = pairs_of(p);
  // As many blocks as fit on the SMs at a time: their registers decide.
  const int on_sm = run == 8 ? backward_on_sm<T, 8>() : run == 4 ? backward_on_sm<T, 4>() : pairs > 64 && pairs <= 128 ? 2 : 4;
  const HeadPlan plan = backward_plan(p, teams, 152 * on_sm, runs);
  const unsigned grid = (unsigned)(plan.blocks[0] + plan.blocks[1]);
  float* sums = p.side[0].dw || p.side[1].dw ? parts : nullptr;
  const size_t angles = Angles::bytes(p.half, (runs ? 2 : 1) << std::max(plan.tile_log[0], plan.tile_log[1]));
  const size_t smem = runs ? std::max(angles, (size_t)teams * p.D * 4) : angles + (size_t)teams * p.D * 4;
  cudaError_t e = cudaSuccess;
  auto go = [&](auto kernel, auto... more) {
    // One bound for every call: it is the kernel's, and threads that set their own would lower each other's.
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kHeadSmem);
    if (e == cudaSuccess) kernel<<<grid, kHeadThreads, smem, stream>>>(p, plan, more..., sums);
    if (e == cudaSuccess) e = cudaGetLastError();
  };
  if (run == 8)
    p.neighbours ? go(head_norm_backward_kernel<T, true, 8>, lanes) : go(head_norm_backward_kernel<T, false, 8>, lanes);
  else if (run == 4)
    p.neighbours ? go(head_norm_backward_kernel<T, true, 4>, lanes) : go(head_norm_backward_kernel<T, false, 4>, lanes);
  else if (pairs <= 32)
    go(head_norm_backward_any_kernel<T, 1>);
  else if (pairs <= 64)
    go(head_norm_backward_any_kernel<T, 2>);
  else if (pairs <= 128)
    go(head_norm_backward_any_kernel<T, 4>);
  else
    go(head_norm_backward_any_kernel<T, 0>);
  if (e != cudaSuccess || !sums) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.D + 31) / 32, 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, head_norm_join_kernel, (const float*)parts, plan.blocks[0], plan.blocks[1], p.D, p.side[0].dw,
                            p.side[1].dw);
}

}  // namespace

size_t head_norm_backward_workspace_bytes(int64_t T, int64_t D) {
  return (size_t)std::min<int64_t>(2 * T, kBackBlocks) * D * 4;
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
