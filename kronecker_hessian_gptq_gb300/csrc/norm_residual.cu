// norm_residual.cu -- the norms around a block, fused with the block's gate
// and the residual sum, and their backward pass.
//
// Forward, for the residual stream x and the block's output h (T x D):
//     u = N(h; post),  y = alpha x + g * u,  z = N(y; pre),
//     N(v; w, b) = (v - m) rsqrt(mean((v - m)^2) + eps) * w + b,
// m = mean(v) for a layer norm, 0 for an RMS norm; g is one gate row for
// each group of T / groups consecutive tokens.  z is computed from the sum in
// fp32, not from the y that is stored in 16 bits, and is stored as values or
// as 8-bit codes with one scale for each token.
//
// Backward, from y, h and the gradients dy, dz:
//     dt = dy + r_y (k - mean(k) - n_y mean(k n_y)),  k = dz * pre,
//     dx = alpha dt,  dg = sum over the group's tokens of dt * u,
//     du = g * dt,  dh = r_h (q - mean(q) - n_h mean(q n_h)),  q = du * post,
//     dpre = sum_t dz * n_y,  dpost = sum_t du * n_h, biases alike,
// with n = (v - m) r the unit rows and the plain means only for layer norms.
//
// Everything is bound by memory: each thread keeps its part of a row in
// registers, so every input is read once and every output written once.
#include <algorithm>
#include <initializer_list>
#include <utility>

#include "elem.cuh"
#include "layers.h"
#include "quantize_tokens.cuh"

namespace bakron {
namespace {

constexpr int kSms = 152;  // that rows are shared out over: a whole GB300; with fewer, some blocks wait their turn

// Where a thread's 8 N columns of a row lie: vectors of VEC elements at
// (i * stride + t) * VEC, i.e. 16 bytes where rows start on 16 bytes (eight
// 16-bit or twice four 32-bit values), else single elements.
template <class T, int VEC, int N>
struct Columns {
  static constexpr int kV = 8 * N / VEC;
  static constexpr int kWords = 2 * sizeof(T);  // 32-bit words of a Raw8
  int first, step;  // the first vector's column, columns from one vector to the next
  int have;         // vectors within the row
  __device__ __forceinline__ Columns(int t, int stride, int D) : first(t * VEC), step(stride * VEC) {
    have = 0;
#pragma unroll
    for (int i = 0; i < kV; ++i) have += first + i * step < D;
  }
  __device__ __forceinline__ bool in(int i) const { return i < have; }
  __device__ __forceinline__ int64_t col(int i) const { return first + i * step; }
  // Zeros where the row ends, or where there is no array.
  __device__ __forceinline__ void fetch(const T* row, Raw8<T> (&raw)[N]) const {
    auto w = [&](int i) -> uint32_t& { return raw[i / kWords].w[i % kWords]; };
    if constexpr (VEC > 1) {
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (row && in(i)) u = *reinterpret_cast<const uint4*>(row + col(i));
        w(4 * i) = u.x, w(4 * i + 1) = u.y, w(4 * i + 2) = u.z, w(4 * i + 3) = u.w;
      }
    } else {
      constexpr int kW = 4 / sizeof(T);  // elements of a 32-bit word
#pragma unroll
      for (int i = 0; i < kV; i += kW) {
        T e[kW];
#pragma unroll
        for (int k = 0; k < kW; ++k) e[k] = row && in(i + k) ? row[col(i + k)] : from_f32<T>(0.f);
        memcpy(&w(i / kW), e, 4);
      }
    }
  }
  __device__ __forceinline__ void put(T* row, const Raw8<T> (&raw)[N]) const {
    auto w = [&](int i) -> const uint32_t& { return raw[i / kWords].w[i % kWords]; };
    if constexpr (VEC > 1) {
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (in(i)) *reinterpret_cast<uint4*>(row + col(i)) = make_uint4(w(4 * i), w(4 * i + 1), w(4 * i + 2), w(4 * i + 3));
    } else {
      constexpr int kW = 4 / sizeof(T);
#pragma unroll
      for (int i = 0; i < kV; i += kW) {
        T e[kW];
        memcpy(e, &w(i / kW), 4);
#pragma unroll
        for (int k = 0; k < kW; ++k)
          if (in(i + k)) row[col(i + k)] = e[k];
      }
    }
  }
  // The row's columns on their way into shared memory: a vector for each
  // thread and `i`, `threads` vectors apart, zeros where the row ends.
  // (32-bit elements only: the copies are of 4 or 16 bytes.)
  __device__ __forceinline__ void fetch_async(const T* row, T* to, int t, int threads) const {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to + (i * threads + t) * VEC);
      const T* src = in(i) ? row + col(i) : row;
      if constexpr (VEC == 4)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(in(i) ? 16 : 0) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(in(i) ? 4 : 0) : "memory");
    }
  }
  __device__ __forceinline__ void fetched(const T* from, int t, int threads, F2 (&v)[4 * N]) const {
    static_assert(N == 1, "");
    Raw8<T> raw[1];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const T* at = from + (i * threads + t) * VEC;
      if constexpr (VEC == 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(at);
        raw[0].w[4 * i] = u.x, raw[0].w[4 * i + 1] = u.y, raw[0].w[4 * i + 2] = u.z, raw[0].w[4 * i + 3] = u.w;
      } else {
        raw[0].w[i] = *reinterpret_cast<const uint32_t*>(at);
      }
    }
    open8<T>(raw[0], v);
  }
  // The same columns of an fp32 array.
  __device__ __forceinline__ void fetch32(const float* row, float none, F2 (&v)[4 * N]) const {
    float e[8 * N];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      float f[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) f[k] = in(i) ? none : 0.f;
      if (row && in(i)) load_vec<float, VEC>(row + col(i), f);
#pragma unroll
      for (int k = 0; k < VEC; ++k) e[i * VEC + k] = f[k];
    }
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) v[i] = f2(e[2 * i], e[2 * i + 1]);
  }
  __device__ __forceinline__ void put32(float* row, const F2 (&v)[4 * N]) const {
    float e[8 * N];
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) split(v[i], e[2 * i], e[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      float f[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) f[k] = e[i * VEC + k];
      if (in(i)) store_vec<float, VEC>(row + col(i), f);
    }
  }
  // Zeros beyond the row, where something was added to all columns.
  __device__ __forceinline__ void mask(F2 (&v)[4 * N]) const {
    if (have == kV) return;
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) {
      float a, b;
      split(v[i], a, b);
      v[i] = f2(in(2 * i / VEC) ? a : 0.f, in((2 * i + 1) / VEC) ? b : 0.f);
    }
  }
};
template <class T, int N>
__device__ __forceinline__ void open_all(const Raw8<T> (&raw)[N], F2 (&v)[4 * N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) open8<T>(raw[i], *reinterpret_cast<F2(*)[4]>(v + 4 * i));
}
template <class T, int N>
__device__ __forceinline__ void close_all(const F2 (&v)[4 * N], Raw8<T> (&raw)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) close8<T>(*reinterpret_cast<const F2(*)[4]>(v + 4 * i), raw[i]);
}

// A block walks over a range of rows, 8 N columns for each thread, with the
// next row on its way.  kLayer false: RMS norms, whose weights stay in
// registers (with the gate's row multiplied in) where N is 1; else they are
// read again for each row, from the L1 cache.
template <class T, int VEC, int N, bool kLayer, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) norm_residual_kernel(NormResidual p) {
  constexpr int P = 4 * N;  // pairs
  constexpr bool kKeep = !kLayer && N == 1;
  __shared__ float red[128];
  int turn = 0;
  const int D = (int)p.D;
  const float invd = 1.f / (float)D;
  const Columns<T, VEC, N> c(threadIdx.x, blockDim.x, D);
  const int64_t lo = p.T * blockIdx.x / gridDim.x, rows = p.T * (blockIdx.x + 1) / gridDim.x - lo;
  const uint32_t each = (uint32_t)(p.T / p.groups);
  uint32_t group = (uint32_t)lo / each, left = each - (uint32_t)lo % each;  // rows left in the group
  const T* x = static_cast<const T*>(p.X) + lo * p.ldx;
  const T* hin = p.H ? static_cast<const T*>(p.H) + lo * p.ldh : nullptr;
  T* yout = static_cast<T*>(p.Y) + lo * D;
  T* zout = p.Z ? static_cast<T*>(p.Z) + lo * D : nullptr;
  int8_t* codes = p.C ? p.C + lo * D : nullptr;
  // mean and reciprocal deviation; v is left without its mean
  auto stats = [&](F2(&v)[P]) {
    if constexpr (kLayer) {
      F2 s = f2(0.f);
#pragma unroll
      for (int k = 0; k < P; ++k) s = s + v[k];
      const F2 m = f2(-block_one(sum(s), red, turn, SumOp()) * invd);
#pragma unroll
      for (int k = 0; k < P; ++k) v[k] = v[k] + m;
      c.mask(v);
    }
    F2 s = f2(0.f);
#pragma unroll
    for (int k = 0; k < P; ++k) s = fma2(v[k], v[k], s);
    return rsqrtf(fmaf(block_one(sum(s), red, turn, SumOp()), invd, p.eps));
  };
  auto gate_row = [&](F2(&g)[P]) {
    Raw8<T> raw[N];
    c.fetch(static_cast<const T*>(p.gate) + group * p.ldg, raw);
    open_all<T, N>(raw, g);
  };
  F2 kept_post[kKeep ? P : 1], kept_pre[kKeep ? P : 1];
  auto keep_post = [&] {  // the weight times the gate
    if constexpr (kKeep) {
      c.fetch32(p.post, 1.f, kept_post);
      if (p.gate) {
        F2 g[P];
        gate_row(g);
#pragma unroll
        for (int k = 0; k < P; ++k) kept_post[k] = kept_post[k] * g[k];
      }
    }
  };
  if constexpr (kKeep) c.fetch32(p.pre, 1.f, kept_pre);
  keep_post();
  Raw8<T> rx[N], rh[N];
  c.fetch(x, rx);
  c.fetch(hin, rh);
  const F2 alpha = f2(p.alpha);
  for (int64_t i = 0; i < rows; ++i) {
    if (left == 0) {
      ++group;
      left = each;
      if (p.gate) keep_post();
    }
    --left;
    F2 y[P], h[P];
    open_all<T, N>(rx, y);
    open_all<T, N>(rh, h);
    if (i + 1 < rows) {
      x += p.ldx;
      c.fetch(x, rx);
      if (hin) {
        hin += p.ldh;
        c.fetch(hin, rh);
      }
    }
#pragma unroll
    for (int k = 0; k < P; ++k) y[k] = y[k] * alpha;
    if (p.H) {
      const F2 r = f2(p.post ? stats(h) : 1.f);
      if constexpr (kKeep) {
#pragma unroll
        for (int k = 0; k < P; ++k) y[k] = fma2(h[k], r * kept_post[k], y[k]);
      } else {
        if (p.post) {
          F2 w[P];
          c.fetch32(p.post, 1.f, w);
#pragma unroll
          for (int k = 0; k < P; ++k) h[k] = h[k] * (r * w[k]);
        }
        if (kLayer && p.post_bias) {
          F2 w[P];
          c.fetch32(p.post_bias, 0.f, w);
#pragma unroll
          for (int k = 0; k < P; ++k) h[k] = h[k] + w[k];
        }
        if (p.gate) {
          F2 g[P];
          gate_row(g);
#pragma unroll
          for (int k = 0; k < P; ++k) h[k] = h[k] * g[k];
        }
#pragma unroll
        for (int k = 0; k < P; ++k) y[k] = y[k] + h[k];
      }
    }
    {
      Raw8<T> raw[N];
      close_all<T, N>(y, raw);
      c.put(yout, raw);
      yout += D;
    }
    if (!p.pre) continue;
    const F2 r = f2(stats(y));
    if constexpr (kKeep) {
#pragma unroll
      for (int k = 0; k < P; ++k) y[k] = y[k] * (r * kept_pre[k]);
    } else {
      F2 w[P];
      c.fetch32(p.pre, 1.f, w);
#pragma unroll
      for (int k = 0; k < P; ++k) y[k] = y[k] * (r * w[k]);
      if (kLayer && p.pre_bias) {
        c.fetch32(p.pre_bias, 0.f, w);
#pragma unroll
        for (int k = 0; k < P; ++k) y[k] = y[k] + w[k];
      }
    }
    if (zout) {
      Raw8<T> raw[N];
      close_all<T, N>(y, raw);
      c.put(zout, raw);
      zout += D;
      continue;
    }
    float e[2 * P], top = 0.f;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      split(y[k], e[2 * k], e[2 * k + 1]);
      top = MaxOp()(fabsf(e[2 * k]), MaxOp()(fabsf(e[2 * k + 1]), top));
    }
    const float s = token_scale(block_one(top, red, turn, MaxOp())), inv = token_inv(s);
    if (threadIdx.x == 0) p.cs[lo + i] = s;
#pragma unroll
    for (int q = 0; q < Columns<T, VEC, N>::kV; ++q) {
      uint32_t w[VEC > 4 ? 2 : 1] = {};
#pragma unroll
      for (int k = 0; k < VEC; ++k) w[k / 4] |= (uint32_t)(token_code(e[q * VEC + k], s, inv) & 255) << (8 * (k % 4));
      if (!c.in(q)) continue;
      int8_t* to = codes + c.col(q);
      if constexpr (VEC == 8)
        *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
      else if constexpr (VEC == 4)
        *reinterpret_cast<uint32_t*>(to) = w[0];
      else
        *to = (int8_t)w[0];
    }
    codes += D;
  }
}

// Threads for a row: enough for 8 columns each up to 8192 columns, for 16 and
// 32 beyond.  Blocks: as many as fill the SMs, or one for each row.
template <class T, int VEC, bool kLayer>
cudaError_t norm_residual_typed(const NormResidual& p, cudaStream_t stream) {
  const int64_t n = p.D <= 8192 ? 1 : p.D <= 16384 ? 2 : 4;
  const unsigned threads = (unsigned)((p.D + 256 * n - 1) / (256 * n) * 32);
  const unsigned grid = (unsigned)std::min<int64_t>(p.T, (int64_t)kSms * (1024 / threads));
  if (p.D <= 4096)
    norm_residual_kernel<T, VEC, 1, kLayer, 512, 2><<<grid, threads, 0, stream>>>(p);
  else if (n == 1)
    norm_residual_kernel<T, VEC, 1, kLayer, 1024, 1><<<grid, threads, 0, stream>>>(p);
  else if (n == 2)
    norm_residual_kernel<T, VEC, 2, kLayer, 1024, 1><<<grid, threads, 0, stream>>>(p);
  else
    norm_residual_kernel<T, VEC, 4, kLayer, 1024, 1><<<grid, threads, 0, stream>>>(p);
  return cudaGetLastError();
}
template <class T, int VEC>
cudaError_t norm_residual_typed(const NormResidual& p, cudaStream_t stream) {
  return p.layer ? norm_residual_typed<T, VEC, true>(p, stream) : norm_residual_typed<T, VEC, false>(p, stream);
}

// ------------------------------------------------------------------ backward

// Values a column keeps in a block: the weights pre, post and the gate's row,
// the sums of their gradients; the same of the biases.
constexpr int bwd_held(bool layer) { return layer ? 9 : 6; }
constexpr int kBwdSharedBytes = 220 * 1024;  // of a block whose sums are in shared memory, at most
constexpr int kBwdRegisterD = 4096;  // columns up to which they are in registers, 512 threads of 8
constexpr int kBwdPerSm = 8;         // blocks of an SM at most
// Rows on their way in shared memory: of 32-bit elements, whose 32 registers
// for the next row would be spilled as they arrive (1531 x 1999: 47 -> 29 us).
// 16-bit elements come straight into registers (16384 x 4096 in bf16: 173 us,
// 189 through shared memory).
template <class T>
constexpr int kBwdStages = sizeof(T) == 4 ? 2 : 0;

struct BackwardPlan {
  int64_t groups;  // at least 1
  int64_t nb;      // row ranges
  int64_t bpg;     // ranges that share a group; 1 where a range holds whole groups
  int cluster;     // thread blocks that share a row range, each with a part of the columns
  int threads;
  bool shared;
  int smem;
};

BackwardPlan backward_plan(int64_t T, int64_t D, int64_t groups, bool layer, int staged_bytes = 0) {
  BackwardPlan b;
  b.groups = std::max<int64_t>(1, groups);
  b.shared = D > kBwdRegisterD;
  const int64_t each = T / b.groups;
  // columns of a block: 32 bytes of shared memory hold a value for 8 of them
  const int64_t most_cols = !b.shared ? kBwdRegisterD : std::min(1024, kBwdSharedBytes / 32 / bwd_held(layer) / 32 * 32) * 8;
  b.cluster = 1;
  while (b.cluster * most_cols < D) b.cluster *= 2;
  const int64_t per = (D + b.cluster - 1) / b.cluster;
  b.threads = (int)((per + 255) / 256) * 32;
  b.smem = b.shared ? b.threads * 32 * bwd_held(layer) : b.threads * 32 * staged_bytes;
  // ranges that run at once
  const int64_t most = std::max<int64_t>(1, kSms * (b.shared ? 1 : std::min(512 / b.threads, kBwdPerSm)) / b.cluster);
  if (b.groups <= most) {
    b.bpg = std::max<int64_t>(1, std::min(each, most / b.groups));
    b.nb = b.groups * b.bpg;
  } else {
    b.bpg = 1;
    b.nb = most;
  }
  return b;
}

// Sums over the whole cluster's threads.  A cluster barrier separates the
// writes of a use from its reads, and `slot` alternates, so that a block
// writes a slot again only after a later barrier, which every reader of it
// has passed.
template <int N>
__device__ __forceinline__ void cluster_sums(float (&v)[N], float* red, float (*slot)[8], int cluster, int& turn) {
  float* mine = slot[turn];
  block_sums<N>(v, red, turn);
  if (cluster == 1) return;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) mine[k] = v[k];
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(mine);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.f;
  for (int c = 0; c < cluster; ++c) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(remote) : "r"(at), "r"(c));
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float f;
      asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(f) : "r"(remote + 4u * k) : "memory");
      v[k] += f;
    }
  }
}

// Planes of the partial column sums, nb x D fp32 each.
enum Plane { kPost = 0, kPre = 1, kGate = 2, kPostBias = 3, kPreBias = 4, kPlanes = 5 };

// An fp32 value for each of a thread's 8 columns: in registers, or in shared
// memory as two vectors of four that lie `blockDim.x` vectors apart, free of
// bank conflicts.
template <bool kShared>
struct Held {
  F2 v[kShared ? 1 : 4];
  float4* p;
  __device__ __forceinline__ Held(float* base, int which)
      : p(kShared ? reinterpret_cast<float4*>(base) + which * 2 * blockDim.x + threadIdx.x : nullptr) {}
  __device__ __forceinline__ void get(F2 (&x)[4]) const {
    if constexpr (kShared) {
      const float4 a = p[0], b = p[blockDim.x];
      x[0] = f2(a.x, a.y), x[1] = f2(a.z, a.w), x[2] = f2(b.x, b.y), x[3] = f2(b.z, b.w);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = v[k];
    }
  }
  __device__ __forceinline__ void set(const F2 (&x)[4]) {
    if constexpr (kShared) {
      float e[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) split(x[k], e[2 * k], e[2 * k + 1]);
      p[0] = make_float4(e[0], e[1], e[2], e[3]);
      p[blockDim.x] = make_float4(e[4], e[5], e[6], e[7]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = x[k];
    }
  }
  __device__ __forceinline__ void fill(float x) {
    const F2 e[4] = {f2(x), f2(x), f2(x), f2(x)};
    set(e);
  }
  // += a b
  __device__ __forceinline__ void add(const F2 (&a)[4], const F2 (&b)[4]) {
    F2 x[4];
    get(x);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = fma2(a[k], b[k], x[k]);
    set(x);
  }
  __device__ __forceinline__ void add(const F2 (&a)[4]) {
    F2 x[4];
    get(x);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = x[k] + a[k];
    set(x);
  }
};

// A block (or, for the widest rows, a cluster of them) walks over a range of
// rows, 8 columns for each thread, with the next row on its way.  The weights
// and the columns' sums are each thread's own: in registers up to 4096 columns
// (16384 x 4096 in bf16: 168 us; 222 with them in shared memory, which adds
// instructions to a kernel that issues one in 57% of the cycles with 4 warps
// on a scheduler), in shared memory for wider rows, which halves the blocks
// that share a row and wait for one another twice in each (4096 x 14336 in
// bf16: 270 us, 550 with registers).
template <class T, int VEC, bool kLayer, bool kShared>
__global__ void __launch_bounds__(kShared ? 1024 : 512, 1) norm_backward_kernel(NormBackward p, BackwardPlan plan, float* part) {
  extern __shared__ __align__(16) float bwd_smem[];
  __shared__ __align__(16) float red[2 * 256];
  __shared__ float slot[2][8];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  for (int i = threadIdx.x; i < 2 * 256; i += blockDim.x) red[i] = 0.f;
  __syncthreads();
  int turn = 0;
  const int cluster = plan.cluster;
  const int64_t b = blockIdx.x / cluster;
  const int rank = (int)(blockIdx.x % cluster);
  const int D = (int)p.D;
  const float invd = 1.f / (float)D;
  const int64_t each = p.T / plan.groups;
  int64_t lo, hi;
  if (plan.bpg > 1) {
    const int64_t g = b / plan.bpg, j = b % plan.bpg;
    lo = g * each + j * each / plan.bpg;
    hi = g * each + (j + 1) * each / plan.bpg;
  } else {
    lo = b * plan.groups / plan.nb * each;
    hi = (b + 1) * plan.groups / plan.nb * each;
  }
  const Columns<T, VEC, 1> c(rank * (int)blockDim.x + (int)threadIdx.x, cluster * (int)blockDim.x, D);
  Held<kShared> wpre(bwd_smem, 0), wpost(bwd_smem, 1), gate(bwd_smem, 2), apre(bwd_smem, 3), apost(bwd_smem, 4),
      agate(bwd_smem, 5), bpost(bwd_smem, 6), apreb(bwd_smem, 7), apostb(bwd_smem, 8);  // the last three: layer norms only
  {
    F2 v[4];
    c.fetch32(p.pre, 0.f, v);
    wpre.set(v);
    c.fetch32(p.post, 1.f, v);
    wpost.set(v);
    gate.fill(1.f);
    apre.fill(0.f);
    apost.fill(0.f);
    agate.fill(0.f);
    if constexpr (kLayer) {
      apreb.fill(0.f);
      apostb.fill(0.f);
      c.fetch32(p.post_bias, 0.f, v);
      bpost.set(v);
    }
  }
  const T *py = static_cast<const T*>(p.Y) + lo * p.ldy, *ph = p.H ? static_cast<const T*>(p.H) + lo * p.ldh : nullptr;
  const T* pdy = p.dY ? static_cast<const T*>(p.dY) + lo * p.lddy : nullptr;
  const T* pdz = p.dZ ? static_cast<const T*>(p.dZ) + lo * p.lddz : nullptr;
  T *px = static_cast<T*>(p.dX) + lo * D, *pdh = p.dH ? static_cast<T*>(p.dH) + lo * D : nullptr;
  Raw8<T> ry[1], rh[1], rdy[1], rdz[1];
  constexpr int kStages = kShared ? 0 : kBwdStages<T>;
  const int t = (int)threadIdx.x, n = (int)blockDim.x;
  T* const staged = reinterpret_cast<T*>(bwd_smem);
  int stage = 0;
  auto fetch_row = [&] {
    if constexpr (kStages > 0) {
      T* to = staged + stage * 32 * n;
      c.fetch_async(py, to, t, n);
      if (ph) c.fetch_async(ph, to + 8 * n, t, n);
      if (pdy) c.fetch_async(pdy, to + 16 * n, t, n);
      if (pdz) c.fetch_async(pdz, to + 24 * n, t, n);
    } else {
      c.fetch(py, ry);
      c.fetch(ph, rh);
      c.fetch(pdy, rdy);
      c.fetch(pdz, rdz);
    }
  };
  auto advance = [&] {
    py += p.ldy;
    if (ph) ph += p.ldh;
    if (pdy) pdy += p.lddy;
    if (pdz) pdz += p.lddz;
  };
  if constexpr (kStages > 0) {
    for (stage = 0; stage < kStages; ++stage) {
      if (lo + stage < hi) fetch_row();
      asm volatile("cp.async.commit_group;\n" ::: "memory");
      advance();
    }
    stage = 0;
  } else if (lo < hi) {
    fetch_row();
  }
  // A later row into the place of the row at hand, after a barrier of its
  // sums, which follows all reads of that place.
  auto fetch_over = [&](int64_t row) {
    if constexpr (kStages > 0) {
      if (row + kStages < hi) fetch_row();
      asm volatile("cp.async.commit_group;\n" ::: "memory");
      advance();
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
  };
  int64_t group = 0, left = 0;  // rows left in the group
  for (int64_t row = lo; row < hi; ++row) {
    if (left == 0) {
      group = row / each;
      left = (group + 1) * each - row;
      if (p.gate) {
        Raw8<T> g[1];
        F2 v[4];
        c.fetch(static_cast<const T*>(p.gate) + group * p.ldg, g);
        open_all<T, 1>(g, v);
        gate.set(v);
      }
    }
    --left;
    F2 y[4], h[4], dt[4], dz[4];
    if constexpr (kStages > 0) {
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 1) : "memory");
      const T* from = staged + stage * 32 * n;
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = dt[k] = dz[k] = f2(0.f);
      c.fetched(from, t, n, y);
      if (ph) c.fetched(from + 8 * n, t, n, h);
      if (pdy) c.fetched(from + 16 * n, t, n, dt);
      if (pdz) c.fetched(from + 24 * n, t, n, dz);
    } else {
      open_all<T, 1>(ry, y);
      open_all<T, 1>(rh, h);
      open_all<T, 1>(rdy, dt);
      open_all<T, 1>(rdz, dz);
      if (row + 1 < hi) {
        advance();
        fetch_row();
      }
    }
    if constexpr (kLayer) {
      F2 sy = f2(0.f), sh = f2(0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) sy = sy + y[k], sh = sh + h[k];
      float s[2] = {sum(sy), sum(sh)};
      cluster_sums<2>(s, red, slot, cluster, turn);
      const F2 my = f2(-s[0] * invd), mh = f2(p.post ? -s[1] * invd : 0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = y[k] + my, h[k] = h[k] + mh;
      c.mask(y);
      c.mask(h);
      if (p.dZ) apreb.add(dz);
    }
    // One exchange for all sums of a row where that pays: with q = g * post,
    // mean(q dt n_h) is linear in dt = dy + r_y k + c n_y, whose c comes from
    // the same exchange (16384 x 4096 in bf16: 168 us, 173 with two).  Layer
    // norms would need four sums more; the wide form has no registers left
    // for it (4096 x 14336: 270 us, 328 with one exchange).
    constexpr bool kOne = !kLayer && !kShared;
    float s[kOne ? 6 : 4];
    F2 w[4];
    wpre.get(w);
    {
      F2 yy = f2(0.f), qy = f2(0.f), hh = f2(0.f), qq = f2(0.f), hd = f2(0.f), hk = f2(0.f), hy = f2(0.f);
      F2 q[4];
      if constexpr (kOne) {
        wpost.get(q);
        if (p.gate) {
          F2 g[4];
          gate.get(g);
#pragma unroll
          for (int k = 0; k < 4; ++k) q[k] = q[k] * g[k];
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[k] = dz[k] * w[k];
        yy = fma2(y[k], y[k], yy);
        qy = fma2(w[k], y[k], qy);
        hh = fma2(h[k], h[k], hh);
        if constexpr (kLayer) qq = qq + w[k];
        if constexpr (kOne) {
          q[k] = q[k] * h[k];
          hd = fma2(q[k], dt[k], hd);
          hk = fma2(q[k], w[k], hk);
          hy = fma2(q[k], y[k], hy);
        }
      }
      s[0] = sum(yy), s[1] = sum(qy), s[2] = sum(hh);
      if constexpr (!kOne)
        s[3] = kLayer ? sum(qq) : 0.f;
      else
        s[3] = sum(hd), s[4] = sum(hk), s[5] = sum(hy);
    }
    cluster_sums<kOne ? 6 : 4>(s, red, slot, cluster, turn);
    fetch_over(row);
    if (p.dZ) {
      const float r = rsqrtf(fmaf(s[0], invd, p.eps));
      const float cn = -r * r * s[1] * invd;
      const F2 r2 = f2(r), c1 = f2(cn), c0 = f2(kLayer ? -r * s[3] * invd : 0.f);
      if constexpr (kOne) s[3] = fmaf(cn * r, s[5], fmaf(r, s[4], s[3]));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        y[k] = y[k] * r2;
        dt[k] = fma2(y[k], c1, fma2(w[k], r2, dt[k]));
        if constexpr (kLayer) dt[k] = dt[k] + c0;
      }
      apre.add(dz, y);
      if constexpr (kLayer) c.mask(dt);
    }
    Raw8<T> out[1];
    {
      F2 dx[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) dx[k] = dt[k] * f2(p.alpha);
      close_all<T, 1>(dx, out);
      c.put(px, out);
      px += D;
    }
    if (!p.H) continue;
    const float r = p.post ? rsqrtf(fmaf(s[2], invd, p.eps)) : 1.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = h[k] * f2(r);  // the unit row
    wpost.get(w);
    if (p.dgate) {
      F2 u[4];
      if constexpr (kLayer) {
        bpost.get(u);
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = fma2(h[k], w[k], u[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = h[k] * w[k];
      }
      agate.add(dt, u);
    }
    if (p.gate) {
      F2 g[4];
      gate.get(g);
#pragma unroll
      for (int k = 0; k < 4; ++k) dt[k] = dt[k] * g[k];
    }
    if (p.post) {
      apost.add(dt, h);
      if constexpr (kLayer) apostb.add(dt);
      float t[2] = {s[3] * r, 0.f};
      F2 tn = f2(0.f), tq = f2(0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dt[k] = dt[k] * w[k];
        if constexpr (!kOne) tn = fma2(dt[k], h[k], tn);
        if constexpr (kLayer) tq = tq + dt[k];
      }
      if constexpr (!kOne) {
        t[0] = sum(tn), t[1] = kLayer ? sum(tq) : 0.f;
        cluster_sums<2>(t, red, slot, cluster, turn);
      }
      const F2 c1 = f2(-t[0] * invd * r), c0 = f2(-t[1] * invd * r);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dt[k] = fma2(h[k], c1, dt[k] * f2(r));
        if constexpr (kLayer) dt[k] = dt[k] + c0;
      }
    }
    close_all<T, 1>(dt, out);
    c.put(pdh, out);
    pdh += D;
    if (p.dgate && left == 0 && plan.bpg == 1) {  // this range holds the whole group
      F2 v[4];
      agate.get(v);
      c.put32(p.dgate + group * p.D, v);
      agate.fill(0.f);
    }
  }
  const int64_t plane = plan.nb * p.D;
  float* mine = part + b * p.D;
  auto put = [&](const float* want, const Held<kShared>& from, int q) {
    if (!want) return;
    F2 v[4];
    from.get(v);
    c.put32(mine + q * plane, v);
  };
  put(p.dpost, apost, kPost);
  put(p.dpre, apre, kPre);
  put(plan.bpg > 1 ? p.dgate : nullptr, agate, kGate);
  if constexpr (kLayer) {
    put(p.dpost_bias, apostb, kPostBias);
    put(p.dpre_bias, apreb, kPreBias);
  }
  if (cluster > 1)  // the others may still read this block's slots
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// Sums the ranges' partial rows in a fixed order: 32 columns for each block,
// 32 threads for each column.
struct ColumnSums {
  float* out[kPlanes];
  const float* part;
  int64_t nb, bpg, D;
  int first[kPlanes + 1];  // blockIdx.y of a plane's first output row
};
__global__ void __launch_bounds__(1024) column_sums_kernel(ColumnSums a) {
  __shared__ float red[32][33];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // it may have been launched before the rows were done
  const int row = (int)blockIdx.y;
  int q = 0, first = 0;
  float* out = a.out[0];
#pragma unroll
  for (int k = 1; k < kPlanes; ++k)
    if (row >= a.first[k]) q = k, first = a.first[k], out = a.out[k];
  const int64_t r = row - first;
  const int n = (int)(q == kGate ? a.bpg : a.nb);
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < a.D) {
    const float* x = a.part + (q * a.nb + (q == kGate ? r * a.bpg : 0) + threadIdx.y) * a.D + c;
#pragma unroll 4
    for (int i = threadIdx.y; i < n; i += 32, x += 32 * a.D) s += *x;
  }
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  // a warp for each column, a lane for each of its threads' sums
  s = warp_reduce(red[threadIdx.x][threadIdx.y], SumOp());
  const int64_t to = (int64_t)blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && to < a.D) out[r * a.D + to] = s;
}

template <class T, int VEC>
cudaError_t norm_backward_typed(const NormBackward& p, float* part, cudaStream_t stream) {
  const BackwardPlan plan = backward_plan(p.T, p.D, p.groups, p.layer, kBwdStages<T> * (int)sizeof(T));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(plan.nb * plan.cluster));
  cfg.blockDim = dim3((unsigned)plan.threads);
  cfg.dynamicSmemBytes = (size_t)plan.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)plan.cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = plan.shared ? (p.layer ? norm_backward_kernel<T, VEC, true, true> : norm_backward_kernel<T, VEC, false, true>)
                            : (p.layer ? norm_backward_kernel<T, VEC, true, false> : norm_backward_kernel<T, VEC, false, false>);
  // What the kernel may take at most, whatever the width: threads that set their own would lower each other's.
  const int most = plan.shared ? kBwdSharedBytes : kBwdRegisterD / 8 * 32 * kBwdStages<T> * (int)sizeof(T);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, kernel, p, plan, part);
  if (e != cudaSuccess) return e;
  ColumnSums a = {};
  a.part = part;
  a.nb = plan.nb, a.bpg = plan.bpg, a.D = p.D;
  float* outs[kPlanes] = {p.dpost, p.dpre, plan.bpg > 1 ? p.dgate : nullptr, p.dpost_bias, p.dpre_bias};
  int rows = 0;
  for (int q = 0; q < kPlanes; ++q) {
    a.out[q] = outs[q];
    a.first[q] = rows;
    if (outs[q]) rows += q == kGate ? (int)plan.groups : 1;
  }
  a.first[kPlanes] = rows;
  if (!rows) return cudaSuccess;
  cfg.gridDim = dim3((unsigned)((p.D + 31) / 32), (unsigned)rows);
  cfg.blockDim = dim3(32, 32);
  cfg.dynamicSmemBytes = 0;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, column_sums_kernel, a);
}

// Vectors of 16 bytes where every row of every array starts on 16 bytes and
// the width is a whole number of them, else single elements.
bool vectors(int dtype, int64_t D, std::initializer_list<std::pair<const void*, int64_t>> arrays) {
  const int64_t v = 16 / (int64_t)elem_size(dtype);
  if (D % v) return false;
  for (const auto& a : arrays)
    if (a.first && (!aligned_to(a.first, 16) || a.second % v)) return false;
  return true;
}

bool on16(std::initializer_list<const float*> weights) {
  for (const float* w : weights)
    if (!aligned_to(w, 16)) return false;
  return true;
}

}  // namespace

cudaError_t norm_residual_launch(const NormResidual& p, cudaStream_t stream) {
  const bool vec = vectors(p.dtype, p.D, {{p.X, p.ldx}, {p.H, p.ldh}, {p.gate, p.ldg}, {p.Y, p.D}, {p.Z, p.D}}) &&
                   (!p.C || aligned_to(p.C, 8)) && on16({p.post, p.post_bias, p.pre, p.pre_bias});
  switch (p.dtype) {
    case kF32: return vec ? norm_residual_typed<float, 4>(p, stream) : norm_residual_typed<float, 1>(p, stream);
    case kF16: return vec ? norm_residual_typed<__half, 8>(p, stream) : norm_residual_typed<__half, 1>(p, stream);
    default:
      return vec ? norm_residual_typed<__nv_bfloat16, 8>(p, stream) : norm_residual_typed<__nv_bfloat16, 1>(p, stream);
  }
}

size_t norm_backward_workspace_bytes(int64_t T, int64_t D, int64_t groups) {
  return (size_t)kPlanes * std::max(backward_plan(T, D, groups, false).nb, backward_plan(T, D, groups, true).nb) * D * 4;
}

cudaError_t norm_backward_launch(const NormBackward& p, void* ws, cudaStream_t stream) {
  const bool vec = vectors(p.dtype, p.D, {{p.dY, p.lddy}, {p.dZ, p.lddz}, {p.Y, p.ldy}, {p.H, p.ldh}, {p.gate, p.ldg},
                                          {p.dX, p.D}, {p.dH, p.D}}) &&
                   on16({p.post, p.post_bias, p.pre, p.dpost, p.dpost_bias, p.dgate, p.dpre, p.dpre_bias});
  float* part = static_cast<float*>(ws);
  switch (p.dtype) {
    case kF32: return vec ? norm_backward_typed<float, 4>(p, part, stream) : norm_backward_typed<float, 1>(p, part, stream);
    case kF16: return vec ? norm_backward_typed<__half, 8>(p, part, stream) : norm_backward_typed<__half, 1>(p, part, stream);
    default:
      return vec ? norm_backward_typed<__nv_bfloat16, 8>(p, part, stream)
                 : norm_backward_typed<__nv_bfloat16, 1>(p, part, stream);
  }
}

}  // namespace bakron
