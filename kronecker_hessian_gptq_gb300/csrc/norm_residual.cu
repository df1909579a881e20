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

constexpr int kSms = 152;

// A block walks over rows with the next one on its way: thread t holds the NV
// vectors of VEC elements at columns (i * blockDim.x + t) * VEC.  kKeep: the
// weights stay in registers (RMS norms, 8 elements for each thread), else they
// are read again for each row, from the L1 cache.
template <class T, int VEC, int NV, int kThreads, int kBlocks, bool kKeep>
__global__ void __launch_bounds__(kThreads, kBlocks) norm_residual_kernel(NormResidual p) {
  constexpr int E = VEC * NV;
  __shared__ float red[128];
  int turn = 0;
  const int D = (int)p.D;
  const float invd = 1.f / (float)D;
  const int64_t each = p.T / p.groups;
  int col[NV];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = (i * (int)blockDim.x + (int)threadIdx.x) * VEC;
    in[i] = col[i] < D;
  }
  struct Raw {
    T e[E];
  };
  auto fetch = [&](const void* base, int64_t at, Raw& raw) {
    const T* r = static_cast<const T*>(base) + at;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (VEC * sizeof(T) == 16) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (base && in[i]) u = *reinterpret_cast<const uint4*>(r + col[i]);
        memcpy(raw.e + i * VEC, &u, 16);
      } else {
        raw.e[i] = base && in[i] ? r[col[i]] : from_f32<T>(0.f);
      }
    }
  };
  auto param = [&](const float* w, int i, float none, float(&v)[VEC]) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = none;
    if (w && in[i]) load_vec<float, VEC>(w + col[i], v);
  };
  // mean and reciprocal deviation of the row held in v
  auto stats = [&](const float(&v)[E], float& m, float& r) {
    m = 0.f;
    if (!kKeep && p.layer) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < E; ++k) s += v[k];
      m = block_one(s, red, turn, SumOp()) * invd;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (kKeep || in[i]) {  // without a mean the zeros beyond the row add nothing
#pragma unroll
        for (int k = 0; k < VEC; ++k) s = fmaf(v[i * VEC + k] - m, v[i * VEC + k] - m, s);
      }
    r = rsqrtf(fmaf(block_one(s, red, turn, SumOp()), invd, p.eps));
  };
  float kept_post[NV][VEC], kept_pre[NV][VEC];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      param(p.post, i, 1.f, kept_post[i]);
      param(p.pre, i, 1.f, kept_pre[i]);
    }
  }
  Raw rx, rh;
  fetch(p.X, blockIdx.x * p.ldx, rx);
  fetch(p.H, blockIdx.x * p.ldh, rh);
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    float y[E], h[E];
#pragma unroll
    for (int k = 0; k < E; ++k) y[k] = to_f32<T>(rx.e[k]), h[k] = to_f32<T>(rh.e[k]);
    if (row + gridDim.x < p.T) {
      fetch(p.X, (row + gridDim.x) * p.ldx, rx);
      fetch(p.H, (row + gridDim.x) * p.ldh, rh);
    }
    if (p.H) {
      Raw gate;
      if (p.gate) fetch(p.gate, (row / each) * p.ldg, gate);
      float m = 0.f, r = 1.f;
      if (p.post) stats(h, m, r);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float w[VEC], b[VEC];
        if constexpr (!kKeep) {
          param(p.post, i, 1.f, w);
          param(p.post_bias, i, 0.f, b);
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const int e = i * VEC + k;
          float u = kKeep ? h[e] * r * kept_post[i][k] : fmaf((h[e] - m) * r, w[k], b[k]);
          if (p.gate) u *= to_f32<T>(gate.e[e]);
          y[e] = fmaf(p.alpha, y[e], u);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) y[k] *= p.alpha;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float e[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        if (!kKeep && !in[i]) y[i * VEC + k] = 0.f;  // a bias may have come in
        e[k] = y[i * VEC + k];
      }
      if (in[i]) store_vec<T, VEC>(static_cast<T*>(p.Y) + row * D + col[i], e);
    }
    if (!p.pre) continue;
    float m, r;
    stats(y, m, r);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float e[VEC], w[VEC], b[VEC];
      if constexpr (!kKeep) {
        param(p.pre, i, 1.f, w);
        param(p.pre_bias, i, 0.f, b);
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        e[k] = kKeep ? y[i * VEC + k] * r * kept_pre[i][k] : fmaf((y[i * VEC + k] - m) * r, w[k], b[k]);
        y[i * VEC + k] = e[k];
        if (in[i]) top = MaxOp()(fabsf(e[k]), top);
      }
      if (!p.C && in[i]) store_vec<T, VEC>(static_cast<T*>(p.Z) + row * D + col[i], e);
    }
    if (!p.C) continue;
    const float s = token_scale(block_one(top, red, turn, MaxOp())), inv = token_inv(s);
    if (threadIdx.x == 0) p.cs[row] = s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      int8_t* to = p.C + row * D + col[i];
      uint32_t w[VEC > 4 ? 2 : 1] = {};
#pragma unroll
      for (int k = 0; k < VEC; ++k) w[k / 4] |= (uint32_t)(token_code(y[i * VEC + k], s, inv) & 255) << (8 * (k % 4));
      if constexpr (VEC == 8)
        *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
      else if constexpr (VEC == 4)
        *reinterpret_cast<uint32_t*>(to) = w[0];
      else
        *to = (int8_t)w[0];
    }
  }
}

// Threads for a row: enough for 8 elements each up to 8192 columns, for 16 and
// 32 beyond.  Blocks: as many as fill the SMs, or one for each row.
template <class T, int VEC>
cudaError_t norm_residual_typed(const NormResidual& p, cudaStream_t stream) {
  const int64_t nvec = (p.D + VEC - 1) / VEC;
  constexpr int kUnit = 8 / VEC;  // vectors that make up 8 elements
  const int64_t per = p.D <= 8192 ? kUnit : p.D <= 16384 ? 2 * kUnit : 4 * kUnit;
  const int64_t threads = std::max<int64_t>(1, (nvec + 32 * per - 1) / (32 * per)) * 32;
  const unsigned grid = (unsigned)std::min<int64_t>(p.T, (int64_t)kSms * (1024 / threads));
  if (p.D <= 4096 && !p.layer)
    norm_residual_kernel<T, VEC, kUnit, 512, 2, true><<<grid, (unsigned)threads, 0, stream>>>(p);
  else if (p.D <= 8192 && !p.layer)
    norm_residual_kernel<T, VEC, kUnit, 1024, 1, true><<<grid, (unsigned)threads, 0, stream>>>(p);
  else if (p.D <= 8192)
    norm_residual_kernel<T, VEC, kUnit, 1024, 1, false><<<grid, (unsigned)threads, 0, stream>>>(p);
  else if (p.D <= 16384)
    norm_residual_kernel<T, VEC, 2 * kUnit, 1024, 1, false><<<grid, (unsigned)threads, 0, stream>>>(p);
  else
    norm_residual_kernel<T, VEC, 4 * kUnit, 1024, 1, false><<<grid, (unsigned)threads, 0, stream>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ backward

constexpr int kBwdThreads = 512;  // 8 elements each: 4096 columns for one block of a cluster

struct BackwardPlan {
  int64_t groups;  // at least 1
  int64_t nb;      // row ranges
  int64_t bpg;     // ranges that share a group; 1 where a range holds whole groups
  int cluster;     // thread blocks that share a row range, each with a part of the columns
  int threads;
};

BackwardPlan backward_plan(int64_t T, int64_t D, int64_t groups) {
  BackwardPlan b;
  b.groups = std::max<int64_t>(1, groups);
  const int64_t each = T / b.groups;
  b.cluster = 1;
  while ((int64_t)b.cluster * kBwdThreads * 8 < D) b.cluster *= 2;
  const int64_t per = (D + b.cluster - 1) / b.cluster;
  b.threads = (int)std::max<int64_t>(1, (per + 255) / 256) * 32;
  const int64_t most = std::max<int64_t>(1, kSms * (kBwdThreads / b.threads) / b.cluster);  // that run at once
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
__device__ __forceinline__ void cluster_sums(float (&v)[N], float* red, float (*slot)[4], int cluster, int& turn) {
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

// A block (or, for wide rows, a cluster of them) walks over a range of rows
// with the weights and the columns' sums in registers: 8 columns for each
// thread.  The next row is on its way while one is worked on; 16 warps with
// 128 registers fill an SM, and nothing else would cover the loads.
template <class T, int VEC, bool kLayer>
__global__ void __launch_bounds__(kBwdThreads, 1) norm_backward_kernel(NormBackward p, BackwardPlan plan, float* part) {
  constexpr int E = 8, NV = 8 / VEC;
  __shared__ float red[2 * 64];
  __shared__ float slot[2][4];
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
  int col[NV];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = ((i * cluster + rank) * (int)blockDim.x + (int)threadIdx.x) * VEC;
    in[i] = col[i] < D;
  }
  // A thread's part of a row as it comes: 16-byte vectors, or single elements.
  struct Raw {
    T e[E];
  };
  auto fetch = [&](const void* base, int64_t at, Raw& raw) {
    const T* r = static_cast<const T*>(base) + at;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (VEC * sizeof(T) == 16) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (base && in[i]) u = *reinterpret_cast<const uint4*>(r + col[i]);
        memcpy(raw.e + i * VEC, &u, 16);
      } else {
        raw.e[i] = base && in[i] ? r[col[i]] : from_f32<T>(0.f);
      }
    }
  };
  auto open = [&](const Raw& raw, float(&v)[E]) {
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] = to_f32<T>(raw.e[k]);
  };
  auto store = [&](void* base, int64_t at, const float(&v)[E]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float e[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) e[k] = v[i * VEC + k];
      if (in[i]) store_vec<T, VEC>(static_cast<T*>(base) + at + col[i], e);
    }
  };
  auto param = [&](const float* w, float none, float(&v)[E]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float e[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) e[k] = in[i] ? none : 0.f;
      if (in[i] && w) load_vec<float, VEC>(w + col[i], e);
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[i * VEC + k] = e[k];
    }
  };
  auto put = [&](float* to, const float(&v)[E]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float e[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) e[k] = v[i * VEC + k];
      if (in[i]) store_vec<float, VEC>(to + col[i], e);
    }
  };
  const bool masked = !in[NV - 1];  // some columns are beyond the row: their values are zeros
  float wpre[E], wpost[E], bpost[kLayer ? E : 1], gt[E];
  param(p.pre, 0.f, wpre);
  param(p.post, 1.f, wpost);
  if constexpr (kLayer) param(p.post_bias, 0.f, bpost);
#pragma unroll
  for (int k = 0; k < E; ++k) gt[k] = 1.f;
  float apost[E], apre[E], agate[E], apostb[kLayer ? E : 1], apreb[kLayer ? E : 1];
#pragma unroll
  for (int k = 0; k < E; ++k) apost[k] = apre[k] = agate[k] = 0.f;
  if constexpr (kLayer) {
#pragma unroll
    for (int k = 0; k < E; ++k) apostb[k] = apreb[k] = 0.f;
  }
  Raw ry, rh, rdy, rdz;
  auto fetch_row = [&](int64_t row) {
    if (row >= hi) return;
    fetch(p.Y, row * p.ldy, ry);
    fetch(p.H, row * p.ldh, rh);
    fetch(p.dY, row * p.lddy, rdy);
    fetch(p.dZ, row * p.lddz, rdz);
  };
  fetch_row(lo);
  int64_t group = lo < hi ? lo / each : 0, left = 0;  // rows left in the group
  for (int64_t row = lo; row < hi; ++row) {
    if (left == 0) {
      group = row / each;
      left = (group + 1) * each - row;
      if (p.gate) {
        Raw g;
        fetch(p.gate, group * p.ldg, g);
        open(g, gt);
      }
    }
    --left;
    float y[E], h[E], dt[E], dz[E];
    open(ry, y);
    open(rh, h);
    open(rdy, dt);
    open(rdz, dz);
    fetch_row(row + 1);
    if constexpr (kLayer) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < E; ++k) s[0] += y[k], s[1] += h[k];
      cluster_sums<2>(s, red, slot, cluster, turn);
      const float my = s[0] * invd, mh = p.post ? s[1] * invd : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          if (masked && !in[i]) continue;
          y[i * VEC + k] -= my;
          h[i * VEC + k] -= mh;
        }
    }
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float q = dz[k] * wpre[k];
      s[0] = fmaf(y[k], y[k], s[0]);
      s[1] = fmaf(q, y[k], s[1]);
      s[2] = fmaf(h[k], h[k], s[2]);
      if (kLayer) s[3] += q;
    }
    cluster_sums<4>(s, red, slot, cluster, turn);
    if (p.dZ) {
      const float r = rsqrtf(fmaf(s[0], invd, p.eps)), c1 = r * r * r * s[1] * invd, c0 = r * s[3] * invd;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float n = y[k] * r;
        dt[k] += r * (dz[k] * wpre[k]) - (kLayer ? c0 : 0.f) - c1 * y[k];
        apre[k] = fmaf(dz[k], n, apre[k]);
        if constexpr (kLayer) apreb[k] += dz[k];
      }
    }
    {
      float dx[E];
#pragma unroll
      for (int k = 0; k < E; ++k) dx[k] = p.alpha * dt[k];
      store(p.dX, row * p.D, dx);
    }
    if (!p.H) continue;
    const float r = p.post ? rsqrtf(fmaf(s[2], invd, p.eps)) : 1.f;
    float t[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int k = i * VEC + e;
        if (masked && !in[i]) dt[k] = 0.f;
        const float n = h[k] * r;
        float u = n * wpost[k];
        if constexpr (kLayer) u += bpost[k];
        agate[k] = fmaf(dt[k], u, agate[k]);
        const float du = dt[k] * gt[k];
        apost[k] = fmaf(du, n, apost[k]);
        if constexpr (kLayer) apostb[k] += du;
        dt[k] = du * wpost[k];
        t[0] = fmaf(dt[k], n, t[0]);
        if (kLayer) t[1] += dt[k];
      }
    if (p.post) {
      cluster_sums<2>(t, red, slot, cluster, turn);
      const float c1 = t[0] * invd * r * r, c0 = kLayer ? t[1] * invd * r : 0.f;
#pragma unroll
      for (int k = 0; k < E; ++k) dt[k] = r * dt[k] - c0 - c1 * h[k];
    }
    store(p.dH, row * p.D, dt);
    if (p.dgate && left == 0 && plan.bpg == 1) {  // this range holds the whole group
      put(p.dgate + group * p.D, agate);
#pragma unroll
      for (int k = 0; k < E; ++k) agate[k] = 0.f;
    }
  }
  const int64_t plane = plan.nb * p.D;
  float* mine = part + b * p.D;
  if (p.dpost) put(mine + kPost * plane, apost);
  if (p.dpre) put(mine + kPre * plane, apre);
  if (p.dgate && plan.bpg > 1) put(mine + kGate * plane, agate);
  if constexpr (kLayer) {
    if (p.dpost_bias) put(mine + kPostBias * plane, apostb);
    if (p.dpre_bias) put(mine + kPreBias * plane, apreb);
  }
  if (cluster > 1)  // the others may still read this block's slots
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// Sums the ranges' partial rows in a fixed order: 32 columns for each block,
// 16 threads for each column.
struct ColumnSums {
  float* out[kPlanes];
  const float* part;
  int64_t nb, bpg, groups, D;
  int first[kPlanes + 1];  // blockIdx.y of a plane's first output row
};
__global__ void __launch_bounds__(512) column_sums_kernel(ColumnSums a) {
  __shared__ float red[16][33];
  int q = 0;
  while ((int)blockIdx.y >= a.first[q + 1]) ++q;
  const int64_t r = (int64_t)blockIdx.y - a.first[q];
  const int64_t from = q == kGate ? r * a.bpg : 0, n = q == kGate ? a.bpg : a.nb;
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < a.D) {
    const float* x = a.part + (q * a.nb + from) * a.D + c;
#pragma unroll 4
    for (int64_t i = threadIdx.y; i < n; i += 16) s += x[i * a.D];
  }
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < a.D) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += red[i][threadIdx.x];
    a.out[q][r * a.D + c] = t;
  }
}

template <class T, int VEC>
cudaError_t norm_backward_typed(const NormBackward& p, float* part, cudaStream_t stream) {
  const BackwardPlan plan = backward_plan(p.T, p.D, p.groups);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(plan.nb * plan.cluster));
  cfg.blockDim = dim3((unsigned)plan.threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)plan.cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = p.layer ? cudaLaunchKernelEx(&cfg, norm_backward_kernel<T, VEC, true>, p, plan, part)
                          : cudaLaunchKernelEx(&cfg, norm_backward_kernel<T, VEC, false>, p, plan, part);
  if (e != cudaSuccess) return e;
  ColumnSums a = {};
  a.part = part;
  a.nb = plan.nb, a.bpg = plan.bpg, a.groups = plan.groups, a.D = p.D;
  float* outs[kPlanes] = {p.dpost, p.dpre, plan.bpg > 1 ? p.dgate : nullptr, p.dpost_bias, p.dpre_bias};
  int rows = 0;
  for (int q = 0; q < kPlanes; ++q) {
    a.out[q] = outs[q];
    a.first[q] = rows;
    if (outs[q]) rows += q == kGate ? (int)plan.groups : 1;
  }
  a.first[kPlanes] = rows;
  if (rows) column_sums_kernel<<<dim3((unsigned)((p.D + 31) / 32), (unsigned)rows), dim3(32, 16), 0, stream>>>(a);
  return cudaGetLastError();
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
  return (size_t)kPlanes * backward_plan(T, D, groups).nb * D * 4;
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
