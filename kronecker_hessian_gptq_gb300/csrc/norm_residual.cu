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

// One row for each block: thread t holds the NV vectors of VEC elements at
// columns (i * blockDim.x + t) * VEC.
template <class T, int VEC, int NV, int kThreads>
__global__ void __launch_bounds__(kThreads) norm_residual_kernel(NormResidual p) {
  constexpr int E = VEC * NV;
  __shared__ float red[64];
  const int64_t row = blockIdx.x;
  const int D = (int)p.D;
  const float invd = 1.f / (float)D;
  float y[E];
  int col[NV];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = (i * (int)blockDim.x + (int)threadIdx.x) * VEC;
    in[i] = col[i] < D;
  }
  auto load = [&](const void* base, int64_t ld, float(&v)[E]) {
    const T* r = static_cast<const T*>(base) + row * ld;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float e[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) e[k] = 0.f;
      if (in[i]) load_vec<T, VEC>(r + col[i], e);
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[i * VEC + k] = e[k];
    }
  };
  // mean and reciprocal deviation of the row held in v
  auto stats = [&](const float(&v)[E], float& m, float& r) {
    m = 0.f;
    if (p.layer) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < E; ++k) s[0] += v[k];
      block_reduce<1>(s, red, SumOp());
      m = s[0] * invd;
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) s[0] = fmaf(v[i * VEC + k] - m, v[i * VEC + k] - m, s[0]);
      }
    block_reduce<1>(s, red, SumOp());
    r = rsqrtf(fmaf(s[0], invd, p.eps));
  };
  load(p.X, p.ldx, y);
  if (p.H) {
    float h[E];
    load(p.H, p.ldh, h);
    float m = 0.f, r = 1.f;
    if (p.post) stats(h, m, r);
    const T* gate = p.gate ? static_cast<const T*>(p.gate) + (row / (p.T / p.groups)) * p.ldg : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const int c = col[i] + k;
        float u = h[i * VEC + k];
        if (p.post) u = fmaf((u - m) * r, __ldg(p.post + c), p.post_bias ? __ldg(p.post_bias + c) : 0.f);
        if (gate) u *= to_f32<T>(gate[c]);
        y[i * VEC + k] = fmaf(p.alpha, y[i * VEC + k], u);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k) y[k] *= p.alpha;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!in[i]) continue;
    float e[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) e[k] = y[i * VEC + k];
    store_vec<T, VEC>(static_cast<T*>(p.Y) + row * D + col[i], e);
  }
  if (!p.pre) return;
  float m, r;
  stats(y, m, r);
  float top[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!in[i]) continue;
    float e[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int c = col[i] + k;
      e[k] = fmaf((y[i * VEC + k] - m) * r, __ldg(p.pre + c), p.pre_bias ? __ldg(p.pre_bias + c) : 0.f);
      y[i * VEC + k] = e[k];
      top[0] = MaxOp()(fabsf(e[k]), top[0]);
    }
    if (!p.C) store_vec<T, VEC>(static_cast<T*>(p.Z) + row * D + col[i], e);
  }
  if (!p.C) return;
  block_reduce<1>(top, red, MaxOp());
  const float s = token_scale(top[0]), inv = token_inv(s);
  if (threadIdx.x == 0) p.cs[row] = s;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!in[i]) continue;
    int8_t c[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) c[k] = (int8_t)token_code(y[i * VEC + k], s, inv);
    int8_t* to = p.C + row * D + col[i];
    if constexpr (VEC == 8) {
      uint2 u;
      memcpy(&u, c, 8);
      *reinterpret_cast<uint2*>(to) = u;
    } else if constexpr (VEC == 4) {
      uint32_t u;
      memcpy(&u, c, 4);
      *reinterpret_cast<uint32_t*>(to) = u;
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) to[k] = c[k];
    }
  }
}

template <class T, int VEC>
cudaError_t norm_residual_typed(const NormResidual& p, cudaStream_t stream) {
  const int64_t nvec = (p.D + VEC - 1) / VEC;
  constexpr int kUnit = 8 / VEC;  // vectors that make up 8 elements
  auto threads = [&](int64_t per) { return (unsigned)(std::max<int64_t>(1, (nvec + 32 * per - 1) / (32 * per)) * 32); };
  const unsigned grid = (unsigned)p.T;
  if (p.D <= 8192) {
    norm_residual_kernel<T, VEC, kUnit, 1024><<<grid, threads(kUnit), 0, stream>>>(p);
  } else if (p.D <= 16384) {
    norm_residual_kernel<T, VEC, 2 * kUnit, 1024><<<grid, threads(2 * kUnit), 0, stream>>>(p);
  } else {
    norm_residual_kernel<T, VEC, 4 * kUnit, 1024><<<grid, threads(4 * kUnit), 0, stream>>>(p);
  }
  return cudaGetLastError();
}

// ------------------------------------------------------------------ backward

constexpr int kBwdThreads = 512;  // 8 elements each: 4096 columns for one block of a cluster
constexpr int kBwdBlocks = 152;   // row ranges (times the cluster size: thread blocks)

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
  const int64_t most = std::max<int64_t>(1, kBwdBlocks * 2 / b.cluster);
  if (b.groups <= most) {
    b.bpg = std::max<int64_t>(1, std::min(each, most / b.groups));
    b.nb = b.groups * b.bpg;
  } else {
    b.bpg = 1;
    b.nb = most;
  }
  return b;
}

// Sum over the whole cluster's threads.  A cluster barrier separates the
// writes of a use from its reads, and `slot` alternates, so that a block
// writes a slot again only after a later barrier, which every reader of it
// has passed.
template <int N>
__device__ __forceinline__ void cluster_reduce(float (&v)[N], float* red, float (*slot)[4], int cluster, int& turn) {
  block_reduce<N>(v, red, SumOp());
  if (cluster == 1) return;
  float* mine = slot[turn];
  turn ^= 1;
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

template <class T, int VEC, bool kLayer>
__global__ void __launch_bounds__(kBwdThreads) norm_backward_kernel(NormBackward p, BackwardPlan plan, float* part) {
  constexpr int E = 8, NV = 8 / VEC;
  __shared__ float red[4 * 32];
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
  auto load = [&](const void* base, int64_t at, float(&v)[E]) {
    const T* r = static_cast<const T*>(base) + at;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float e[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) e[k] = 0.f;
      if (base && in[i]) load_vec<T, VEC>(r + col[i], e);
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[i * VEC + k] = e[k];
    }
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
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[i * VEC + k] = !in[i] ? 0.f : w ? __ldg(w + col[i] + k) : none;
  };
  float apost[E], apre[E], agate[E], apostb[kLayer ? E : 1], apreb[kLayer ? E : 1];
#pragma unroll
  for (int k = 0; k < E; ++k) apost[k] = apre[k] = agate[k] = 0.f;
  if constexpr (kLayer) {
#pragma unroll
    for (int k = 0; k < E; ++k) apostb[k] = apreb[k] = 0.f;
  }
  auto put = [&](float* to, const float(&v)[E]) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        if (in[i]) to[col[i] + k] = v[i * VEC + k];
  };
  const bool masked = !in[NV - 1];
  for (int64_t row = lo; row < hi; ++row) {
    const int64_t g = row / each;
    float y[E], h[E], dt[E], dz[E], w[E];
    load(p.Y, row * p.ldy, y);
    load(p.H, row * p.ldh, h);
    load(p.dY, row * p.lddy, dt);
    load(p.dZ, row * p.lddz, dz);
    float my = 0.f, mh = 0.f;
    if constexpr (kLayer) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < E; ++k) s[0] += y[k], s[1] += h[k];
      cluster_reduce<2>(s, red, slot, cluster, turn);
      my = s[0] * invd, mh = s[1] * invd;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          if (masked && !in[i]) continue;
          y[i * VEC + k] -= my;
          if (p.post) h[i * VEC + k] -= mh;
        }
    }
    float ry = 0.f, rh = 1.f;
    {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      param(p.pre, 0.f, w);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float kk = dz[k] * w[k];
        s[0] = fmaf(y[k], y[k], s[0]);
        s[1] = fmaf(kk, y[k], s[1]);
        s[2] = fmaf(h[k], h[k], s[2]);
        if (kLayer) s[3] += kk;
      }
      cluster_reduce<4>(s, red, slot, cluster, turn);
      if (p.pre && p.dZ) {
        ry = rsqrtf(fmaf(s[0], invd, p.eps));
        const float c1 = ry * ry * s[1] * invd, c0 = s[3] * invd;
#pragma unroll
        for (int k = 0; k < E; ++k) {
          dt[k] = fmaf(ry, fmaf(dz[k], w[k], -c0) - c1 * y[k], dt[k]);
          apre[k] = fmaf(dz[k], y[k] * ry, apre[k]);
          if constexpr (kLayer) apreb[k] += dz[k];
        }
      }
      if (p.post) rh = rsqrtf(fmaf(s[2], invd, p.eps));
    }
    {
      float dx[E];
#pragma unroll
      for (int k = 0; k < E; ++k) dx[k] = p.alpha * dt[k];
      store(p.dX, row * p.D, dx);
    }
    if (!p.H) continue;
    float gt[E];
    if (p.gate) {
      load(p.gate, g * p.ldg, gt);
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) gt[k] = 1.f;
    }
    param(p.post, 1.f, w);
    float wb[E];
    param(p.post_bias, 0.f, wb);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int kk = 0; kk < VEC; ++kk) {
        const int k = i * VEC + kk;
        if (masked && !in[i]) dt[k] = 0.f;
        const float n = h[k] * rh;
        agate[k] = fmaf(dt[k], fmaf(n, w[k], wb[k]), agate[k]);
        const float du = dt[k] * gt[k];
        apost[k] = fmaf(du, n, apost[k]);
        if constexpr (kLayer) apostb[k] += du;
        dt[k] = du * w[k];
        s[0] = fmaf(dt[k], n, s[0]);
        s[1] += dt[k];
      }
    if (p.post) {
      cluster_reduce<2>(s, red, slot, cluster, turn);
      const float c1 = s[0] * invd * rh, c0 = kLayer ? s[1] * invd : 0.f;
#pragma unroll
      for (int k = 0; k < E; ++k) dt[k] = rh * (dt[k] - c0 - c1 * h[k]);
    }
    store(p.dH, row * p.D, dt);
    if (p.dgate && row + 1 == (g + 1) * each && plan.bpg == 1) {  // this range holds the whole group
      put(p.dgate + g * p.D, agate);
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

}  // namespace

cudaError_t norm_residual_launch(const NormResidual& p, cudaStream_t stream) {
  const bool vec = vectors(p.dtype, p.D, {{p.X, p.ldx}, {p.H, p.ldh}, {p.gate, p.ldg}, {p.Y, p.D}, {p.Z, p.D}}) &&
                   (!p.C || aligned_to(p.C, 8));
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
                                          {p.dX, p.D}, {p.dH, p.D}});
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
