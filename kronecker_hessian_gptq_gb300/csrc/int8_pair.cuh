// int8_pair.cuh -- the product of 8-bit weights with a batch of tokens on
// pairs of SMs, for batches that are bound by reading the weights.
//
// The chip has no fast 8-bit integer products (tcgen05 kind::i8 is absent from
// sm_103a), but an 8-bit integer is exact in fp16, its products are exact in
// fp32, and sums of 1024 of them stay below 2^24: so the weights are read as
// bytes, converted on their way through shared memory, and multiplied with
// kind::f16, and sums of at most 1024 terms are joined as 32-bit integers.
//
// A cluster of two blocks takes 256 outputs (the MMA's rows, 128 for each
// block) against up to 256 tokens (its columns) and one part of K.  For every
// 64 of K a stage holds, in each block, 128 x 64 bytes of weights as they come
// (TMA), the same as fp16 in the swizzled layout (eight warps convert, four
// for even and four for odd stages), and half of the tokens' codes (TMA,
// already fp16).  Each part of K is added to a 32-bit sum in memory with
// integer atomics, whose order does not matter; the last to arrive scales a
// slice's sums and writes the results.
#pragma once

#include "elem.cuh"
#include "pair_gemm.cuh"

namespace bakron {

constexpr int kI8Raw = 128 * kPairK;       // bytes of weights of a stage: 8 KB
constexpr int kI8A = 128 * kPairK * 2;     // the same in fp16: 16 KB
constexpr int kI8MaxStages = 8;
constexpr int kI8Steps = 16;               // stages of a part at most: 1024 of K
constexpr int kI8Threads = (4 + 8 + 8) * 32;
constexpr int kI8SmemMost = 220 * 1024;

struct I8Work {
  int tiles_m, tiles_n, nt;  // outputs / 256, token tiles of nt tokens (a multiple of 32)
  int ksteps, parts;
  int stages;
  __host__ __device__ int units() const { return tiles_m * tiles_n * parts; }
  __host__ __device__ int stage_bytes() const { return kI8Raw + kI8A + nt / 2 * 128; }
};

template <class T>
struct I8Out {
  int64_t tokens, outputs;
  const float *x_scales, *w_scales, *bias;
  T* y;
  int32_t* sums;      // tokens x outputs, zero; used where parts > 1
  uint32_t* arrived;  // a counter for each slice of 32 outputs and half a token tile, zero
};

struct I8Barriers {
  uint64_t raw[kI8MaxStages], ready[kI8MaxStages], empty[kI8MaxStages], sum_full[2], sum_empty[2];
  uint32_t tmem;
};

// Four 8-bit integers as fp16: with the sign bit flipped a byte b is the
// value + 128, and 0x6400 + b is the fp16 number 1024 + b, exactly.
__device__ __forceinline__ void i8_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u, magic = 0x64646464u, off = 0x64806480u;  // 1152
  const uint32_t a = __byte_perm(u, magic, 0x4140), b = __byte_perm(u, magic, 0x4342);
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(lo) : "r"(a), "r"(off));
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(hi) : "r"(b), "r"(off));
}

template <class T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kI8Threads, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, I8Work work,
                     I8Out<T> out, int32_t* status) {
  extern __shared__ unsigned char i8_smem_raw[];
  const uint32_t base = (smem_u32(i8_smem_raw) + 1023u) & ~1023u;
  __shared__ I8Barriers bar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pairs = gridDim.x / 2, mine = blockIdx.x / 2, units = work.units(), stages = work.stages;
  const uint32_t stage = (uint32_t)work.stage_bytes(), half = (uint32_t)(work.nt / 2 * 128);
  bool broken = false;

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(smem_u32(&bar.raw[i])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 9;\n" ::"r"(smem_u32(&bar.ready[i])));  // copies, 2 x 4 warps
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(smem_u32(&bar.empty[i])));
    }
    for (int i = 0; i < 2; ++i) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(smem_u32(&bar.sum_full[i])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 16;\n" ::"r"(smem_u32(&bar.sum_empty[i])));
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&bar.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  auto unit = [&](int u, int& tm, int& tn, int& k0, int& k1) {
    tn = u % work.tiles_n;
    tm = u / work.tiles_n % work.tiles_m;
    const int part = u / (work.tiles_n * work.tiles_m);
    k0 = (int)((int64_t)work.ksteps * part / work.parts);
    k1 = (int)((int64_t)work.ksteps * (part + 1) / work.parts);
  };

  if (warp == 0) {  // copies: the weights' bytes and half of the tokens' codes
    int tm, tn, k0, k1;
    Ring ring;
    for (int u = mine; u < units && !broken; u += pairs) {
      unit(u, tm, tn, k0, k1);
      const int o0 = tm * 256 + (int)rank * 128, t0 = tn * work.nt + (int)rank * (work.nt / 2);
      for (int k = k0; k < k1; ++k, ring.next(stages)) {
        const int slot = ring.slot;
        if (ring.round) ring_wait(&bar.empty[slot], ring.turn ^ 1u, broken);
        if ((broken = __any_sync(0xffffffffu, broken))) break;
        const uint32_t raw = base + (uint32_t)slot * stage, x = raw + kI8Raw + kI8A;
        const uint32_t ready = in_even_block(&bar.ready[slot]);
        if (elect_one()) {
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(&bar.raw[slot])), "r"(kI8Raw)
                       : "memory");
          asm volatile(
              "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
                  raw),
              "l"(&map_w), "r"(k * kPairK), "r"(o0), "r"(smem_u32(&bar.raw[slot]))
              : "memory");
          if (rank == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(&bar.ready[slot])),
                         "r"(2u * half)
                         : "memory");
          pair_copy(x, &map_x, k * kPairK, t0, ready);
        }
        __syncwarp();
      }
    }
    // See pair_gemm_kernel: nothing is on its way into a block that leaves.
    for (int i = 0; i < stages; ++i, ring.next(stages)) {
      if (!ring.round) continue;  // this stage's first use would come here
      bool late = false;
      if (!broken) {
        ring_wait(&bar.empty[ring.slot], ring.turn ^ 1u, broken);
      } else {
        ring_wait(&bar.raw[ring.slot], ring.turn ^ 1u, late);
        if (rank == 0) ring_wait(&bar.ready[ring.slot], ring.turn ^ 1u, late);
      }
    }
  } else if (warp == 1 && rank == 0) {  // products
    // fp32 sums of fp16 products, both with K contiguous, M = 256, N = nt
    const uint32_t idesc = (1u << 4) | ((uint32_t)(work.nt >> 3) << 17) | ((256u >> 4) << 24);
    int sums = 0, tm, tn, k0, k1;
    Ring ring;
    for (int u = mine; u < units && !broken; u += pairs, ++sums) {
      unit(u, tm, tn, k0, k1);
      const uint32_t acc = tmem + (uint32_t)(sums & 1) * 256u;
      if (sums >= 2) ring_wait(&bar.sum_empty[sums & 1], (uint32_t)(sums / 2 - 1) & 1u, broken);
      tc_fence_after();
      for (int k = k0; k < k1; ++k, ring.next(stages)) {
        const int slot = ring.slot;
        ring_wait(&bar.ready[ring.slot], ring.turn, broken);
        if ((broken = __any_sync(0xffffffffu, broken))) break;
        tc_fence_after();
        const uint32_t a = base + (uint32_t)slot * stage + kI8Raw, b = a + kI8A;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kPairK / 16; ++j)
            pair_mma(acc, pair_desc<false>(a + j * 32u), pair_desc<false>(b + j * 32u), idesc, (k > k0 || j > 0) ? 1u : 0u);
          pair_commit(&bar.empty[slot]);
          if (k + 1 == k1) pair_commit(&bar.sum_full[sums & 1]);
        }
        __syncwarp();
      }
    }
  } else if (warp >= 4 && warp < 12) {  // bytes to fp16: 32 rows of every second stage for each warp
    const int group = (warp - 4) >> 2, quarter = (warp - 4) & 3;
    int n = 0, tm, tn, k0, k1;
    Ring ring;
    for (int u = mine; u < units && !broken; u += pairs) {
      unit(u, tm, tn, k0, k1);
      for (int k = k0; k < k1; ++k, ++n, ring.next(stages)) {
        if ((n & 1) != group) continue;
        const int slot = ring.slot;
        ring_wait(&bar.raw[slot], ring.turn, broken);
        if ((broken = __any_sync(0xffffffffu, broken))) break;
        const uint32_t raw = base + (uint32_t)slot * stage, a = raw + kI8Raw;
        uint32_t w[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)  // 16 bytes of row 32 quarter + 8 i + lane / 4
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                       : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                       : "r"(raw + (uint32_t)(32 * quarter + 8 * i) * 64u + (uint32_t)lane * 16u)
                       : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 32 * quarter + 8 * i + (lane >> 2), j = 2 * (lane & 3);
          uint32_t h[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) i8_to_f16(w[i][q], h[2 * q], h[2 * q + 1]);
#pragma unroll
          for (int q = 0; q < 2; ++q)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(a + (uint32_t)(r * 128 + (((j + q) ^ (r & 7)) << 4))),
                         "r"(h[4 * q]), "r"(h[4 * q + 1]), "r"(h[4 * q + 2]), "r"(h[4 * q + 3])
                         : "memory");
        }
        // Each thread's fence makes what it wrote visible to the MMAs before
        // the arrival; a release of cluster scope on top of it would stall the
        // warp for half a microsecond in every stage.
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(in_even_block(&bar.ready[slot])) : "memory");
      }
    }
  } else if (warp >= 12) {  // epilogue: 32 outputs (lanes) and half of the tokens for each warp
    const int quarter = warp & 3, part = (warp - 12) >> 2;
    const int cols = work.nt / 2, c0 = part * cols;
    const uint32_t lanes = ((uint32_t)(32 * quarter) << 16) + (uint32_t)c0;
    int sums = 0, tm, tn, k0, k1;
    for (int u = mine; u < units && !broken; u += pairs, ++sums) {
      unit(u, tm, tn, k0, k1);
      ring_wait(&bar.sum_full[sums & 1], (uint32_t)(sums / 2) & 1u, broken);
      if ((broken = __any_sync(0xffffffffu, broken))) break;
      tc_fence_after();
      const int64_t o = (int64_t)tm * 256 + rank * 128 + 32 * quarter + lane;
      const int64_t t0 = (int64_t)tn * work.nt + c0;
      const int live = (int)(out.tokens - t0 < cols ? out.tokens - t0 : cols);  // may be negative
      const bool in = o < out.outputs;
      const float ws = in ? out.w_scales[o] : 0.f, bias = in && out.bias ? out.bias[o] : 0.f;
      const uint32_t from = tmem + (uint32_t)(sums & 1) * 256u + lanes;
      for (int c = 0; c < live; c += 8) {  // the same for the whole warp
        float v[8];
        tmem_ld(from + (uint32_t)c, v);
        asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
        if (!in) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (c + i >= live) break;
          const int64_t t = t0 + c + i, at = t * out.outputs + o;
          if (work.parts == 1)
            out.y[at] = from_f32<T>(fmaf(v[i] * out.x_scales[t], ws, bias));
          else
            atomicAdd(out.sums + at, __float2int_rn(v[i]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(in_even_block(&bar.sum_empty[sums & 1]))
                     : "memory");
      if (work.parts == 1) continue;
      // The last of a slice's parts to arrive reads the joined sums.
      __threadfence();
      __syncwarp();
      uint32_t before = 0;
      if (lane == 0)
        before = atomicAdd(out.arrived + (((int64_t)tm * work.tiles_n + tn) * 2 + rank) * 8 + part * 4 + quarter, 1u);
      before = __shfl_sync(0xffffffffu, before, 0);
      if (before + 1 != (uint32_t)work.parts) continue;
      __threadfence();
      if (!in) continue;
#pragma unroll 8
      for (int c = 0; c < live; ++c) {
        const int64_t t = t0 + c, at = t * out.outputs + o;
        out.y[at] = from_f32<T>(fmaf((float)__ldcg(out.sums + at) * out.x_scales[t], ws, bias));
      }
    }
  }
  if (broken) atomicOr(status, BAKRON_DEV_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
}

inline I8Work i8_work(int64_t T, int64_t K, int64_t N, int pairs) {
  I8Work w;
  w.tiles_m = (int)((N + 255) / 256);
  w.tiles_n = (int)((T + 255) / 256);
  w.nt = (int)(((T + w.tiles_n - 1) / w.tiles_n + 31) / 32 * 32);
  w.tiles_n = (int)((T + w.nt - 1) / w.nt);
  w.ksteps = (int)((K + kPairK - 1) / kPairK);
  // Parts of at most kI8Steps, and as many as make the pairs' longest share
  // shortest; a part's start and end cost about 6 steps.
  const int tiles = w.tiles_m * w.tiles_n, least = (w.ksteps + kI8Steps - 1) / kI8Steps;
  int64_t cost = INT64_MAX;
  for (int p = least; p <= w.ksteps && p <= 4 * least + 16; ++p) {
    const int64_t c = (int64_t)((tiles * (int64_t)p + pairs - 1) / pairs) * ((w.ksteps + p - 1) / p + 6);
    if (c < cost) cost = c, w.parts = p;
  }
  w.stages = std::min(kI8MaxStages, kI8SmemMost / w.stage_bytes());
  return w;
}
inline int64_t i8_slices(const I8Work& w) { return (int64_t)w.tiles_m * w.tiles_n * 16; }

template <class T>
cudaError_t int8_pair_launch(const int8_t* V, int64_t ldv, const void* codes, int64_t ldc, int64_t K, const I8Work& w,
                             const I8Out<T>& out, int32_t* status, cudaStream_t stream) {
  CUtensorMap mw, mx;
  cudaError_t e = make_tensor_map(&mw, TileMap{V, CU_TENSOR_MAP_DATA_TYPE_UINT8, out.outputs, K, ldv, 128, kPairK, false});
  if (e == cudaSuccess)
    e = make_tensor_map(&mx, TileMap{codes, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, out.tokens, K, ldc, (uint32_t)w.nt / 2, kPairK, true});
  const int smem = w.stages * w.stage_bytes() + 1024;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(int8_pair_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kI8SmemMost + 1024);
  if (e != cudaSuccess) return e;
  const unsigned grid = 2u * (unsigned)std::min(w.units(), pair_count());
  int8_pair_kernel<T><<<grid, kI8Threads, smem, stream>>>(mw, mx, w, out, status);
  return cudaGetLastError();
}

}  // namespace bakron
