// fp8_pair.cuh -- products of e4m3 codes with one scale for each 128 of K, on
// pairs of SMs:
//     C[m, n] = sum over blocks b of sa[m, b] sb[n, b] sum_{k in b} A[m, k] B[n, k].
//
// A cluster of two blocks computes a tile of 256 x kN.  A stage holds one block
// of K: 128 codes of 128 rows of A and of kN / 2 rows of B in each block of the
// pair (TMA, 128-byte swizzle), four tcgen05.mma of kind::f8f6f4 with
// cta_group::2.  The tensor cores sum one block of K alone; the sums (fp32, in
// tensor memory, two or four in turn) are read by eight epilogue warps, scaled and
// added to sums in registers, a thread for a row and kN / 2 columns, while the
// next block is multiplied.  For kN = 256 the tensor cores take 512 cycles for a
// block of K, and the scaled additions as many where the columns share a scale
// (weights: one for 128 x 128), for the packed ones go at half rate; twice as many
// where they do not (kColumns).  Measured at 4096 x 4864 x 16384: 0.46 us a block
// (950 cycles), of which the tensor cores and copies alone take 0.37 (the two
// SMs fetch 64 KB for it, 13 TB/s over all of them); 4096 tokens 4096 x 14336
// 216 us, quantized in the call (2.2 PFLOP/s).  16 epilogue warps with half the
// columns each issue more for waits and scales (236 us).
//
// Either operand may be stored with K contiguous or with its rows contiguous
// (a weight's gradient sums over tokens, a row each).  Where there are fewer
// tiles than pairs of SMs, K is cut into parts whose sums meet in memory: the
// last part of a tile to arrive adds them up in their order.
//
// One warp copies the weights' side, one the other, which a kernel before may
// still be writing (griddepcontrol): the weights are then on their way already.
#pragma once

#include <algorithm>
#include <cstdint>

#include "pair_gemm.cuh"

namespace bakron {

constexpr int kF8K = 128;  // K of a stage, and of a scale
constexpr int kF8Warps = 8;  // of the epilogue
constexpr int kF8Threads = 128 + 32 * kF8Warps;
constexpr int kF8MostStages = 10;
constexpr int kF8Ring = 2;  // batches of scales on their way
constexpr int kF8Smem = 226 * 1024;

// Shared memory of a variant: stages, boxes for results in whole lines, scales
// (of the columns, of the block's 128 rows).
template <int kN, bool kBRows, bool kColumns, bool kRows, bool kBoxes>
struct F8Shape {
  // Rows of B that a block copies: with its rows contiguous whole lines of 128, of which 64 may count.
  static constexpr int kCopied = kBRows && kN < 256 ? 128 : kN / 2;
  static constexpr int kA = 128 * kF8K, kB = kCopied * kF8K, kStage = kA + kB;
  static constexpr int kHalves = kN > 128 ? 2 : 1;  // products of half the columns each
  static constexpr int kBufs = kN > 128 ? 2 : 4;
  static constexpr int kCols = kN / (kF8Warps / 4);  // of a thread
  static constexpr int kScales = ((kColumns ? kN : 0) + (kRows ? 128 : 0)) * 4;  // of a block of K
  static constexpr int kBatch = kColumns && kN > 64 ? 4 : 8;  // blocks whose scales come together
  static constexpr int kBox = kBoxes ? kN / 128 * kPairBox : 0;  // of a warp: one for each run
  static constexpr int kOther = kF8Warps * kBox + kF8Ring * kBatch * kScales + 1024;
  static constexpr int kFit = (kF8Smem - kOther) / kStage;
  static constexpr int kStages = kFit < kF8MostStages ? kFit : kF8MostStages;
  static constexpr int kBytes = kStages * kStage + kOther;
};

// Scales in block k of K.  Those of activations differ from row to row: the
// one of row (or column) i is p[k step + i], step a multiple of 4 and at least
// what the tiles cover.  Those of weights are one for 128: p[(i >> 7) each + k step].
struct F8Scales {
  const float *a, *b;
  int64_t a_step, b_step, each;
  int64_t weights;  // rows or columns that weights have
};
struct F8Join {
  float* sums;        // a tile's parts: [part][tile][block of the pair][warp][column][lane]
  uint32_t* arrived;  // for each tile, block and warp, zero
};

struct F8Barriers {
  uint64_t full[kF8MostStages], empty[kF8MostStages], sum_full[4], sum_empty[4], scale_full[kF8Ring], scale_empty[kF8Ring];
  uint32_t tmem;
};

__device__ __forceinline__ void pair_mma_f8(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 da, db;\nmov.b64 da, {%1, %2};\nmov.b64 db, {%3, %2};\nsetp.ne.b32 p, %5, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(kPairDescHigh), "r"(b), "r"(idesc), "r"(acc));
}
// 16 bytes' units from one K = 32 to the next within a stage: 32 bytes of a
// row, or 32 rows of 128 bytes.
template <bool kRows>
__host__ __device__ constexpr uint32_t f8_kstep() { return kRows ? 4096u >> 4 : 32u >> 4; }
// 16 columns of the warp's 32 lanes of tensor memory.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Whether the phase of a barrier, given by its address, is done, for a whole warp.
__device__ __forceinline__ bool phase_done_at(uint32_t mbar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(done)
               : "r"(mbar), "r"(parity)
               : "memory");
  return __all_sync(0xffffffffu, done) != 0;
}
__device__ __forceinline__ void warp_wait_at(uint32_t mbar, uint32_t parity, bool& broken) {
  if (broken || phase_done_at(mbar, parity)) return;
  const uint32_t t0 = clock();
  while (!phase_done_at(mbar, parity)) {
    if (__any_sync(0xffffffffu, clock() - t0 > (1u << 28))) {
      broken = true;
      return;
    }
  }
}
__device__ __forceinline__ void arrive_if(bool p, uint32_t mbar) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %1, 0;\n@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n}\n" ::"r"(mbar),
      "r"((uint32_t)p)
      : "memory");
}

// A warp's box for one of kRuns runs: only those before the last kRuns - 1 groups of
// copies have to have been read.  So every run is a group, in turn: one that lies
// outside the matrix commits an empty one (skip), without which the next tile's first
// run would take its own box's copy for the other's.
template <int kRuns>
struct F8Box : PairBox {
  __device__ __forceinline__ void open() const {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;\n" ::"n"(kRuns - 1) : "memory");
    __syncwarp();
  }
  __device__ __forceinline__ void skip() const {
    if (lane == 0) asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
  }
};
// pair_unit without divisions where K is whole, and with few where it is not: they
// would take an epilogue warp a thousand cycles of each tile.
__device__ __forceinline__ PairUnit f8_unit(const PairWork& w, int u) {
  PairUnit r;
  const uint32_t tiles = (uint32_t)w.tiles_m * w.tiles_n, whole = (uint32_t)w.group * w.tiles_n;
  uint32_t t = u;
  r.part = 0, r.k0 = 0, r.k1 = w.ksteps;
  if (w.parts > 1) {
    r.part = t / tiles, t -= r.part * tiles;
    r.k0 = (uint32_t)w.ksteps * r.part / w.parts;
    r.k1 = (uint32_t)w.ksteps * (r.part + 1) / w.parts;
  }
  const uint32_t g = t / whole, first = g * w.group, in = t - g * whole;
  const uint32_t rows = w.tiles_m - first < w.group ? w.tiles_m - first : w.group;
  r.tn = in / rows;
  r.tm = first + (in - r.tn * rows);
  return r;
}

// kWeights: which operand the weights are, 1 for A, 2 for B, 0 for neither
// (then both have a scale for each row).  No kernel before writes them.
template <bool kARows, bool kBRows, int kN, int kWeights, bool kJoin, class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kF8Threads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, PairWork work,
                    F8Scales sc, F8Join join, const __grid_constant__ Epi epi, int32_t* status, int32_t first_status) {
  constexpr bool kColumns = kWeights != 2, kRows = kWeights != 1;  // have scales of their own
  using Shape = F8Shape<kN, kBRows, kColumns, kRows, Epi::kBoxes>;
  static_assert(2 * kF8Warps * 32 * Shape::kCols == 256 * kN, "the slices make up a tile");
  constexpr int kStages = Shape::kStages, kBufs = Shape::kBufs, kHalves = Shape::kHalves, kCols = Shape::kCols;
  extern __shared__ unsigned char f8_smem_raw[];
  const uint32_t base = (smem_u32(f8_smem_raw) + 1023u) & ~1023u;
  const uint32_t boxes = base + kStages * Shape::kStage;
  const uint32_t scales = boxes + kF8Warps * Shape::kBox;
  __shared__ F8Barriers bar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pairs = gridDim.x / 2, mine = blockIdx.x / 2, units = work.units();
  bool broken = false;

  // Blocks of a kernel that may start early take the SMs that this one's leave.
  asm volatile("griddepcontrol.launch_dependents;\n");
  // This early nothing can have been reported.
  if (first_status >= 0 && blockIdx.x == 0 && threadIdx.x == 0) *status = first_status;
  if (threadIdx.x == 0) {
    auto init = [](uint64_t* b, int n) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(b)), "r"(n));
    };
    for (int i = 0; i < kStages; ++i) init(&bar.full[i], 1), init(&bar.empty[i], kHalves);
    for (int i = 0; i < kBufs * kHalves; ++i) init(&bar.sum_full[i], 1), init(&bar.sum_empty[i], 2 * kF8Warps / kHalves);
    for (int i = 0; i < kF8Ring; ++i) init(&bar.scale_full[i], 1), init(&bar.scale_empty[i], kF8Warps);
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
  // 384 threads start with 168 registers each.  Where that is not enough the first
  // four warps hand 96 of theirs on, 48 to each of the other eight (128 x 72 +
  // 256 x 216 = 384 x 168): with sums that meet in memory and with columns' scales.
  // Where it is, the compiler does better without (220 us, with 230).
  constexpr bool kHandOn = kCols == 128 && (kJoin || kWeights == 0);
  if (warp < 4) {
  if (kHandOn) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
  if (warp == 0 || warp == 3) {  // copies: warp 0 the weights' side, warp 3 the other and the scales
    const bool is_a = (warp == 0) == (kWeights == 1);
    if (warp == 3 || kWeights == 0) asm volatile("griddepcontrol.wait;\n" ::: "memory");
    auto fetch = [&](uint32_t to, const float* from, uint32_t bytes, uint32_t full) {
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(to),
                   "l"(from), "r"(bytes), "r"(full)
                   : "memory");
    };
    Ring ring, batch;
    for (int u = mine; u < units && !broken; u += pairs) {
      const PairUnit q = f8_unit(work, u);
      const int row = is_a ? q.tm * 256 + (int)rank * 128 : q.tn * kN + (int)rank * (kN / 2);
      for (int k = q.k0; k < q.k1; ++k, ring.next(kStages)) {
        const int slot = ring.slot;
        if (warp == 3 && (k - q.k0) % Shape::kBatch == 0) {
          if (batch.round) warp_wait(&bar.scale_empty[batch.slot], batch.turn ^ 1u, broken);
          if (broken) break;
          if (elect_one()) {
            const uint32_t full = smem_u32(&bar.scale_full[batch.slot]);
            const int here = q.k1 - k < Shape::kBatch ? q.k1 - k : Shape::kBatch;
            uint32_t to = scales + (uint32_t)(batch.slot * Shape::kBatch * Shape::kScales);
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(full), "r"(here * Shape::kScales)
                         : "memory");
            for (int j = 0; j < here; ++j, to += Shape::kScales) {
              if (kColumns) fetch(to, sc.b + (k + j) * sc.b_step + (int64_t)q.tn * kN, kN * 4, full);
              if (kRows)
                fetch(to + (kColumns ? kN * 4 : 0), sc.a + (k + j) * sc.a_step + (int64_t)q.tm * 256 + rank * 128, 512, full);
            }
          }
          __syncwarp();
          batch.next(kF8Ring);
        }
        if (ring.round) warp_wait(&bar.empty[slot], ring.turn ^ 1u, broken);
        if (broken) break;
        const uint32_t full = in_even_block(&bar.full[slot]);
        const uint32_t at = base + (uint32_t)slot * Shape::kStage + (is_a ? 0u : (uint32_t)Shape::kA);
        if (elect_one()) {
          // The other warp's bytes may be counted before they are expected.
          if (warp == 0 && rank == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(&bar.full[slot])),
                         "r"(2u * Shape::kStage)
                         : "memory");
          if (is_a)
            pair_copy(at, &map_a, kARows ? row : k * kF8K, kARows ? k * kF8K : row, full);
          else
            pair_copy(at, &map_b, kBRows ? row : k * kF8K, kBRows ? k * kF8K : row, full);
        }
        __syncwarp();
      }
    }
    // No block leaves while copies into it, or arrivals at its barriers, are on their way (see pair_gemm_kernel).
    for (int i = 0; i < kStages; ++i, ring.next(kStages)) {
      if (!ring.round) continue;
      bool late = false;
      if (!broken)
        warp_wait(&bar.empty[ring.slot], ring.turn ^ 1u, broken);
      else if (rank == 0)
        warp_wait(&bar.full[ring.slot], ring.turn ^ 1u, late);
    }
    for (int i = 0; warp == 3 && i < kF8Ring; ++i, batch.next(kF8Ring)) {
      bool late = false;
      if (batch.round) warp_wait(&bar.scale_full[batch.slot], batch.turn ^ 1u, late);
    }
  } else if (rank == 0 && warp - 1 < kHalves) {  // products, a warp for each half of the columns
    // fp32 sums of e4m3 products, which operands have their rows contiguous, N, M = 256
    constexpr uint32_t idesc = (1u << 4) | ((kARows ? 1u : 0u) << 15) | ((kBRows ? 1u : 0u) << 16) |
                               ((uint32_t)((kN / kHalves) >> 3) << 17) | ((256u >> 4) << 24);
    const int half = warp - 1;
    // Rows of B: with K contiguous 64 rows are 8 KB on, else 64 bytes of each.
    const uint32_t b_half = (uint32_t)half * (kBRows ? 64u >> 4 : 8192u >> 4);
    int sums = 0;
    Ring ring;
    for (int u = mine; u < units && !broken; u += pairs) {
      const PairUnit q = f8_unit(work, u);
      for (int k = q.k0; k < q.k1; ++k, ring.next(kStages), ++sums) {
        const int buf = sums % kBufs, sum = buf * kHalves + half;
        warp_wait(&bar.full[ring.slot], ring.turn, broken);
        if (sums >= kBufs) warp_wait(&bar.sum_empty[sum], (uint32_t)(sums / kBufs - 1) & 1u, broken);
        if (broken) break;
        tc_fence_after();
        const uint32_t at = base + (uint32_t)ring.slot * Shape::kStage, acc = tmem + (uint32_t)(sum * (kN / kHalves));
        const uint32_t a = pair_desc_low<kARows>(at), b = pair_desc_low<kBRows>(at + Shape::kA) + b_half;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kF8K / 32; ++j) pair_mma_f8(acc, a + j * f8_kstep<kARows>(), b + j * f8_kstep<kBRows>(), idesc, j > 0);
          pair_commit(&bar.sum_full[sum]);
          pair_commit(&bar.empty[ring.slot]);
        }
        __syncwarp();
      }
    }
  }
  } else {  // epilogue: 32 rows of the block and kCols columns for each warp, in runs of at most 64
    if (kHandOn) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;\n");
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    // A half's products have 64 columns of the even block's rows of B, then 64 of the odd block's.
    constexpr int kRuns = kCols > 64 ? 2 : 1, kRun = kCols / kRuns;
    static_assert(kRuns == kHalves, "a warp has one half's columns, or its share of them all");
    const int half = kHalves > 1 ? part : 0, first = part * kRun;  // of the thread's columns in the tile; the second run is 128 on
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(kHalves > 1 ? half * (kN / 2) : part * kCols);
    const uint32_t full_at = smem_u32(&bar.sum_full[half]), empty_at = in_even_block(&bar.sum_empty[half]);
    const uint32_t row_at = (uint32_t)((kColumns ? kN : 0) + 32 * quarter + lane) * 4u, col_at = (uint32_t)first * 4u;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    // The weights' scales are the whole warp's: a lane reads those of one block,
    // 32 blocks at a time, and those of the next unit while this one is at hand.
    constexpr int kShared = kWeights == 2 ? kRuns : 1;
    auto shared_scale = [&](const PairUnit& q, int k, int run) {
      if (kWeights == 0 || k >= q.k1) return 0.f;
      int64_t at = kWeights == 1 ? (int64_t)q.tm * 256 + rank * 128 : (int64_t)q.tn * kN + first + 128 * run;
      at = at < sc.weights ? at : sc.weights - 1;  // beyond the matrix, where sums are 0, the last
      return kWeights == 1 ? sc.a[(at >> 7) * sc.each + k * sc.a_step] : sc.b[(at >> 7) * sc.each + k * sc.b_step];
    };
    auto arrive = [&](uint64_t* b) {
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(b)) : "memory");
    };
    uint32_t buf = 0, turn = 0;
    Ring ring;
    PairUnit next = f8_unit(work, mine);
    float of_32[kShared], ahead[kShared];
#pragma unroll
    for (int i = 0; i < kShared; ++i) ahead[i] = shared_scale(next, next.k0 + lane, i);
    for (int u = mine; u < units && !broken; u += pairs) {
      const PairUnit q = next;
#pragma unroll
      for (int i = 0; i < kShared; ++i) of_32[i] = ahead[i];
      if (u + pairs < units) {
        next = f8_unit(work, u + pairs);
#pragma unroll
        for (int i = 0; i < kShared; ++i) ahead[i] = shared_scale(next, next.k0 + lane, i);
      }
      const int64_t row0 = (int64_t)q.tm * 256 + rank * 128 + 32 * quarter, col = (int64_t)q.tn * kN + first;
      F2 acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = f2(0.f);
      const int blocks = q.k1 - q.k0;
      for (int first_in = 0; first_in < blocks && !broken; first_in += Shape::kBatch) {
        warp_wait_at(smem_u32(&bar.scale_full[ring.slot]), ring.turn, broken);
        if (kWeights && first_in % 32 == 0 && first_in > 0) {  // 32 is a multiple of a batch
#pragma unroll
          for (int i = 0; i < kShared; ++i) of_32[i] = shared_scale(q, q.k0 + first_in + lane, i);
        }
        const uint32_t batch = scales + (uint32_t)(ring.slot * Shape::kBatch * Shape::kScales);
        const int here = blocks - first_in < Shape::kBatch ? blocks - first_in : Shape::kBatch;
#pragma unroll 1
        for (int j = 0; j < here; ++j) {
        const uint32_t from = batch + (uint32_t)j * Shape::kScales;
        float of_row = 1.f;
        if (kRows) asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(of_row) : "r"(from + row_at) : "memory");
        F2 scale[kShared];
#pragma unroll
        for (int i = 0; i < kShared; ++i) scale[i] = f2(of_row) * f2(kWeights ? __shfl_sync(0xffffffffu, of_32[i], (first_in + j) & 31) : 1.f);
        warp_wait_at(full_at + buf * (kHalves * 8), turn, broken);
        if (broken) break;
        tc_fence_after();
        const uint32_t at = lanes + buf * kN;
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          float v[16];
          tmem_ld16(at + c, v);
          if (c + 16 == kCols) {  // all read: the buffer may be filled again
            tc_fence_before();
            // A release of cluster scope would stall the warp for half a
            // microsecond; the tensor-memory loads are complete.
            arrive_if(lane == 0, empty_at + buf * (kHalves * 8));
          }
          const F2 by = scale[kShared > 1 ? c / kRun : 0];
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            F2 x = f2(v[i], v[i + 1]), y = f2(v[i + 2], v[i + 3]);
            if constexpr (kColumns) {
              float f[4];
              asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];\n"
                           : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
                           : "r"(from + col_at + (uint32_t)(c + i + (c >= 64 ? 64 : 0)) * 4u)
                           : "memory");
              x = x * f2(f[0], f[1]);
              y = y * f2(f[2], f[3]);
            }
            acc[(c + i) / 2] = fma2(x, by, acc[(c + i) / 2]);
            acc[(c + i) / 2 + 1] = fma2(y, by, acc[(c + i) / 2 + 1]);
          }
        }
        if (++buf == kBufs) buf = 0, turn ^= 1u;
        }
        if (broken) break;
        arrive(&bar.scale_empty[ring.slot]);
        ring.next(kF8Ring);
      }
      if (broken) break;
      bool last = true;
      if (kJoin && work.parts > 1) {
        if (row0 >= epi.rows() || col >= epi.cols()) continue;  // for every part alike
        const int64_t tile = (int64_t)q.tm * work.tiles_n + q.tn, tiles = (int64_t)work.tiles_m * work.tiles_n;
        const int64_t slice = (tile * 2 + rank) * kF8Warps + (warp - 4), stride = tiles * 2 * kF8Warps * 32 * kCols;
        float2* to = reinterpret_cast<float2*>(join.sums + slice * (32 * kCols)) + lane;
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) {
          float2 x;
          split(acc[i], x.x, x.y);
          to[q.part * (stride / 2) + 32 * i] = x;
        }
        __threadfence();
        __syncwarp();
        uint32_t before = 0;
        if (lane == 0) before = atomicAdd(join.arrived + slice, 1u);
        last = __shfl_sync(0xffffffffu, before, 0) + 1 == (uint32_t)work.parts;
        if (last) {
          __threadfence();
#pragma unroll
          for (int i = 0; i < kCols / 2; ++i) acc[i] = f2(0.f);
          for (int p = 0; p < work.parts; ++p) {
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) {
              const float2 x = __ldcg(to + p * (stride / 2) + 32 * i);
              acc[i] = acc[i] + f2(x.x, x.y);
            }
          }
        }
      }
      if (!last) continue;
#pragma unroll
      for (int run = 0; run < kRuns; ++run) {
        float out[kRun];
#pragma unroll
        for (int i = 0; i < kRun / 2; ++i) split(acc[run * (kRun / 2) + i], out[2 * i], out[2 * i + 1]);
        epi(row0, col + 128 * run, out, F8Box<kRuns>{{boxes + (uint32_t)((warp - 4) * Shape::kBox + run * kPairBox), lane}});
      }
    }
    if (Epi::kBoxes && lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
  }
  if (broken) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    atomicOr(status, BAKRON_DEV_TIMEOUT);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
}

// Rows of C as they are stored, in whole lines: 16-bit results whose rows
// start on 16 bytes by TMA, others row by row.
template <class T>
struct F8Rows {
  static constexpr bool kBoxes = true;
  CUtensorMap map;
  int64_t m, n;
  const float* bias;  // n, or null
  T* y;               // m x n
  bool tma;           // then n is a multiple of 8, and the bias starts on 16 bytes
  __device__ __forceinline__ int64_t rows() const { return m; }
  __device__ __forceinline__ int64_t cols() const { return n; }
  template <int kCols, int kRuns>
  __device__ __forceinline__ void operator()(int64_t row0, int64_t col, float (&v)[kCols], const F8Box<kRuns>& box) const {
    if (row0 >= m || col >= n) {
      if (sizeof(T) == 2 && tma) box.skip();
      return;
    }
    if constexpr (sizeof(T) == 2) {
      if (tma) {
        box.open();
#pragma unroll
        for (int c = 0; c < kCols; c += 8) {
          float b[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] = 0.f;
          if (bias && col + c < n) load_vec<float, 8>(bias + col + c, b);
          box.put(c / 8, pack2<T>(v[c] + b[0], v[c + 1] + b[1]), pack2<T>(v[c + 2] + b[2], v[c + 3] + b[3]),
                  pack2<T>(v[c + 4] + b[4], v[c + 5] + b[5]), pack2<T>(v[c + 6] + b[6], v[c + 7] + b[7]));
        }
        box.send(&map, (int)col, (int)row0);
        return;
      }
    }
    const int here = (int)(m - row0 < 32 ? m - row0 : 32);
#pragma unroll
    for (int c = 0; c < kCols; c += 32) {
      if (col + c >= n) break;
      float w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = v[c + i];
      const int64_t o = col + c + box.lane;
      const bool in = o < n;
      const float b = in && bias ? bias[o] : 0.f;
      T* to = y + row0 * n + o;
      box.by_row(w, here, in, [&](int r, float x) { to[r * n] = from_f32<T>(x + b); });
    }
  }
};

// Columns of C as the stored rows: lanes hold neighbours of a stored row.
template <class T>
struct F8Columns {
  static constexpr bool kBoxes = false;
  int64_t m, n;
  const float* bias;  // m, or null
  T* y;               // n x m
  __device__ __forceinline__ int64_t rows() const { return m; }
  __device__ __forceinline__ int64_t cols() const { return n; }
  template <int kCols, int kRuns>
  __device__ __forceinline__ void operator()(int64_t row0, int64_t col, float (&v)[kCols], const F8Box<kRuns>& box) const {
    const int64_t o = row0 + box.lane;
    const bool in = o < m;
    const int here = in ? (int)(n - col < kCols ? n - col : kCols) : 0;  // may be negative
    const float b = in && bias ? bias[o] : 0.f;
    T* to = y + col * m + o;
#pragma unroll
    for (int i = 0; i < kCols; ++i, to += m) store_if(i < here, to, v[i] + b);
  }
};

struct F8Operand {
  const void* p;
  int64_t rows, ld;  // with K contiguous rows x K; else K x rows
};

// early: the kernel before may still run when this one starts.
template <bool kARows, bool kBRows, int kN, int kWeights, bool kJoin, class Epi>
cudaError_t fp8_pair_launch_as(F8Operand a, F8Operand b, int64_t K, const PairWork& work, const F8Scales& sc, const F8Join& join,
                            const Epi& epi, bool early, int32_t* status, cudaStream_t stream, int32_t first_status) {
  using Shape = F8Shape<kN, kBRows, kWeights != 2, kWeights != 1, Epi::kBoxes>;
  CUtensorMap ma, mb;
  const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  cudaError_t e = make_tensor_map(&ma, kARows ? TileMap{a.p, type, K, a.rows, a.ld, kF8K, 128, true}
                                              : TileMap{a.p, type, a.rows, K, a.ld, 128, kF8K, true});
  if (e == cudaSuccess)
    e = make_tensor_map(&mb, kBRows ? TileMap{b.p, type, K, b.rows, b.ld, kF8K, Shape::kCopied, true}
                                    : TileMap{b.p, type, b.rows, K, b.ld, kN / 2, kF8K, true});
  auto kernel = fp8_pair_kernel<kARows, kBRows, kN, kWeights, kJoin, Epi>;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)std::min(work.units(), pair_count()));
  cfg.blockDim = dim3(kF8Threads);
  cfg.dynamicSmemBytes = Shape::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = early ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, ma, mb, work, sc, join, epi, status, first_status);
}
template <bool kARows, bool kBRows, int kN, int kWeights, class Epi>
cudaError_t fp8_pair_launch(F8Operand a, F8Operand b, int64_t K, const PairWork& work, const F8Scales& sc, const F8Join& join,
                            const Epi& epi, bool early, int32_t* status, cudaStream_t stream, int32_t first_status) {
  if (kN == 256 && kWeights == 2 && work.parts == 1)
    return fp8_pair_launch_as<kARows, kBRows, kN, kWeights, false>(a, b, K, work, sc, join, epi, early, status, stream, first_status);
  return fp8_pair_launch_as<kARows, kBRows, kN, kWeights, true>(a, b, K, work, sc, join, epi, early, status, stream, first_status);
}

}  // namespace bakron
