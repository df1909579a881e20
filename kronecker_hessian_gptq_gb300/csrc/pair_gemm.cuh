// pair_gemm.cuh -- C = A B^T in 16-bit floats with fp32 sums on pairs of SMs,
// for the layer operators whose work is one large matrix product each.
//
// A cluster of two blocks computes one 256 x 256 tile at a time: each block
// keeps 128 rows of A and 128 rows of B for every 64 of K in shared memory
// (five or six stages of 32 KB, filled by TMA with the 128-byte swizzle), the even
// block's MMA thread issues tcgen05.mma with cta_group::2 (M = N = 256,
// K = 16), which reads both blocks' operands, and each block's tensor memory
// receives 128 rows of the sums.  Two sums of 256 columns take turns, so that
// the epilogue warps read one while the MMAs fill the other.  One pair stays
// on two SMs and walks over the units (tile, part of K) it is given.
//
// Either operand may be stored with K contiguous or with its rows (M or N)
// contiguous: the canonical layouts differ only in the boxes TMA copies and
// in the descriptors' offsets.
//
// With kSegment > 0 the sums are restarted every kSegment steps of 64 and
// added up by the epilogue: in integers, so that products of 8-bit codes stay
// exact (1024 products of at most 2^14 reach 2^24, where fp32 integers end), or
// in fp32, rounded to nearest where the tensor cores round towards zero.
#pragma once

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "bakron.h"
#include "elem.cuh"
#include "tc.cuh"
#include "tma.h"

namespace bakron {

constexpr int kPairTile = 256;    // rows and columns of a pair's tile
constexpr int kPairK = 64;        // K of a stage: 128 bytes
constexpr int kPairHalf = 128 * kPairK * 2;        // one block's part of an operand's stage: 16 KB
constexpr uint32_t kPairStageTx = 4u * kPairHalf;  // bytes of a stage in both blocks
constexpr int kPairBox = 4096;  // shared memory of an epilogue warp: 32 rows of 128 bytes
// Epilogue warps are 4 kQuads; more of them leave room for fewer stages.
template <int kQuads>
__host__ __device__ constexpr int pair_stages() { return kQuads > 2 ? 5 : 6; }
template <int kQuads>
constexpr int pair_smem() { return pair_stages<kQuads>() * 2 * kPairHalf + 4 * kQuads * kPairBox + 1024; }

// Units of a product: unit u = (tile, part of K); tiles run down groups of
// `group` tile rows first, so that what runs at the same time shares operands
// in the L2 cache.
struct PairWork {
  int tiles_m, tiles_n, group;
  int ksteps;  // stages of K
  int parts;   // parts that K is cut into
  __host__ __device__ int units() const { return tiles_m * tiles_n * parts; }
};
struct PairUnit {
  int tm, tn, part, k0, k1;
};
__host__ __device__ inline PairUnit pair_unit(const PairWork& w, int u) {
  PairUnit r;
  const int tiles = w.tiles_m * w.tiles_n;
  r.part = u / tiles;
  const int t = u % tiles;
  const int g = t / (w.group * w.tiles_n), first = g * w.group;
  const int rows = w.tiles_m - first < w.group ? w.tiles_m - first : w.group;
  const int in = t - g * w.group * w.tiles_n;
  r.tm = first + in % rows;
  r.tn = in / rows;
  r.k0 = (int)((int64_t)w.ksteps * r.part / w.parts);
  r.k1 = (int)((int64_t)w.ksteps * (r.part + 1) / w.parts);
  return r;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
// Address of the even block's copy of a shared variable.
__device__ __forceinline__ uint32_t in_even_block(const void* p) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// Place in a ring of stages: the slot, the parity of its barriers in this
// round, and whether the slot has been used before.
struct Ring {
  int slot = 0;
  uint32_t turn = 0;
  bool round = false;
  __device__ __forceinline__ void next(int stages) {
    if (++slot == stages) slot = 0, turn ^= 1u, round = true;
  }
};
// A converged warp's wait for the phase of the given parity, for at most about
// 0.1 s (2^28 cycles); afterwards `broken` is set for the whole warp, and
// later waits return at once.  Every branch is taken by a vote, so that the
// compiler knows the warp to stay together: the descriptors of the MMAs then
// live in uniform registers (issuing four with the wait takes 360 to 480
// cycles, so 480 to 600 without), and the first look costs no clock reading.
__device__ __forceinline__ bool phase_done(uint64_t* mbar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(done)
               : "r"(smem_u32(mbar)), "r"(parity)
               : "memory");
  return __all_sync(0xffffffffu, done) != 0;
}
__device__ __forceinline__ void warp_wait(uint64_t* mbar, uint32_t parity, bool& broken) {
  if (broken || phase_done(mbar, parity)) return;
  const long long t0 = clock64();
  while (!phase_done(mbar, parity)) {
    if (__any_sync(0xffffffffu, clock64() - t0 > (1ll << 28))) {
      broken = true;
      return;
    }
  }
}
// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// A box into this block's shared memory; its bytes count on the even block's barrier.
__device__ __forceinline__ void pair_copy(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(mbar)
      : "memory");
}
// Arrives on the barrier at this offset in both blocks once all MMAs issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t* mbar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
          smem_u32(mbar)),
      "h"((uint16_t)3)
      : "memory");
}
// The operands' descriptors come as their low words, which hold the address in
// units of 16 bytes, and the high words that all steps share.
__device__ __forceinline__ void pair_mma(uint32_t d, uint32_t a, uint32_t a_high, uint32_t b, uint32_t b_high, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 da, db;\nmov.b64 da, {%1, %2};\nmov.b64 db, {%3, %4};\nsetp.ne.b32 p, %6, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n}\n" ::"r"(d),
      "r"(a), "r"(a_high), "r"(b), "r"(b_high), "r"(idesc), "r"(acc));
}
// 32 consecutive columns of this warp's 32 tensor-memory lanes; complete after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// A store to memory under a predicate: as a branch for each value it costs a
// warp 150 cycles a value.
__device__ __forceinline__ void store_if(bool p, float* to, float x) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %2, 0;\n@p st.global.f32 [%0], %1;\n}\n" ::"l"(to), "f"(x), "r"((int)p)
               : "memory");
}
template <class T>
__device__ __forceinline__ void store_if(bool p, T* to, float x) {
  const T v = from_f32<T>(x);
  uint16_t bits;
  memcpy(&bits, &v, 2);
  asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %2, 0;\n@p st.global.b16 [%0], %1;\n}\n" ::"l"(to), "h"(bits), "r"((int)p)
               : "memory");
}

// Shared memory descriptors with the 128-byte swizzle (layout type 2).  K
// contiguous: 8-row groups of 1024 bytes (stride offset).  Rows contiguous:
// 64 rows by 8 of K take 1024 bytes, the next 8 of K follow (stride offset),
// the next 64 rows are 8 KB on (leading offset).
template <bool kRows>
__device__ __forceinline__ uint32_t pair_desc_low(uint32_t saddr) { return (saddr >> 4) | ((kRows ? 8192u >> 4 : 1u) << 16); }
constexpr uint32_t kPairDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride offset, version, swizzle
// Units of 16 bytes from one K = 16 step to the next within a stage.
template <bool kRows>
__host__ __device__ constexpr uint32_t pair_kstep() { return kRows ? 2048u >> 4 : 32u >> 4; }

struct PairBarriers {
  uint64_t full[6], empty[6], sum_full[2], sum_empty[2];
  uint32_t tmem;
};

// The epilogue (which may hold tensor maps: it stays in the parameters) is called by every thread of 4 kQuads warps for each unit,
//   epi(unit, row0, col, ahead, sums, box)
// with the warp's first row (the thread's own is lane further) and first
// column, what epi.ahead(row) read for the thread's row while the unit before
// was at hand (Epi::kAhead: 0 without it), and a source of its 256 / kQuads
// columns: sums.load(c, v) gives 32 of them from column c on.  With kSegment it
// is an array of Epi::Sum instead.
struct PairSums {
  uint32_t taddr;
  __device__ __forceinline__ void load(int c, float (&v)[32]) const { tmem_ld32(taddr + (uint32_t)c, v); }
};

// An epilogue warp's 4 KB of shared memory, 32 rows of 128 bytes, through
// which its results leave in whole lines: a thread holds one row's sums, so
// storing them from registers would write 16 bytes of 32 different lines at a
// time (measured: 11 us for a 256 x 256 tile of 16-bit results, more than the
// products of 1024 terms take).  The 16-byte pieces of row r are kept at
// place j ^ (r % 8), the 128-byte swizzle of TMA, free of bank conflicts.
struct PairBox {
  uint32_t smem;
  int lane;
  __device__ __forceinline__ uint32_t piece(int row, int j) const { return smem + (uint32_t)(row * 128 + ((j ^ (row & 7)) << 4)); }
  // Before the first put() of a box: the last one's copy has been read.
  __device__ __forceinline__ void open() const {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
    __syncwarp();
  }
  __device__ __forceinline__ void put(int j, uint32_t a, uint32_t b, uint32_t c, uint32_t d) const {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(piece(lane, j)), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
  }
  // The box to column x and row y of the map's matrix; what lies outside it is left out.
  __device__ __forceinline__ void send(const CUtensorMap* map, int x, int y) const {
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(map), "r"(x),
                   "r"(y), "r"(smem)
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
    }
  }
  // 32 fp32 sums of each row, then given back row by row, a column for each
  // thread: f(r, v) with row r's sum in column `lane`, for the threads with
  // `in`.  One branch for all rows: a branch in each row would cost more than
  // the row.
  template <class F>
  __device__ __forceinline__ void by_row(const float (&v)[32], int rows, bool in, F f) const {
    open();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      put(j, __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
    __syncwarp();
    if (in) {
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += 8) {
        float x[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          asm volatile("ld.shared.f32 %0, [%1];\n"
                       : "=f"(x[r])
                       : "r"(piece(r0 + r, lane >> 2) + (uint32_t)(lane & 3) * 4u)
                       : "memory");
        if (r0 + 8 <= rows) {
#pragma unroll
          for (int r = 0; r < 8; ++r) f(r0 + r, x[r]);
        } else {
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r0 + r < rows) f(r0 + r, x[r]);
        }
      }
    }
    __syncwarp();
  }
};

template <bool kARows, bool kBRows, int kQuads, int kSegment, class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(128 + 128 * kQuads, 1)
    pair_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, PairWork work,
                     uint32_t idesc, const __grid_constant__ Epi epi, int32_t* status, int32_t first_status) {
  extern __shared__ unsigned char pair_smem_raw[];
  const uint32_t base = (smem_u32(pair_smem_raw) + 1023u) & ~1023u;
  __shared__ PairBarriers bar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  constexpr int kPairStages = pair_stages<kQuads>();
  const uint32_t boxes = base + kPairStages * 2u * kPairHalf;
  const int pairs = gridDim.x / 2, mine = blockIdx.x / 2, units = work.units();
  bool broken = false;

  asm volatile("griddepcontrol.launch_dependents;\n");
  // This early nothing can have been reported.
  if (first_status >= 0 && blockIdx.x == 0 && threadIdx.x == 0) *status = first_status;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(smem_u32(&bar.full[i])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(smem_u32(&bar.empty[i])));
    }
    for (int i = 0; i < 2; ++i) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(smem_u32(&bar.sum_full[i])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(&bar.sum_empty[i])), "r"(8 * kQuads));
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

  if (warp == 0) {  // copies: 16 KB of A and of B for each stage, in both blocks
    Ring ring;
    for (int u = mine; u < units && !broken; u += pairs) {
      const PairUnit q = pair_unit(work, u);
      const int a0 = q.tm * kPairTile + (int)rank * 128, b0 = q.tn * kPairTile + (int)rank * 128;
      for (int k = q.k0; k < q.k1; ++k, ring.next(kPairStages)) {
        const int slot = ring.slot;
        if (ring.round) warp_wait(&bar.empty[slot], ring.turn ^ 1u, broken);
        if (broken) break;
        const uint32_t full = in_even_block(&bar.full[slot]);
        const uint32_t a = base + (uint32_t)slot * 2u * kPairHalf, b = a + kPairHalf;
        if (elect_one()) {
          if (rank == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(&bar.full[slot])),
                         "r"(kPairStageTx)
                         : "memory");
          if constexpr (kARows) {
            pair_copy(a, &map_a, a0, k * kPairK, full);
            pair_copy(a + 8192, &map_a, a0 + 64, k * kPairK, full);
          } else {
            pair_copy(a, &map_a, k * kPairK, a0, full);
          }
          if constexpr (kBRows) {
            pair_copy(b, &map_b, b0, k * kPairK, full);
            pair_copy(b + 8192, &map_b, b0 + 64, k * kPairK, full);
          } else {
            pair_copy(b, &map_b, k * kPairK, b0, full);
          }
        }
        __syncwarp();
      }
    }
    // No block leaves while copies into it, or arrivals at its barriers, are
    // on their way: every stage's last use has been released by the MMAs (or,
    // after a wait that ran out, has at least landed).
    for (int i = 0; i < kPairStages; ++i, ring.next(kPairStages)) {
      if (!ring.round) continue;  // this stage's first use would come here
      bool late = false;
      if (!broken)
        warp_wait(&bar.empty[ring.slot], ring.turn ^ 1u, broken);
      else if (rank == 0)
        warp_wait(&bar.full[ring.slot], ring.turn ^ 1u, late);
    }
  } else if (warp == 1 && rank == 0) {  // products
    // The whole warp walks the loop and one elected thread issues: with the
    // warp converged the descriptors stay in uniform registers (under a
    // branch on the lane a step of K took 670 cycles, so 590).
    int sums = 0;
    Ring ring;
    for (int u = mine; u < units && !broken; u += pairs) {
      const PairUnit q = pair_unit(work, u);
      uint32_t acc = 0;
      for (int k = q.k0; k < q.k1; ++k, ring.next(kPairStages)) {
        const int in_segment = kSegment ? (k - q.k0) % kSegment : k - q.k0;
        if (in_segment == 0) {  // the next of the two sums, once the epilogue has read it
          acc = tmem + (uint32_t)(sums & 1) * 256u;
          if (sums >= 2) warp_wait(&bar.sum_empty[sums & 1], (uint32_t)(sums / 2 - 1) & 1u, broken);
          tc_fence_after();
        }
        const int slot = ring.slot;
        warp_wait(&bar.full[slot], ring.turn, broken);
        if (broken) break;
        tc_fence_after();
        const uint32_t at = base + (uint32_t)slot * 2u * kPairHalf;
        const uint32_t a = pair_desc_low<kARows>(at), b = pair_desc_low<kBRows>(at + kPairHalf);
        const bool sum_done = k + 1 == q.k1 || (kSegment && in_segment == kSegment - 1);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kPairK / 16; ++j)
            pair_mma(acc, a + j * pair_kstep<kARows>(), kPairDescHigh, b + j * pair_kstep<kBRows>(), kPairDescHigh, idesc,
                     (in_segment > 0 || j > 0) ? 1u : 0u);
          pair_commit(&bar.empty[slot]);
          if (sum_done) pair_commit(&bar.sum_full[sums & 1]);
        }
        __syncwarp();
        if (sum_done) ++sums;
      }
    }
  } else if (warp >= 4) {  // epilogue: 32 rows of the block and 256 / kQuads columns for each warp
    constexpr int kCols = 256 / kQuads;
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    const uint32_t lanes = ((uint32_t)(32 * quarter) << 16) + (uint32_t)(part * kCols);
    const PairBox box{boxes + (uint32_t)(warp - 4) * kPairBox, lane};
    int sums = 0;
    auto row_of = [&](const PairUnit& q) { return (int64_t)q.tm * kPairTile + rank * 128 + 32 * quarter; };
    PairUnit q = pair_unit(work, mine), next = q;
    int64_t read = 0, ahead = 0;
    if constexpr (Epi::kAhead) ahead = epi.ahead(row_of(q) + lane);
    for (int u = mine; u < units && !broken; u += pairs) {
      if constexpr (Epi::kAhead) {
        q = next, read = ahead;
        if (u + pairs < units) {
          next = pair_unit(work, u + pairs);
          ahead = epi.ahead(row_of(next) + lane);
        }
      } else {
        q = pair_unit(work, u);
      }
      const int64_t row = row_of(q);
      const int64_t col = (int64_t)q.tn * kPairTile + part * kCols;
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(
                           in_even_block(&bar.sum_empty[sums & 1]))
                       : "memory");
        ++sums;
      };
      if constexpr (kSegment == 0) {
        warp_wait(&bar.sum_full[sums & 1], (uint32_t)(sums / 2) & 1u, broken);
        if (broken) break;
        tc_fence_after();
        epi(q, row, col, read, PairSums{tmem + (uint32_t)(sums & 1) * 256u + lanes}, box);
        release();
      } else {
        typename Epi::Sum acc[kCols];
        for (int k = q.k0; k < q.k1; k += kSegment) {
          warp_wait(&bar.sum_full[sums & 1], (uint32_t)(sums / 2) & 1u, broken);
          if (broken) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kCols; c += 32) {
            float v[32];
            tmem_ld32(tmem + (uint32_t)(sums & 1) * 256u + lanes + (uint32_t)c, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if constexpr (std::is_same<typename Epi::Sum, int>::value)
                acc[c + i] = __float2int_rn(v[i]) + (k == q.k0 ? 0 : acc[c + i]);
              else
                acc[c + i] = k == q.k0 ? v[i] : acc[c + i] + v[i];
            }
          }
          release();
        }
        if (!broken) epi(q, row, col, read, acc, box);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
  }
  if (broken) atomicOr(status, BAKRON_DEV_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
}

// An operand, 16-bit: rows x K with K contiguous, or K x rows with its rows
// contiguous (kARows, kBRows).
struct PairOperand {
  const void* p;
  int64_t rows, ld;
};

// Pairs of SMs on the current device.
inline int pair_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 1;
  return std::max(1, sms / 2);
}

// M x N tiles of A (M x K) and B (N x K).  bf16: both bf16, else both fp16.
// first_status >= 0: the status word is set to it first.
template <bool kARows, bool kBRows, int kQuads, int kSegment, class Epi>
cudaError_t pair_gemm_launch(PairOperand a, PairOperand b, int64_t K, bool bf16, PairWork work, const Epi& epi,
                             int32_t* status, cudaStream_t stream, int32_t first_status = -1) {
  const CUtensorMapDataType type = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap ma, mb;
  auto map = [&](CUtensorMap* m, const PairOperand& o, bool rows) {
    return rows ? make_tensor_map(m, TileMap{o.p, type, K, o.rows, o.ld, kPairK, 64, true})
                : make_tensor_map(m, TileMap{o.p, type, o.rows, K, o.ld, 128, kPairK, true});
  };
  cudaError_t e = map(&ma, a, kARows);
  if (e == cudaSuccess) e = map(&mb, b, kBRows);
  if (e != cudaSuccess) return e;
  auto kernel = pair_gemm_kernel<kARows, kBRows, kQuads, kSegment, Epi>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pair_smem<kQuads>());
  if (e != cudaSuccess) return e;
  const unsigned grid = 2u * (unsigned)std::min(work.units(), pair_count());
  // fp32 sums, operand types, which operands have their rows contiguous, N = 256, M = 256
  const uint32_t t = bf16 ? 1u : 0u;
  const uint32_t idesc = (1u << 4) | (t << 7) | (t << 10) | ((kARows ? 1u : 0u) << 15) | ((kBRows ? 1u : 0u) << 16) |
                         ((256u >> 3) << 17) | ((256u >> 4) << 24);
  kernel<<<grid, 128 + 128 * kQuads, pair_smem<kQuads>(), stream>>>(ma, mb, work, idesc, epi, status, first_status);
  return cudaGetLastError();
}

}  // namespace bakron
