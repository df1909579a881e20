// int8_pair.cuh -- the product of 8-bit weights with a batch of tokens on
// pairs of SMs, for batches that are bound by reading the weights.
//
// The chip has no fast 8-bit integer products (tcgen05 kind::i8 is absent from
// sm_103a), but an 8-bit integer is exact in fp16, its products are exact in
// fp32, and sums of 1024 of them stay below 2^24: so the weights are read as
// bytes, converted on their way to the tensor cores and multiplied with
// kind::f16, and sums of at most 1024 terms are joined as 32-bit integers.
//
// A cluster of two blocks takes 256 outputs (the MMA's rows, 128 for each
// block) against up to 128 tokens (its columns).  The weights' bytes come by
// TMA (128 of K, 16 KB a step in each block, up to ten steps on their way).
// Two groups of four warps turn every second step into fp16 each and put it
// straight into tensor memory, where the MMAs read their A operand: a thread
// holds a row's 128 values in registers and stores 64 columns.  Through shared
// memory the fp16 would be written and read once more.  The tokens' codes are
// the MMAs' B operand in shared memory (TMA, already fp16).  A step is as long
// as tensor memory allows, because the loop that issues the MMAs takes about
// 400 cycles for its wait, its commit and sharing the scheduler with the
// converting warps, besides 50 for each MMA (39 is the least, whatever the
// number of tokens); memory can bring a step every 700.
//
// Every 1024 of K the epilogue adds the fp32 sums to integers, which stay in
// tensor memory while a piece is longer than that.  A pair of SMs is given
// either whole tiles or, where that would leave too many pairs idle, an equal
// part of one tile or an equal share of all tiles' steps; then the pieces of a tile are joined in memory
// with integer atomics, whose order does not matter, and the last to arrive
// scales a slice's sums and writes the results.
#pragma once

#include "elem.cuh"
#include "pair_gemm.cuh"

namespace bakron {

constexpr int kI8K = 128;                  // K of a step
constexpr int kI8Raw = 128 * kI8K;         // bytes of weights of a step: 16 KB
constexpr int kI8A = kI8K / 2;             // a step's weights in fp16: columns of tensor memory
constexpr int kI8Tokens = 128;             // tokens of a tile at most
constexpr int kI8Groups = 2;               // converting groups
constexpr int kI8MostOps = 4;              // steps of operands
constexpr int kI8MostRaw = 10;
constexpr int kI8Segment = 8;              // steps of a sum in fp32: 1024 of K
constexpr int kI8Convert = 4 * kI8Groups;  // converting warps
constexpr int kI8Threads = (4 + kI8Convert + 8) * 32;
constexpr int kI8SmemMost = 224 * 1024;

struct I8Work {
  int tiles_m, tiles_n, nt;  // outputs / 256, token tiles of nt tokens (a multiple of 32)
  int ksteps;
  int raws, ops;  // steps of the rings of bytes and of operands
  int bufs;       // sums in tensor memory: two take turns where they leave room for enough operands
  int pairs;     // that have work
  bool shared;   // each has an equal share of the steps, else whole tiles in turn
  // A step's codes of the half of the tile's tokens that a block holds: two panels of 64 of K.
  __host__ __device__ int op_bytes() const { return nt / 2 * kI8K * 2; }
  __host__ __device__ int tiles() const { return tiles_m * tiles_n; }
  // Pieces that a tile is cut into: the pairs that the first to the last of its steps belong to.
  __host__ __device__ int pieces(int tile) const {
    if (!shared) return 1;
    const int64_t all = (int64_t)tiles() * ksteps, first = (int64_t)tile * ksteps;
    const int64_t p0 = ((first + 1) * pairs - 1) / all, p1 = ((first + ksteps) * pairs - 1) / all;
    return (int)(p1 - p0) + 1;
  }
};
// The pieces of one pair: steps k0 .. k1 - 1 of a tile each.  Tiles that share
// weights follow one another.
struct I8Walk {
  int64_t at, end;
  int tile, tm, tn, k0, k1;
  __device__ I8Walk(const I8Work& w, int pair) {
    const int64_t all = (int64_t)w.tiles() * w.ksteps;
    at = w.shared ? all * pair / w.pairs : pair;
    end = w.shared ? all * (pair + 1) / w.pairs : w.tiles();
  }
  __device__ __forceinline__ bool next(const I8Work& w) {
    if (at >= end) return false;
    if (w.shared) {
      tile = (int)(at / w.ksteps);
      k0 = (int)(at - (int64_t)tile * w.ksteps);
      const int64_t left = end - at;
      k1 = left < w.ksteps - k0 ? k0 + (int)left : w.ksteps;
      at += k1 - k0;
    } else {
      tile = (int)at;
      k0 = 0, k1 = w.ksteps;
      at += w.pairs;
    }
    tn = tile % w.tiles_n;
    tm = tile / w.tiles_n;
    return true;
  }
};

template <class T>
struct I8Out {
  int64_t tokens, outputs;
  const float *x_scales, *w_scales, *bias;
  T* y;
  int32_t* sums;      // tokens x outputs, zero; used where tiles are shared
  uint32_t* arrived;  // a counter for each slice of 32 outputs and half a token tile, zero
};

struct I8Barriers {
  uint64_t raw_full[kI8MostRaw], raw_empty[kI8MostRaw], ready[kI8MostOps], empty[kI8MostOps], sum_full[2], sum_empty[2];
  uint32_t tmem;
};

// As pair_mma with the A operand in tensor memory (in both blocks' own).
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_high, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 db;\nmov.b64 db, {%2, %3};\nsetp.ne.b32 p, %5, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], db, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(b_high), "r"(idesc), "r"(acc));
}

// Four 8-bit integers as fp16: with the sign bit flipped a byte b is the
// value + 128, and 0x6400 + b is the fp16 number 1024 + b, exactly.
__device__ __forceinline__ void i8_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u, magic = 0x64646464u, off = 0x64806480u;  // 1152
  const uint32_t a = __byte_perm(u, magic, 0x4140), b = __byte_perm(u, magic, 0x4342);
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(lo) : "r"(a), "r"(off));
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(hi) : "r"(b), "r"(off));
}

// 32 columns of 32 lanes from and to tensor memory; several may be under way,
// complete after the wait for loads or stores.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]),
        "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
// The loads of v are complete (and nothing that reads v moves ahead of this).
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]),
      "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31])
      : "memory");
}
// An integer sum to memory under a predicate (see store_if).
__device__ __forceinline__ void add_if(bool p, int32_t* to, int x) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %2, 0;\n@p red.global.add.s32 [%0], %1;\n}\n" ::"l"(to), "r"(x), "r"((int)p)
               : "memory");
}

// 16 of v, from the kFrom-th on.
template <int kFrom>
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(v[kFrom]), "r"(v[kFrom + 1]), "r"(v[kFrom + 2]), "r"(v[kFrom + 3]), "r"(v[kFrom + 4]), "r"(v[kFrom + 5]),
      "r"(v[kFrom + 6]), "r"(v[kFrom + 7]), "r"(v[kFrom + 8]), "r"(v[kFrom + 9]), "r"(v[kFrom + 10]), "r"(v[kFrom + 11]),
      "r"(v[kFrom + 12]), "r"(v[kFrom + 13]), "r"(v[kFrom + 14]), "r"(v[kFrom + 15])
      : "memory");
}

template <class T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kI8Threads, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, I8Work work,
                     I8Out<T> out, int32_t* status) {
  // The kernel may start before the one that prepares the tokens' codes, their
  // scales and the zeros has ended: the weights are read at once, and who
  // needs the others waits (griddepcontrol.wait).
  extern __shared__ unsigned char i8_smem_raw[];
  __shared__ I8Barriers bar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int mine = blockIdx.x / 2, raws = work.raws, ops = work.ops;
  const uint32_t codes = (smem_u32(i8_smem_raw) + 1023u) & ~1023u, op = (uint32_t)work.op_bytes();
  const uint32_t bytes = codes + (uint32_t)ops * op;
  bool broken = false;

  if (threadIdx.x == 0) {
    auto init = [](uint64_t* b, int n) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(b)), "r"(n));
    };
    for (int i = 0; i < raws; ++i) {
      init(&bar.raw_full[i], 1);
      init(&bar.raw_empty[i], 4);  // a group's warps
    }
    for (int i = 0; i < ops; ++i) {
      init(&bar.ready[i], 1 + 2 * 4);  // the tokens' copies, and a group's warps in both blocks
      init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      init(&bar.sum_full[i], 1);
      init(&bar.sum_empty[i], 2 * 8);
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
  // tensor memory: the kept integers and the sums, a column for each token; the weights
  const uint32_t nt = (uint32_t)work.nt, weights = tmem + (1 + work.bufs) * nt;
  const int two = work.bufs - 1;  // sum n is in buffer n & two, for the (n >> two)-th time
  I8Walk q(work, mine);

  if (warp == 0) {  // the weights' bytes
    Ring ring;
    while (!broken && q.next(work)) {
      for (int k = q.k0; k < q.k1; ++k, ring.next(raws)) {
        if (ring.round) warp_wait(&bar.raw_empty[ring.slot], ring.turn ^ 1u, broken);
        if (broken) break;
        if (elect_one()) {
          const uint32_t full = smem_u32(&bar.raw_full[ring.slot]);
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(full), "r"(kI8Raw) : "memory");
          asm volatile(
              "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
                  bytes + (uint32_t)ring.slot * kI8Raw),
              "l"(&map_w), "r"(k * kI8K), "r"(q.tm * 256 + (int)rank * 128), "r"(full)
              : "memory");
        }
        __syncwarp();
      }
    }
    // Nothing is on its way into a block that leaves (see pair_gemm_kernel).
    for (int i = 0; i < raws; ++i, ring.next(raws)) {
      bool late = false;
      if (ring.round) warp_wait(&bar.raw_full[ring.slot], ring.turn ^ 1u, late);
    }
  } else if (warp == 3) {  // the tokens' codes
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    Ring ring;
    while (!broken && q.next(work)) {
      const int t0 = q.tn * work.nt + (int)rank * (work.nt / 2);
      for (int k = q.k0; k < q.k1; ++k, ring.next(ops)) {
        if (ring.round) warp_wait(&bar.empty[ring.slot], ring.turn ^ 1u, broken);
        if (broken) break;
        const uint32_t ready = in_even_block(&bar.ready[ring.slot]), x = codes + (uint32_t)ring.slot * op;
        if (elect_one()) {
          if (rank == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(&bar.ready[ring.slot])),
                         "r"(2u * op)
                         : "memory");
          pair_copy(x, &map_x, k * kI8K, t0, ready);
          pair_copy(x + op / 2, &map_x, k * kI8K + 64, t0, ready);
        }
        __syncwarp();
      }
    }
    for (int i = 0; i < ops; ++i, ring.next(ops)) {
      bool late = false;
      if (!ring.round) continue;
      if (!broken)
        warp_wait(&bar.empty[ring.slot], ring.turn ^ 1u, broken);
      else if (rank == 0)
        warp_wait(&bar.ready[ring.slot], ring.turn ^ 1u, late);
    }
  } else if (warp == 1 && rank == 0) {  // products
    // fp32 sums of fp16 products, both with K contiguous, M = 256, N = nt
    const uint32_t idesc = (1u << 4) | ((uint32_t)(work.nt >> 3) << 17) | ((256u >> 4) << 24);
    int sums = 0;
    Ring ring;
    while (!broken && q.next(work)) {
      int in_segment = 0;
      for (int k = q.k0; k < q.k1; ++k, ring.next(ops)) {
        const uint32_t acc = tmem + (1 + (uint32_t)(sums & two)) * nt;
        if (in_segment == 0 && sums > two) warp_wait(&bar.sum_empty[sums & two], (uint32_t)((sums >> two) - 1) & 1u, broken);
        warp_wait(&bar.ready[ring.slot], ring.turn, broken);
        if (broken) break;
        tc_fence_after();
        const uint32_t a = weights + (uint32_t)(ring.slot * kI8A), x = pair_desc_low<false>(codes + (uint32_t)ring.slot * op);
        const bool sum_done = k + 1 == q.k1 || in_segment == kI8Segment - 1;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kI8K / 16; ++j)
            pair_mma_ts(acc, a + 8 * j, x + (j / 4) * (op >> 5) + 2 * (j % 4), kPairDescHigh, idesc,
                        (in_segment > 0 || j > 0) ? 1u : 0u);
          pair_commit(&bar.empty[ring.slot]);
          if (sum_done) pair_commit(&bar.sum_full[sums & two]);
        }
        __syncwarp();
        ++in_segment;
        if (sum_done) ++sums, in_segment = 0;
      }
    }
  } else if (warp >= 4 && warp < 4 + kI8Convert) {  // bytes to fp16: 32 rows of every second step for each warp
    const int group = (warp - 4) >> 2, quarter = (warp - 4) & 3;
    // A thread takes a row; its 16-byte pieces lie where the 128-byte swizzle
    // of TMA puts them, so that eight rows' pieces touch all banks.
    const int row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    int turn = 0;
    Ring ring, raw;
    while (!broken && q.next(work)) {
      for (int k = q.k0; k < q.k1; ++k, turn ^= 1, ring.next(ops), raw.next(raws)) {
        if (turn != group) continue;
        warp_wait(&bar.raw_full[raw.slot], raw.turn, broken);
        if (broken) break;
        const uint32_t from = bytes + (uint32_t)(raw.slot * kI8Raw + row * kI8K);
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                       : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                       : "r"(from + (uint32_t)((i ^ (row & 7)) << 4))
                       : "memory");
        uint32_t h[2][32];
#pragma unroll
        for (int i = 0; i < 32; ++i) i8_to_f16(w[i], h[i / 16][2 * (i % 16)], h[i / 16][2 * (i % 16) + 1]);
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(&bar.raw_empty[raw.slot])) : "memory");
        if (ring.round) warp_wait(&bar.empty[ring.slot], ring.turn ^ 1u, broken);
        if (broken) break;
        const uint32_t to = weights + lanes + (uint32_t)(ring.slot * kI8A);
        tmem_st32(to, h[0]);
        tmem_st32(to + 32, h[1]);
        asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
        tc_fence_before();
        __syncwarp();
        // A release of cluster scope here would stall the warp for half a
        // microsecond in every step; the tensor-memory stores are complete.
        if (lane == 0)
          asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(in_even_block(&bar.ready[ring.slot])) : "memory");
      }
    }
  } else if (warp >= 4 + kI8Convert) {  // epilogue: 32 outputs (lanes) and half of a tile's tokens for each warp
    const int quarter = warp & 3, part = (warp - 4 - kI8Convert) >> 2;
    const int cols = work.nt / 2, c0 = part * cols;
    const uint32_t lanes = ((uint32_t)(32 * quarter) << 16) + (uint32_t)c0;
    const uint32_t kept = tmem + lanes;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    int sums = 0;
    while (!broken && q.next(work)) {
      const int64_t o = (int64_t)q.tm * 256 + rank * 128 + 32 * quarter + lane;
      const int64_t t0 = (int64_t)q.tn * work.nt + c0;
      const int pieces = work.pieces(q.tile);
      const int live = (int)(out.tokens - t0 < cols ? out.tokens - t0 : cols);  // may be negative
      const bool in = o < out.outputs;
      const float ws = in ? out.w_scales[o] : 0.f, bias = in && out.bias ? out.bias[o] : 0.f;
      // scales of the slice's tokens, one for each lane, handed out by shuffles
      const float xs[2] = {lane < live ? out.x_scales[t0 + lane] : 0.f, 32 + lane < live ? out.x_scales[t0 + 32 + lane] : 0.f};
      auto finish = [&](int c, uint32_t(&v)[32]) {  // 32 tokens' results
#pragma unroll
        for (int i = 0; i < 32; ++i)
          v[i] = __float_as_uint(fmaf((float)(int)v[i] * __shfl_sync(0xffffffffu, xs[c >> 5], i), ws, bias));
        T* to = out.y + (t0 + c) * out.outputs + o;
        const int rows = in ? live - c : 0;
#pragma unroll
        for (int i = 0; i < 32; ++i, to += out.outputs) store_if(i < rows, to, __uint_as_float(v[i]));
      };
      for (int k = q.k0; k < q.k1; k += kI8Segment, ++sums) {
        warp_wait(&bar.sum_full[sums & two], (uint32_t)(sums >> two) & 1u, broken);
        if (broken) break;
        tc_fence_after();
        const uint32_t from = kept + (1 + (uint32_t)(sums & two)) * nt;
        const bool last = k + kI8Segment >= q.k1;
        // 32 tokens at a time, the same for the whole warp; a load from tensor
        // memory takes hundreds of cycles, so both are under way together.
#pragma unroll
        for (int c = 0; c < kI8Tokens / 2; c += 32) {
          if (c >= live) break;
          uint32_t v[32], w[32];
          tmem_ld32_async(from + (uint32_t)c, v);
          if (k > q.k0) {
            tmem_ld32_async(kept + (uint32_t)c, w);
            tmem_wait(w);
          }
          tmem_wait(v);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = (uint32_t)__float2int_rn(__uint_as_float(v[i])) + (k > q.k0 ? w[i] : 0u);
          if (!last) {
            tmem_st16<0>(kept + (uint32_t)c, v);
            if (c + 16 < cols) tmem_st16<16>(kept + (uint32_t)c + 16, v);  // what follows is the other warps'
          } else if (pieces == 1) {
            finish(c, v);
          } else {
            int32_t* to = out.sums + (t0 + c) * out.outputs + o;
            const int rows = in ? live - c : 0;
#pragma unroll
            for (int i = 0; i < 32; ++i, to += out.outputs) add_if(i < rows, to, (int)v[i]);
          }
        }
        if (!last) asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(in_even_block(&bar.sum_empty[sums & two])) : "memory");
      }
      if (broken || pieces == 1 || live <= 0) continue;
      // The last of a slice's pieces to arrive reads the joined sums.
      __threadfence();
      __syncwarp();
      uint32_t before = 0;
      if (lane == 0)
        before = atomicAdd(out.arrived + ((int64_t)q.tile * 2 + rank) * 8 + part * 4 + quarter, 1u);
      before = __shfl_sync(0xffffffffu, before, 0);
      if (before + 1 != (uint32_t)pieces) continue;
      __threadfence();
#pragma unroll
      for (int c = 0; c < kI8Tokens / 2; c += 32) {
        if (c >= live) break;
        // 32 reads on their way at once; beyond the tokens or the outputs the last one's
        const int rows = live - c;
        const int32_t* sum = out.sums + (t0 + c) * out.outputs + (in ? o : out.outputs - 1);
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          v[i] = (uint32_t)__ldcg(sum);
          if (i + 1 < rows) sum += out.outputs;
        }
        finish(c, v);
      }
    }
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

inline I8Work i8_work(int64_t T, int64_t K, int64_t N, int pairs) {
  I8Work w;
  w.tiles_m = (int)((N + 255) / 256);
  w.tiles_n = (int)((T + kI8Tokens - 1) / kI8Tokens);
  // At least 64: an MMA takes no less time for 32 (24 tokens 4096 -> 14336: 25
  // us, so 21).
  w.nt = std::max(64, (int)(((T + w.tiles_n - 1) / w.tiles_n + 31) / 32 * 32));
  w.tiles_n = (int)((T + w.nt - 1) / w.nt);
  w.ksteps = (int)((K + kI8K - 1) / kI8K);
  // Whole tiles, or equal shares of all steps?  In steps of K: a tile's end
  // costs about 2, a shared tile's 6 and 1 more for every 16 tokens, which
  // are added up in memory.
  const int64_t tiles = w.tiles(), all = tiles * w.ksteps;
  const int64_t whole = (tiles + pairs - 1) / pairs * (w.ksteps + 2), share = (all + pairs - 1) / pairs + 6 + w.nt / 16;
  w.shared = share < whole;
  w.pairs = (int)std::min<int64_t>(w.shared ? all : tiles, pairs);
  // A share that ends one tile and begins another has two ends to wait for.
  // As many pairs for each tile have one, at 2 steps and 1 for every 32 tokens
  // less (128 tokens 4096 -> 4096: 17.0 us, 20.3 with 76 pairs for 16 tiles;
  // 256: 21.0, 23.8; 200 tokens 14336 -> 4096, 56 steps for 48: 42.2, 42.5).
  if (w.shared && tiles < pairs) {
    const int64_t each = pairs / tiles;
    if ((w.ksteps + each - 1) / each <= (all + pairs - 1) / pairs + 2 + w.nt / 32)
      w.pairs = (int)std::min(all, tiles * each);
  }
  // 512 columns: with 64 tokens two sums leave room for all operands, and with
  // more a wait at the end of a segment costs less than an operand's.
  w.bufs = w.nt <= 64 ? 2 : 1;
  w.ops = std::min(kI8MostOps, (512 - (1 + w.bufs) * w.nt) / kI8A);
  w.raws = std::min(kI8MostRaw, (kI8SmemMost - w.ops * w.op_bytes()) / kI8Raw);
  return w;
}
inline int64_t i8_slices(const I8Work& w) { return (int64_t)w.tiles_m * w.tiles_n * 16; }

// early: the weights are not written by the kernel before, so this one may start during it.
template <class T>
cudaError_t int8_pair_launch(const int8_t* V, int64_t ldv, const void* codes, int64_t ldc, int64_t K, const I8Work& w,
                             const I8Out<T>& out, bool early, int32_t* status, cudaStream_t stream) {
  CUtensorMap mw, mx;
  cudaError_t e = make_tensor_map(&mw, TileMap{V, CU_TENSOR_MAP_DATA_TYPE_UINT8, out.outputs, K, ldv, 128, kI8K, true});
  if (e == cudaSuccess)
    e = make_tensor_map(&mx, TileMap{codes, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, out.tokens, K, ldc, (uint32_t)w.nt / 2, 64, true});
  const int smem = w.ops * w.op_bytes() + w.raws * kI8Raw + 1024;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(int8_pair_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kI8SmemMost + 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)w.pairs);
  cfg.blockDim = dim3(kI8Threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = early ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, int8_pair_kernel<T>, mw, mx, w, out, status);
}

}  // namespace bakron
