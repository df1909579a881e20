// cross_entropy.cu -- softmax cross entropy of a large vocabulary without
// keeping the logits, and its gradients.
//
//     x = H W^T,  lse_t = log sum_v exp(x_tv),  loss_t = lse_t - x_t,y(t),
//     G_tv = c_t (exp(x_tv - lse_t) - [v = y(t)]),  dH = G W,  dW = G^T H
//
// for hidden states H (T x D), output embedding W (V x D) and targets y; a
// token with a negative target has loss 0 and c_t = 0.
//
// The logits come out of the tensor cores a 256 x 256 tile at a time
// (pair_gemm.cuh).  The epilogue reduces each row's 64 columns to their
// maximum and the sum of exponentials below it, and a second kernel joins a
// row's pieces: the loss alone stores 8 bytes for 64 logits.
//
// The target is left out of these sums, and its logit is summed again, in fp32:
// with r_t the log-sum of the other words and d_t = r_t - x_t,y(t),
//     loss_t = log(1 + exp(d_t)),  lse_t = x_t,y(t) + loss_t,
//     G_t,y(t) = -c_t (1 - exp(-loss_t)).
// The tensor cores round towards zero in their long sums (3e-4 of a logit of 30
// over 4096 terms).  Over the other words that is an error of their log-sum,
// which counts with their share 1 - p; as a difference between two versions of
// the target's logit it would count in full, and a loss near zero would come
// out below it.
//
// For the gradients a logit is kept, for one piece of the tokens at a time,
// as the 16-bit fixed-point number round(2048 (m - x) log2 e), m the maximum
// of its 64 columns: a relative error of exp(x) of at most 1.7e-4 (1e-4 rms,
// against 1.7e-3 rms of rounding to bf16 or 2.1e-4 to fp16), and a range of
// 2^-32 below the maximum.  (The difference is taken first and then scaled: a
// rounded m log2 e in place of m would leave its remainder, which for logits
// in the thousands is more than a step, and for a mask's value is anything.)  A pass over the piece turns it into G in place,
// and G, 16-bit, is the operand of the two other products.  This reads and
// writes 6 bytes for each logit, where computing the logits a second time
// would cost a third of the products again.  A piece's logits take at most 1
// GiB, and for the loss alone its statistics 256 MiB, or what 256 tokens take.
#include <algorithm>
#include <type_traits>

#include "bakron.h"
#include "elem.cuh"
#include "layers.h"
#include "pair_gemm.cuh"

namespace bakron {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kChunk = 64;              // columns that share a maximum
constexpr float kSteps = 2048.f;        // fixed-point steps in a factor of two
constexpr float kGScale = 32768.f;      // G is stored times this, so that fp16 keeps p down to 2^-29
constexpr int kSumTerms = 512;          // terms that the tensor cores sum at a stretch, and
constexpr int64_t kFewLogits = 8192;    // the vocabulary up to which they do: see logits_launch()
constexpr int64_t kPieceBytes = (int64_t)1 << 30;       // of kept logits
constexpr int64_t kPieceStatsBytes = (int64_t)1 << 28;  // of statistics, for the loss alone
constexpr int64_t kPieceTokens = (int64_t)1 << 20;  // keeps the number of tiles and the length of a sum bounded

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// exp(from - to), 1 where both are the same infinity.
__device__ __forceinline__ float exp_diff(float from, float to) {
  return from == to ? 1.f : exp2_approx((from - to) * kLog2e);
}

// c_t / max |c| of every token, and what the gradients are scaled by in the
// end, max |c| / kGScale.  The largest of the finite ones: another stays what
// it is and reaches its own row of G only.  One block.  (Targets that are too
// large are reported by join_kernel.)
__global__ void __launch_bounds__(1024) coefficients_kernel(const int64_t* target, int64_t T, int64_t V, const float* given,
                                                            float* coef, float* scale) {
  __shared__ int with;
  __shared__ float red[32];
  if (threadIdx.x == 0) with = 0;
  __syncthreads();
  int n = 0;
  float top[1] = {0.f};
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    const int64_t y = target[t];
    if (y >= 0 && y < V) {
      ++n;
      if (given && isfinite(given[t])) top[0] = fmaxf(fabsf(given[t]), top[0]);
    }
  }
  if (n) atomicAdd(&with, n);
  block_reduce<1>(top, red, MaxOp());
  __syncthreads();
  const float most = !given ? 1.f / (float)max(with, 1) : top[0] > 0.f ? top[0] : 1.f;
  if (threadIdx.x == 0) *scale = most / kGScale;
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    const bool has = target[t] >= 0 && target[t] < V;
    coef[t] = !has ? 0.f : given ? given[t] / most : 1.f;
  }
}

// Epilogue of the logits: rows are tokens of the piece, columns the vocabulary.
template <bool kKeep>
struct LogitsEpilogue {
  using Sum = float;
  static constexpr bool kAhead = true;
  CUtensorMap map;  // of the kept logits
  int64_t rows, V;
  const int64_t* target;
  float2* stats;  // rows x chunks, of all words but the target: maximum, sum of exp(x - maximum)
  int64_t chunks;

  // The target's column among a unit's 128 or 64, -1 without one there.
  __device__ __forceinline__ static int column(int64_t y) { return (uint64_t)y < 128u ? (int)y : -1; }
  // The target of a row, as it is: looked at, it would be waited for.
  __device__ __forceinline__ int64_t ahead(int64_t row) const {
    int64_t y = -1;
    if (row < rows) y = target[row];
    return y;
  }
  __device__ __forceinline__ void operator()(const PairUnit&, int64_t row0, int64_t col, int64_t y, const PairSums& sums,
                                             const PairBox& box) const {
    if (row0 >= rows) return;
    const int at = column(y - col);
#pragma unroll 1
    for (int c = 0; c < 128 && col + c < V; c += kChunk) {
      float v[kChunk];
      sums.load(c, *reinterpret_cast<float(*)[32]>(v));
      sums.load(c + 32, *reinterpret_cast<float(*)[32]>(v + 32));
      chunk(row0, col + c, at - c, v, box);
    }
  }
  __device__ __forceinline__ void operator()(const PairUnit&, int64_t row0, int64_t col, int64_t y, float (&v)[kChunk],
                                             const PairBox& box) const {
    if (row0 < rows && col < V) chunk(row0, col, column(y - col), v, box);
  }
  __device__ __forceinline__ void chunk(int64_t row0, int64_t col, int y, float (&v)[kChunk], const PairBox& box) const {
    // One branch for the warp: few chunks hold the target of any of its rows.
    // By a bit for each column: a comparison with the index would become an
    // indexed store, and v would live in local memory.
    const bool here = (uint32_t)y < (uint32_t)kChunk;
    if (__any_sync(0xffffffffu, here)) {
      const uint64_t bit = here ? 1ull << y : 0;
      const uint32_t lo = (uint32_t)bit, hi = (uint32_t)(bit >> 32);
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if ((i < 32 ? lo >> i : hi >> (i - 32)) & 1u) v[i] = -INFINITY;
    }
    const int left = V - col < kChunk ? (int)(V - col) : kChunk;
    if (left < kChunk) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (i >= left) v[i] = -INFINITY;
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) m = fmaxf(m, v[i]);
    // All of them -infinity: their sum is 0, and so it stays below any other maximum.
    const F2 minus_m = f2(m == -INFINITY ? 0.f : -m), log2e = f2(kLog2e);
    if constexpr (kKeep) box.open();
    F2 s = f2(0.f);
#pragma unroll
    for (int j = 0; j < kChunk; j += 8) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const F2 x = (f2(v[j + i], v[j + i + 1]) + minus_m) * log2e;  // at most 0
        if constexpr (kKeep) {
          // -kSteps x rounded to an integer in the low bits of 1.5 2^23 + it.
          // A NaN is lost here; its row's sum is NaN, which is what counts.
          constexpr float kMagic = 12582912.f;
          float a, b;
          split(fma2(x, f2(-kSteps), f2(kMagic)), a, b);
          w[i] = __float_as_uint(fminf(a, kMagic + 65535.f)), w[i + 1] = __float_as_uint(fminf(b, kMagic + 65535.f));
        }
        float a, b;
        split(x, a, b);
        s = s + f2(exp2_approx(a), exp2_approx(b));
      }
      if constexpr (kKeep)
        box.put(j / 8, __byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[4], w[5], 0x5410),
                __byte_perm(w[6], w[7], 0x5410));
    }
    if constexpr (kKeep) box.send(&map, (int)col, (int)row0);
    if (row0 + box.lane < rows) stats[(row0 + box.lane) * chunks + col / kChunk] = make_float2(m, sum(s));
  }
};

// Joins a row's chunks and its target's logit, summed in fp32 with 128 sums:
// lse and loss.  One block for each token.
template <class T>
__global__ void __launch_bounds__(128) join_kernel(const float2* stats, int64_t chunks, int64_t ld, const int64_t* target,
                                                   int64_t V, const T* H, int64_t ldh, const T* W, int64_t ldw, int64_t D,
                                                   float* lse, float* loss, int32_t* status) {
  __shared__ float red[64];
  // Launched while the logits are made: the target's logit needs only H and W.
  const int64_t y = target[blockIdx.x];
  const bool has = y >= 0 && y < V;
  float t[2] = {0.f, 0.f};
  if (has) {
    const T *h = H + (int64_t)blockIdx.x * ldh, *w = W + y * ldw;
    const int64_t whole = D / 8 * 8;
    for (int64_t d = threadIdx.x * 8; d < whole; d += 1024) {
      float a[8], b[8];
      load_vec<T, 8>(h + d, a);
      load_vec<T, 8>(w + d, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[1] = fmaf(a[i], b[i], t[1]);
    }
    if (whole + threadIdx.x < D) t[1] = fmaf(to_f32<T>(h[whole + threadIdx.x]), to_f32<T>(w[whole + threadIdx.x]), t[1]);
  }
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (y >= V && threadIdx.x == 0) atomicOr(status, BAKRON_DEV_BAD_TARGET);
  const float2* row = stats + (int64_t)blockIdx.x * ld;
  float m = -INFINITY, s = 0.f;
  for (int64_t c = threadIdx.x; c < chunks; c += 128) {
    const float2 e = row[c];
    const float to = fmaxf(m, e.x);
    s = s * exp_diff(m, to) + e.y * exp_diff(e.x, to);
    m = to;
  }
  float top = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  t[0] = s * exp_diff(m, top);
  block_reduce<2>(t, red, SumOp());
  if (threadIdx.x == 0) {
    const float sum = logf(t[0]), rest = top + sum;
    const float d = t[1] < INFINITY ? (top - t[1]) + sum : NAN;
    // Either way the larger of the two with what the smaller one adds to it.
    const float more = log1pf(expf(-fabsf(d)));
    const float both = d > 0.f ? rest + more : t[1] + more;
    lse[blockIdx.x] = !has || (rest == -INFINITY && t[1] == -INFINITY) ? rest : both;
    loss[blockIdx.x] = !has ? 0.f : d > 0.f ? d + more : more;
  }
}

// The kept logits of a piece become G, times kGScale: 8 at a time.
template <class T>
__global__ void __launch_bounds__(256) gradient_kernel(uint16_t* kept, int64_t ldk, const float2* stats, int64_t chunks,
                                                       const int64_t* target, int64_t V, const float* coef,
                                                       const float* lse, const float* loss) {
  const int64_t row = blockIdx.y;
  const int64_t col = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (col >= ldk) return;
  const float c = coef[row], nll = loss[row];
  const float l = lse[row], off = (stats[row * chunks + col / kChunk].x - l) * kLog2e;
  const int64_t y = target[row] - col;
  uint16_t* at = kept + row * ldk + col;
  const uint4 q = *reinterpret_cast<const uint4*>(at);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  float g[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = i % 2 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu;
    // 65535: too far below, or -infinity; still NaN where the row's sum is
    const float p = u == 65535u ? l - l : exp2_approx(fmaf((float)u, -1.f / kSteps, off));
    g[i] = c == 0.f ? 0.f : c * kGScale * p;
  }
  if (y >= 0 && y < 8 && c != 0.f) {  // (late, when what it depends on has come)
    const float wrong = c * kGScale * expm1f(-nll);  // p - 1
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = (1u << y) >> i & 1u ? wrong : g[i];
  }
  if (V - col < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= V - col) g[i] = 0.f;
  }
  store_vec<T, 8>(reinterpret_cast<T*>(at), g);
}

// Epilogue of the gradients' products.  `part` not null: fp32 sums of the
// unit's part of K go there (parts x rows x cols).  `acc` not null: sums of
// earlier pieces are in it, and it takes theirs and these unless this is the
// last piece.  Else the scaled sums go to `out`, by TMA where its rows start
// on 16 bytes.
template <class T>
struct GradientEpilogue {
  static constexpr bool kAhead = false;
  CUtensorMap map;
  int64_t rows, cols;
  T* out;
  bool tma;
  const float* scale;
  float* part;
  float* acc;
  bool first, last;
  __device__ __forceinline__ void operator()(const PairUnit& q, int64_t row0, int64_t col, int64_t, const PairSums& sums,
                                             const PairBox& box) const {
    if (row0 >= rows) return;
    const float sc = *scale;
    const int here = (int)(rows - row0 < 32 ? rows - row0 : 32);
#pragma unroll 1
    for (int c = 0; c < 128 && col + c < cols; c += 32) {
      float v[32];
      sums.load(c, v);
      if (tma) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack2<T>(v[2 * i] * sc, v[2 * i + 1] * sc);
        const int half = (c & 32) >> 3;
        if (half == 0) box.open();
#pragma unroll
        for (int j = 0; j < 4; ++j) box.put(half + j, w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        if (half || col + c + 32 >= cols) box.send(&map, (int)col + (c & ~32), (int)row0);
        continue;
      }
      const int64_t at = row0 * cols + col + c + box.lane;
      const bool in = col + c + box.lane < cols;
      if (part) {
        float* to = part + (int64_t)q.part * rows * cols + at;
        box.by_row(v, here, in, [&](int r, float x) { to[r * cols] = x; });
      } else if (!acc) {
        box.by_row(v, here, in, [&](int r, float x) { out[at + r * cols] = from_f32<T>(x * sc); });
      } else {
        box.by_row(v, here, in, [&](int r, float x) {
          const int64_t i = at + r * cols;
          if (!first) x += acc[i];
          if (!last) acc[i] = x;
          else out[i] = from_f32<T>(x * sc);
        });
      }
    }
  }
};

// Adds up the parts of a product in their order.
template <class T>
__global__ void __launch_bounds__(256) join_parts_kernel(const float* part, int parts, int64_t n, const float* scale, T* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float s = 0.f;
  for (int k = 0; k < parts; ++k) s += part[(int64_t)k * n + i];
  out[i] = from_f32<T>(s * *scale);
}

// Rows that do not start on 16 bytes, copied to rows that do.
__global__ void __launch_bounds__(256) align_rows_kernel(const uint16_t* x, int64_t ldx, int64_t cols, uint16_t* y, int64_t ldy) {
  const int64_t row = blockIdx.y;
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c < cols) y[row * ldy + c] = x[row * ldx + c];
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }
int64_t up8(int64_t x) { return (x + 7) / 8 * 8; }
int64_t up64(int64_t x) { return (x + 63) / 64 * 64; }
int64_t tiles(int64_t x) { return (x + kPairTile - 1) / kPairTile; }

// Tokens of a piece: all, or as many whole tiles as the limits allow.
int64_t piece_tokens(int64_t T, int64_t V, bool grad) {
  const int64_t token = grad ? 2 * up64(V) : tiles(V) * 4 * 8, most = grad ? kPieceBytes : kPieceStatsBytes;
  return std::min({T, std::max<int64_t>(1, most / token / kPairTile) * kPairTile, kPieceTokens});
}

// Parts of K for dH: few tiles over a long K leave pairs of SMs idle, or a
// last wave nearly empty, so K is cut where the parts' waves are shorter by
// more than what writing and adding up the parts costs.  In steps of K of one
// pair of SMs (256 x 256 x 64, 0.27 us): a tile's epilogue about 8, a tile's
// part written and read again in fp32 0.3.
int dh_parts(int64_t T, int64_t D, int64_t V, int pairs) {
  const int64_t t = tiles(T) * tiles(D), steps = (V + kPairK - 1) / kPairK;
  int best = 1;
  double cost = (double)((t + pairs - 1) / pairs * (steps + 8));
  for (int p = 2; p <= 16 && p <= steps; ++p) {
    const double c = (double)((t * p + pairs - 1) / pairs * ((steps + p - 1) / p + 8)) + 0.3 * (double)(t * p);
    if (c < cost) best = p, cost = c;
  }
  return best;
}

struct Layout {
  size_t coef, scale, stats, kept, part, acc, h, w, bytes;
};
constexpr int kPlanPairs = 76;  // pairs of SMs that parts of K are planned for: a whole GB300
Layout layout(int64_t T, int64_t D, int64_t V, bool grad, bool copies) {
  const int64_t n = piece_tokens(T, V, grad), chunks = tiles(V) * 4;
  Layout l = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up(bytes);
    return here;
  };
  l.stats = take(n * chunks * 8);
  if (grad) {
    l.coef = take(T * 4);
    l.scale = take(4);
    l.kept = take(n * up64(V) * 2);
    const int p = dh_parts(n, D, V, kPlanPairs), p2 = T % n ? dh_parts(T % n, D, V, kPlanPairs) : 1;
    l.part = take(std::max(p > 1 ? (size_t)p * n * D * 4 : 0, p2 > 1 ? (size_t)p2 * (T % n) * D * 4 : 0));
    l.acc = take(n < T ? V * D * 4 : 0);
  }
  l.h = take(D % 64 || copies ? T * up64(D) * 2 : 0);
  if (copies) l.w = take(V * up8(D) * 2);
  l.bytes = at;
  return l;
}

bool tma_rows(const void* p, int64_t ld) { return aligned_to(p, 16) && ld % 8 == 0; }

// The tensor cores round towards zero as they sum, about 1e-9 of a logit for
// each of its terms.  The target's own is summed apart; what is left of 4096
// terms is an error of 4e-6 of a loss that another word makes alone, and of 1e-6
// (1000 words) to 5e-7 (131072) where the words share it; the plain product in
// fp32 is 8e-7 and 4e-7 to 8e-7 off.  Restarted every 512 terms and added up in
// fp32 the sums are good to 5e-7 and 1e-7, whatever their length and whatever
// the vocabulary.  They cost about 60% of the product, and so the limit is one
// of price: 1024 tokens 25 -> 38 us at 1000 words, 28 -> 41 at 4096, 46 -> 76 at
// 8192, but 147 -> 239 at 32768 and 569 -> 893 at 131072.  (Every 1024 or 2048
// terms: 28 and 17% over large vocabularies, for a quarter and a half of the
// error.)  It is one of the vocabulary and not of the work, so that a token's loss
// does not depend on how many others are in the call.
template <bool kKeep>
cudaError_t logits_launch(const PairOperand& h, const PairOperand& w, int64_t D, bool bf16, const PairWork& work,
                          const LogitsEpilogue<kKeep>& epi, int32_t* status, cudaStream_t stream, int first_status) {
  return D > kSumTerms && epi.V <= kFewLogits
             ? pair_gemm_launch<false, false, 4, kSumTerms / kPairK>(h, w, D, bf16, work, epi, status, stream, first_status)
             : pair_gemm_launch<false, false, 2, 0>(h, w, D, bf16, work, epi, status, stream, first_status);
}

template <class T>
cudaError_t run(const CrossEntropy& p, char* ws, int32_t* status, cudaStream_t stream) {
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const bool grad = p.dH != nullptr;
  const bool copies = !tma_rows(p.H, p.ldh) || !tma_rows(p.W, p.ldw);
  const Layout l = layout(p.T, p.D, p.V, grad, copies);
  const int64_t n = piece_tokens(p.T, p.V, grad), chunks = tiles(p.V) * 4, ldk = up64(p.V);
  float* coef = reinterpret_cast<float*>(ws + l.coef);
  float* scale = reinterpret_cast<float*>(ws + l.scale);
  float2* stats = reinterpret_cast<float2*>(ws + l.stats);
  uint16_t* kept = reinterpret_cast<uint16_t*>(ws + l.kept);
  const T *H = static_cast<const T*>(p.H), *W = static_cast<const T*>(p.W);
  int64_t ldh = p.ldh, ldw = p.ldw;
  auto copy = [&](const T*& x, int64_t& ld, int64_t rows, size_t to, int64_t ldt) {
    uint16_t* y = reinterpret_cast<uint16_t*>(ws + to);
    for (int64_t r = 0; r < rows; r += 65535)
      align_rows_kernel<<<dim3((unsigned)((p.D + 255) / 256), (unsigned)std::min<int64_t>(65535, rows - r)), 256, 0, stream>>>(
          reinterpret_cast<const uint16_t*>(x) + r * ld, ld, p.D, y + r * ldt, ldt);
    x = reinterpret_cast<const T*>(y), ld = ldt;
  };
  // Rows of 16-bit values that do not start on 128 bytes make TMA fetch more
  // lines (1021 x 1000 times 1000 x 50021: 88 us, from 60 with rows of 1024).
  // H is small and read by two products, so it is copied then; W only where
  // TMA cannot read it at all.
  if (copies || (p.D % 64 && !(aligned_to(H, 128) && ldh % 64 == 0))) copy(H, ldh, p.T, l.h, up64(p.D));
  if (!tma_rows(W, ldw)) copy(W, ldw, p.V, l.w, up8(p.D));
  if (grad) coefficients_kernel<<<1, 1024, 0, stream>>>(p.target, p.T, p.V, p.coef, coef, scale);
  const bool vec = grad && p.D % 8 == 0 && aligned_to(p.dH, 16) && aligned_to(p.dW, 16);
  auto out_map = [&](CUtensorMap* map, T* out, int64_t rows) {
    return make_tensor_map(map, TileMap{out, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rows,
                                        p.D, p.D, 32, 64, true});
  };
  const int dsteps = (int)((p.D + kPairK - 1) / kPairK), vsteps = (int)((p.V + kPairK - 1) / kPairK);
  for (int64_t t = 0; t < p.T; t += n) {
    const int64_t m = std::min(n, p.T - t);
    const T* h = H + t * ldh;
    const int64_t* target = p.target + t;
    const PairWork logits{(int)tiles(m), (int)tiles(p.V), 16, dsteps, 1};
    const PairOperand ph{h, m, ldh}, pw{W, p.V, ldw};
    cudaError_t e;
    if (grad) {
      LogitsEpilogue<true> epi{{}, m, p.V, target, stats, chunks};
      e = make_tensor_map(&epi.map, TileMap{kept, CU_TENSOR_MAP_DATA_TYPE_UINT16, m, ldk, ldk, 32, 64, true});
      if (e != cudaSuccess) return e;
      e = logits_launch(ph, pw, p.D, bf16, logits, epi, status, stream, t == 0 ? 0 : -1);
    } else {
      const LogitsEpilogue<false> epi{{}, m, p.V, target, stats, chunks};
      e = logits_launch(ph, pw, p.D, bf16, logits, epi, status, stream, t == 0 ? 0 : -1);
    }
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)m);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = early;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, join_kernel<T>, (const float2*)stats, (p.V + kChunk - 1) / kChunk, chunks, target, p.V, h, ldh,
                           W, ldw, p.D, p.lse + t, p.loss + t, status);
    if (e != cudaSuccess) return e;
    if (!grad) continue;
    for (int64_t r = 0; r < m; r += 65535)
      gradient_kernel<T><<<dim3((unsigned)((ldk / 8 + 255) / 256), (unsigned)std::min<int64_t>(65535, m - r)), 256, 0, stream>>>(
          kept + r * ldk, ldk, stats + r * chunks, chunks, target + r, p.V, coef + t + r, p.lse + t + r,
          p.loss + t + r);
    const PairOperand pg{kept, m, ldk}, pgt{kept, p.V, ldk}, pwt{W, p.D, ldw}, pht{h, p.D, ldh};
    T* dH = static_cast<T*>(p.dH) + t * p.D;
    const int parts = dh_parts(m, p.D, p.V, kPlanPairs);
    float* part = parts > 1 ? reinterpret_cast<float*>(ws + l.part) : nullptr;
    GradientEpilogue<T> eh{{}, m, p.D, dH, vec && !part, scale, part, nullptr, true, true};
    if (eh.tma && (e = out_map(&eh.map, dH, m)) != cudaSuccess) return e;
    e = pair_gemm_launch<false, true, 2, 0>(pg, pwt, p.V, bf16, PairWork{(int)tiles(m), (int)tiles(p.D), 16, vsteps, parts},
                                            eh, status, stream);
    if (e != cudaSuccess) return e;
    if (part)
      join_parts_kernel<T><<<(unsigned)((m * p.D + 255) / 256), 256, 0, stream>>>(part, parts, m * p.D, scale, dH);
    float* acc = n < p.T ? reinterpret_cast<float*>(ws + l.acc) : nullptr;
    GradientEpilogue<T> ew{{}, p.V, p.D, static_cast<T*>(p.dW), vec && !acc, scale, nullptr, acc, t == 0, t + m == p.T};
    if (ew.tma && (e = out_map(&ew.map, ew.out, p.V)) != cudaSuccess) return e;
    e = pair_gemm_launch<true, true, 2, 0>(
        pgt, pht, m, bf16, PairWork{(int)tiles(p.V), (int)tiles(p.D), 16, (int)((m + kPairK - 1) / kPairK), 1}, ew, status,
        stream);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace

size_t cross_entropy_workspace_bytes(int64_t T, int64_t D, int64_t V, bool grad, bool copies) {
  return layout(T, D, V, grad, copies).bytes;
}
bool cross_entropy_needs_copies(const CrossEntropy& p) { return !tma_rows(p.H, p.ldh) || !tma_rows(p.W, p.ldw); }

cudaError_t cross_entropy_launch(const CrossEntropy& p, void* ws, int32_t* status_dev, cudaStream_t stream) {
  char* at = static_cast<char*>(ws);
  return p.dtype == kF16 ? run<__half>(p, at, status_dev, stream) : run<__nv_bfloat16>(p, at, status_dev, stream);
}

}  // namespace bakron
