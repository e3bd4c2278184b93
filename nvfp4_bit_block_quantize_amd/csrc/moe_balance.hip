// moe_balance.hip -- the balance loss of a routing, the counts it needs, and its gradient with respect to the logits.
//
// Sixteen lanes (one DPP row) own a token, each EPL of its experts: a token's maximum and sum are
// four DPP steps each, and a wave takes four tokens at once.  A lane adds its experts' probabilities over the
// workgroup's tokens in registers; rows, then waves, then workgroups meet in one fixed order.  Counts are integers
// (LDS atomics, whose order does not show).  A second kernel, a workgroup a sequence, adds the workgroups' parts and
// forms the sequence's loss; the last of them to finish, found with an integer counter that the first kernel clears,
// adds the sequences' losses in order.
//
// Gradient.  With counts n and c = coef dloss E / (S k N^2), N the sequence's tokens:
//   softmax  dl_e = c p_e (n_e - sum_j p_j n_j)
//   sigmoid  dl_e = c p_e (1 - s_e) (n_e - sum_j p_j n_j),  p = s / (sum s + 1e-20)
// Counts enter as differences (exact integers) from a reference count.  Where one expert has more than half of the score it
// is that expert's: with nearly all of the score its small gradient comes from the others' terms, and nothing cancels.  Else
// it is the integer next to sum_j p_j n_j: what the differences' own sum leaves is then of the size of the counts' spread.
// (From the likeliest expert's count everywhere, one token of 401 experts of equal scores had gradients off by 1.1e-5 of
// themselves, 1 less 400/401; now 3e-8.)
//
// What bounds them: 16384 x 256 in four sequences, sigmoid, fp32: forward 7.2 to 8.9 us (17 MB: 2.7 us at the 6.2 TB/s of a large
// elementwise pass) + the sums 4.6 to 5.8, gradient added to another 12.5 to 13.2 us (50 MB: 8.1).  The forward kernel issues
// about 350 vector instructions a lane, two of them a quarter as fast, of a launch in which every wave takes one group of
// tokens; the sums are a launch and two dependent loads.  64 tokens of 64 experts: one launch of 2.7 to 3.0 us.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "nvfp4_internal.h"
#include "vec_io.hpp"

namespace nvfp4 {
namespace {

// Threads of a workgroup, and its tokens at once: the forward kernel leaves few partial sums, the backward one none.
constexpr int kSumsThreads = 1024, kSumsRows = kSumsThreads / 16, kThreads = 256, kRows = kThreads / 16;
constexpr int kMaxExperts = 512;
constexpr float kNegInf = -__builtin_huge_valf(), kMaxLogit = 3.402823466e38f;
constexpr float kTiny = 1e-20f;  // added to a sum of sigmoid scores
constexpr float kMaxCount = 2147483520.0f;  // the largest float below 2^31

// Over the 16 lanes of a row, in every lane of it.
__device__ __forceinline__ float row_sum(float v) {
  v += dpp_move<0xB1>(v);
  v += dpp_move<0x4E>(v);
  v += dpp_move<0x141>(v);
  v += dpp_move<0x140>(v);
  return v;
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp_move<0xB1>(v));
  v = fmaxf(v, dpp_move<0x4E>(v));
  v = fmaxf(v, dpp_move<0x141>(v));
  v = fmaxf(v, dpp_move<0x140>(v));
  return v;
}
template <int CTRL>
__device__ __forceinline__ int dpp_int(int v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ int row_max(int v) {
  v = max(v, dpp_int<0xB1>(v));
  v = max(v, dpp_int<0x4E>(v));
  v = max(v, dpp_int<0x141>(v));
  v = max(v, dpp_int<0x140>(v));
  return v;
}

// A lane's EPL experts of a row of E <= 16 EPL: pieces of kPiece side by side, and the row's lanes side by side in each.
template <int EPL, bool BF16>
struct Place {
  static constexpr int kPiece = EPL < (BF16 ? 8 : 4) ? EPL : (BF16 ? 8 : 4);  // elements; 16 bytes where there are enough
  static constexpr int kPieces = EPL / kPiece;
  static constexpr bool kWide = kPiece * (BF16 ? 2 : 4) == 16;
  // Expert of the lane's value i.
  static __device__ __forceinline__ int of(int i, int l16) { return (i / kPiece * 16 + l16) * kPiece + i % kPiece; }
};

template <bool BF16>
__device__ __forceinline__ float load_one(const uint8_t *row, int e) {
  return BF16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[e]) << 16)
              : reinterpret_cast<const float *>(row)[e];
}
template <bool BF16>
__device__ __forceinline__ void store_one(uint8_t *row, int e, float v) {
  if constexpr (BF16)
    reinterpret_cast<uint16_t *>(row)[e] = static_cast<uint16_t>(pack_bf16(v, 0.0f));
  else
    reinterpret_cast<float *>(row)[e] = v;
}

// The lane's values of a row: `load` asks for its pieces, and `values` gives them, `fill` beyond E (two steps, so that all of a
// token's loads are under way before the first is waited for).  Pieces may lie at any element (the loads are the same); a row's
// last one, if E ends within it, is read element by element: the others' number says in which of the lanes' pieces it is.  (Both
// directions of 12010 x 317 bf16 and 14368 x 511 fp32 take 29 and 41 us so, 44 and 54 element by element; a path of its own for
// rows of whole pieces would save these 2%.)
template <int EPL, bool BF16>
struct Row {
  using P = Place<EPL, BF16>;
  any_u32x4 w[P::kPieces];
  __device__ __forceinline__ void load(const uint8_t *row, int l16, int E) {
    if constexpr (P::kWide) {
#pragma unroll
      for (int m = 0; m < P::kPieces; ++m) {
        const int e0 = P::of(m * P::kPiece, l16);
        w[m] = (any_u32x4){0, 0, 0, 0};
        if (e0 + P::kPiece <= E) w[m] = *reinterpret_cast<const any_u32x4 *>(row + e0 * (BF16 ? 2 : 4));
      }
    }
  }
  __device__ __forceinline__ void values(const uint8_t *row, int l16, int E, float fill, float (&l)[EPL]) const {
    if constexpr (P::kWide) {
#pragma unroll
      for (int m = 0; m < P::kPieces; ++m) {
        const bool real = P::of(m * P::kPiece, l16) + P::kPiece <= E;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (BF16) {
            l[8 * m + 2 * q] = real ? __uint_as_float(w[m][q] << 16) : fill;
            l[8 * m + 2 * q + 1] = real ? __uint_as_float(w[m][q] & 0xFFFF0000u) : fill;
          } else {
            l[4 * m + q] = real ? __uint_as_float(w[m][q]) : fill;
          }
        }
      }
      if (E % P::kPiece == 0) return;
#pragma unroll
      for (int m = 0; m < P::kPieces; ++m) {
        const int e0 = P::of(m * P::kPiece, l16);
        if (E / P::kPiece / 16 != m || e0 >= E || e0 + P::kPiece <= E) continue;
#pragma unroll
        for (int i = 0; i < P::kPiece - 1; ++i)
          if (e0 + i < E) l[P::kPiece * m + i] = load_one<BF16>(row, e0 + i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = P::of(i, l16);
        l[i] = e < E ? load_one<BF16>(row, e) : fill;
      }
    }
  }
};
template <int EPL, bool BF16>
__device__ __forceinline__ void store_row(uint8_t *row, int l16, int E, const float (&d)[EPL]) {
  using P = Place<EPL, BF16>;
  if constexpr (P::kWide) {
#pragma unroll
    for (int m = 0; m < P::kPieces; ++m) {
      const int e0 = P::of(m * P::kPiece, l16);
      any_u32x4 w;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (BF16)
          w[q] = pack_bf16(d[8 * m + 2 * q], d[8 * m + 2 * q + 1]);
        else
          w[q] = __float_as_uint(d[4 * m + q]);
      }
      if (e0 + P::kPiece <= E) *reinterpret_cast<any_u32x4 *>(row + e0 * (BF16 ? 2 : 4)) = w;
    }
    if (E % P::kPiece == 0) return;
#pragma unroll
    for (int m = 0; m < P::kPieces; ++m) {
      const int e0 = P::of(m * P::kPiece, l16);
      if (E / P::kPiece / 16 != m || e0 >= E || e0 + P::kPiece <= E) continue;
#pragma unroll
      for (int i = 0; i < P::kPiece - 1; ++i)
        if (e0 + i < E) store_one<BF16>(row, e0 + i, d[P::kPiece * m + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = P::of(i, l16);
      if (e < E) store_one<BF16>(row, e, d[i]);
    }
  }
}
// The lane's counts of a row of E, four at a time where four lie together in the lane.
template <int EPL, bool BF16>
__device__ __forceinline__ void load_counts(const int32_t *row, int l16, int E, int (&n)[EPL]) {
  using P = Place<EPL, BF16>;
  if constexpr (P::kPiece >= 4) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      const int e = P::of(i, l16);
      any_u32x4 v = {0, 0, 0, 0};
      if (e + 4 <= E) {
        v = *reinterpret_cast<const any_u32x4 *>(row + e);
      } else {
#pragma unroll
        for (int q = 0; q < 3; ++q)
          if (e + q < E) v[q] = row[e + q];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) n[i + q] = static_cast<int>(v[q]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = P::of(i, l16);
      n[i] = e < E ? row[e] : 0;
    }
  }
}

// exp(x) for x <= 0, off by at most 4 x 2^-24 of itself: what the rounding of x / ln 2 leaves goes in by its first order.  (The
// general function costs twice the instructions.)  -inf and NaN count as -200, whose exponential is zero in 32 bits.
__device__ __forceinline__ float exp_of(float x) {
  constexpr float kInvLn2 = 1.44269502e+00f, kLn2 = 6.93147182e-01f, kLn2Low = -1.90465421e-09f;
  x = fmaxf(x, -200.0f);
  const float t = x * kInvLn2;
  const float left = fmaf(-t, kLn2Low, fmaf(-t, kLn2, x));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, left, e);
}

// Scores of a token from its logits (closed experts: -inf or NaN; others capped at FLT_MAX), before their division by their
// sum: p, and what divides them, `inv` (0 for a token without an open expert, or whose sum is zero).  l is left as the
// logits in this form; `spare` is 1 - sum of the probabilities (0 for a softmax); slope (sigmoid): 1 - s.  Returns half of
// the sum.  A closed expert's score comes out as zero by itself.
// A sigmoid's reciprocal is the hardware's, one unit off, and a Newton step: 0.1 us of the two kernels' 20 at 16384 x 256, where
// the general division costs 1.7 for the same errors.  (Without it the gradient is off by 1.3e-7 of its norm and not 0.9e-7,
// one token of 401 experts.)
template <int EPL, bool SIGMOID, bool SLOPE>
__device__ __forceinline__ float row_scores(float (&l)[EPL], float (&p)[EPL], float (&slope)[EPL], float &inv, float &spare) {
  float top = kNegInf, sum = 0.0f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    l[j] = fminf(fmaxf(l[j], kNegInf), kMaxLogit);  // (the larger of NaN and -inf is -inf)
    if (!SIGMOID) top = fmaxf(top, l[j]);
  }
  if (!SIGMOID) top = row_max(top);
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    if constexpr (SIGMOID) {
      const float e = exp_of(-fabsf(l[j])), d = 1.0f + e, near = __builtin_amdgcn_rcpf(d);
      const float r = fmaf(fmaf(-d, near, 1.0f), near, near), er = e * r;
      p[j] = l[j] > 0.0f ? r : er;
      if (SLOPE) slope[j] = l[j] > 0.0f ? er : r;
    } else {
      p[j] = exp_of(l[j] - top);
    }
    sum += p[j];
  }
  sum = row_sum(sum);
  inv = SIGMOID ? 1.0f / (sum + kTiny) : (sum > 0.0f ? 1.0f / sum : 0.0f);
  spare = SIGMOID ? kTiny * inv : 0.0f;
  return 0.5f * sum;
}

struct BalanceArgs {
  const uint8_t *logits;
  int64_t row_bytes;
  int64_t seq;  // tokens of a sequence
  int E, k, sequences, blocks;  // blocks: workgroups of a sequence
  const int32_t *ids;
  float scale;  // coef / sequences
  float *part_probs;     // [sequences][blocks][E]
  int32_t *part_counts;  // the like
  int32_t *part_tokens;  // [sequences][blocks]
  float *part_loss;      // [sequences][workgroups of a sequence's sums]
  uint32_t *done;
  float *loss, *probs;
  int32_t *counts, *tokens;
};

// Whether a token's row of lanes sees an expert among its ids; counts them in `hist`.
__device__ __forceinline__ bool row_ids(const int32_t *ids, int64_t t, int k, int E, int l16, bool exists, int32_t *hist) {
  int any = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = 16 * h + l16;
    if (exists && j < k) {
      const int e = ids[t * k + j];
      if (e >= 0 && e < E) {
        any = 1;
        if (hist) atomicAdd(&hist[e], 1);
      }
    }
  }
  return row_max(any) != 0;
}

// What a sequence's sums give: mean probabilities, counts, tokens; the loss of it (before scale).  `threads` threads.
__device__ __forceinline__ float seq_term(int count, float prob_sum, int tokens, int E, int k, float &prob) {
  if (tokens == 0) {
    prob = 0.0f;
    return 0.0f;
  }
  const float n = static_cast<float>(tokens);
  prob = prob_sum / n;
  return static_cast<float>(count) * (static_cast<float>(E) / static_cast<float>(k)) / n * prob;
}

// ONE: a single workgroup has all tokens and writes the results itself.
template <int EPL, bool BF16, bool SIGMOID, bool ONE>
__global__ __launch_bounds__(kSumsThreads) void balance_kernel(BalanceArgs p) {
  constexpr int P = 16 * EPL, kWaves = kSumsThreads / 64;
  __shared__ int32_t hist[P];
  __shared__ float sums[kWaves][P];
  __shared__ int32_t live_count[kWaves];
  __shared__ float loss_part[kWaves];
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const int l16 = lane & 15;
  const int64_t s = blockIdx.y, first = s * p.seq;
  for (int e = threadIdx.x; e < P; e += kSumsThreads) hist[e] = 0;
  if (!ONE && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.done = 0;
  __syncthreads();
  float acc[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) acc[j] = 0.0f;
  int live = 0;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kSumsRows; t0 < p.seq; t0 += static_cast<int64_t>(p.blocks) * kSumsRows) {
    const int64_t i = t0 + (threadIdx.x >> 4);
    const bool exists = i < p.seq;
    const int64_t t = first + (exists ? i : p.seq - 1);
    float l[EPL], q[EPL], none[EPL], inv, spare;
    const uint8_t *const row = p.logits + t * p.row_bytes;
    Row<EPL, BF16> raw;
    raw.load(row, l16, p.E);
    const bool on = row_ids(p.ids, t, p.k, p.E, l16, exists, hist);
    raw.values(row, l16, p.E, kNegInf, l);
    row_scores<EPL, SIGMOID, false>(l, q, none, inv, spare);
    if (!on) inv = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) acc[j] = fmaf(q[j], inv, acc[j]);
    live += on;
  }
  // The wave's four rows, then the waves.  A swap of two registers' halves and an add leave one's sum in either half.
  if constexpr (EPL >= 4) {
#pragma unroll
    for (int j = 0; j < EPL / 2; ++j) {
      const auto v = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[j]), __float_as_uint(acc[j + EPL / 2]), false, false);
      acc[j] = __uint_as_float(v[0]) + __uint_as_float(v[1]);
    }
#pragma unroll
    for (int j = 0; j < EPL / 4; ++j) {
      const auto v = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[j]), __float_as_uint(acc[j + EPL / 4]), false, false);
      const float sum = __uint_as_float(v[0]) + __uint_as_float(v[1]);
      const int mine = j + (lane & 32u ? EPL / 2 : 0) + (lane & 16u ? EPL / 4 : 0);
      sums[wave][Place<EPL, BF16>::of(mine, l16)] = sum;
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      acc[j] += __shfl_xor(acc[j], 16);
      acc[j] += __shfl_xor(acc[j], 32);
      if (lane < 16) sums[wave][Place<EPL, BF16>::of(j, l16)] = acc[j];
    }
  }
  live += __shfl_xor(live, 16);
  live += __shfl_xor(live, 32);
  if (lane == 0) live_count[wave] = live;
  __syncthreads();
  int tokens = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) tokens += live_count[w];
  const int64_t block = s * p.blocks + blockIdx.x;
  float loss = 0.0f;
  if (static_cast<int>(threadIdx.x) < p.E) {
    const int e = threadIdx.x;
    float sum = sums[0][e];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += sums[w][e];
    if constexpr (ONE) {
      float prob;
      loss = seq_term(hist[e], sum, tokens, p.E, p.k, prob);
      p.probs[e] = prob;
      p.counts[e] = hist[e];
    } else {
      p.part_probs[block * p.E + e] = sum;
      p.part_counts[block * p.E + e] = hist[e];
    }
  }
  if constexpr (ONE) {
    loss = wave_sum(loss);
    if (lane == 0) loss_part[wave] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
      loss = 0.0f;
      for (int w = 0; w < kWaves; ++w) loss += loss_part[w];
      *p.loss = loss * p.scale;
      *p.tokens = tokens;
    }
  } else if (threadIdx.x == 0) {
    p.part_tokens[block] = tokens;
  }
}

// A workgroup has kSumColumns experts of a sequence, and every (1024 / kSumColumns)-th workgroup's part a thread.  The last
// to finish adds the losses of all.
constexpr int kSumThreads = 1024, kSumColumns = 32;
__global__ __launch_bounds__(kSumThreads) void balance_sum_kernel(BalanceArgs p) {
  constexpr int kStep = kSumThreads / kSumColumns;
  __shared__ float sums[kSumThreads];
  __shared__ int32_t counts[kSumThreads];
  __shared__ int32_t token_part[16];
  __shared__ float loss_part[16];
  __shared__ uint32_t arrived;
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const int64_t s = blockIdx.y;
  const int e = blockIdx.x * kSumColumns + threadIdx.x % kSumColumns;
  float sum = 0.0f;
  int count = 0, tokens = 0;
  if (e < p.E)
#pragma unroll 4
    for (int b = threadIdx.x / kSumColumns; b < p.blocks; b += kStep) {
      sum += p.part_probs[(s * p.blocks + b) * p.E + e];
      count += p.part_counts[(s * p.blocks + b) * p.E + e];
    }
  for (int b = threadIdx.x; b < p.blocks; b += kSumThreads) tokens += p.part_tokens[s * p.blocks + b];
#pragma unroll
  for (int d = 1; d < 64; d *= 2) tokens += __shfl_xor(tokens, d);
  if (lane == 0) token_part[wave] = tokens;
  sums[threadIdx.x] = sum;
  counts[threadIdx.x] = count;
  __syncthreads();
  tokens = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) tokens += token_part[w];
  if (wave == 0) {
    float loss = 0.0f;
    if (lane < kSumColumns && e < p.E) {
#pragma unroll 8
      for (int g = 1; g < kStep; ++g) {
        sum += sums[g * kSumColumns + lane];
        count += counts[g * kSumColumns + lane];
      }
      float prob;
      loss = seq_term(count, sum, tokens, p.E, p.k, prob);
      p.probs[s * p.E + e] = prob;
      p.counts[s * p.E + e] = count;
    }
    loss = wave_sum(loss);
    if (lane == 0) {
      if (blockIdx.x == 0) p.tokens[s] = tokens;
      __hip_atomic_store(&p.part_loss[s * gridDim.x + blockIdx.x], loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      arrived = __hip_atomic_fetch_add(p.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  __syncthreads();
  const uint32_t all = gridDim.x * gridDim.y;
  if (arrived != all - 1) return;
  float loss = 0.0f;
  for (uint32_t i = threadIdx.x; i < all; i += kSumThreads)
    loss += __hip_atomic_load(&p.part_loss[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  loss = wave_sum(loss);
  if (lane == 0) loss_part[wave] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    loss = 0.0f;
    for (int w = 0; w < 16; ++w) loss += loss_part[w];
    *p.loss = loss * p.scale;
  }
}

struct BalanceBwdArgs {
  const uint8_t *logits, *din;
  uint8_t *out;
  int64_t row_bytes, din_row_bytes, out_row_bytes;
  int64_t seq;
  int E, k, blocks;
  const int32_t *ids, *counts, *tokens;
  const float *dloss;  // NULL: 1
  float factor;        // coef E / (sequences k)
};

template <int EPL, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void balance_backward_kernel(BalanceBwdArgs p) {
  const int l16 = threadIdx.x & 15;
  const int64_t s = blockIdx.y, first = s * p.seq;
  int n[EPL];
  load_counts<EPL, BF16>(p.counts + s * p.E, l16, p.E, n);
  const int tokens = p.tokens[s];
  // (in 64 bits: N^2 may pass what 32 hold well)
  double c = tokens > 0 ? static_cast<double>(p.factor) / tokens / tokens : 0.0;
  if (p.dloss) c *= static_cast<double>(*p.dloss);
  const float cf = static_cast<float>(c);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows; t0 < p.seq; t0 += static_cast<int64_t>(p.blocks) * kRows) {
    const int64_t i = t0 + (threadIdx.x >> 4);
    const bool exists = i < p.seq;
    const int64_t t = first + (exists ? i : p.seq - 1);
    float l[EPL], q[EPL], slope[EPL], d[EPL], inv, spare;
    const uint8_t *const row = p.logits + t * p.row_bytes, *const given = p.din + t * p.din_row_bytes;
    Row<EPL, BF16> raw, raw_d;
    raw.load(row, l16, p.E);
    if (p.din) raw_d.load(given, l16, p.E);
    const bool on = row_ids(p.ids, t, p.k, p.E, l16, exists, nullptr);
    raw.values(row, l16, p.E, kNegInf, l);
    const float half = row_scores<EPL, SIGMOID, true>(l, q, slope, inv, spare);
    int ref = -1;
    float mean = 0.0f;  // of the counts
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      ref = max(ref, q[j] > half ? n[j] : -1);
      mean = fmaf(q[j], static_cast<float>(n[j]), mean);
    }
    ref = row_max(ref);
    mean = row_sum(mean) * inv;
    if (ref < 0) ref = static_cast<int>(fminf(rintf(mean), kMaxCount));
    mean = 0.0f;  // of the counts, less ref
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      l[j] = static_cast<float>(n[j] - ref);
      mean = fmaf(q[j], l[j], mean);
    }
    mean = row_sum(mean) * inv;
    if (SIGMOID) mean = fmaf(-spare, static_cast<float>(ref), mean);
    const float factor = on ? cf * inv : 0.0f;
    if (p.din) {
      raw_d.values(given, l16, p.E, 0.0f, d);
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) d[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const float g = factor * q[j] * (l[j] - mean);
      // (what has no score keeps dlogits_in also where dloss is infinite or NaN)
      if (on && q[j] > 0.0f) d[j] += SIGMOID ? g * slope[j] : g;
    }
    if (exists) store_row<EPL, BF16>(p.out + t * p.out_row_bytes, l16, p.E, d);
  }
}

int experts_per_lane(int64_t E) {
  int epl = 1;
  while (16 * epl < E) epl *= 2;
  return epl;
}

// Tokens up to which one workgroup does all of it.
constexpr int64_t kOneBlockTokens = 64;
// Workgroups of a launch along the tokens, over all sequences.
constexpr int64_t kForwardBlocks = 256, kBackwardBlocks = 2048;
int64_t blocks_a_sequence(int64_t seq, int64_t sequences, int64_t rows, int64_t most) {
  const int64_t need = (seq + rows - 1) / rows, share = most / sequences;
  const int64_t blocks = need < share ? need : share;
  return blocks > 1 ? blocks : 1;  // (without tokens a workgroup still writes zeros)
}
template <int EPL, bool BF16, bool SIGMOID>
hipError_t run_forward(const BalanceArgs &p, bool one, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(p.blocks), static_cast<uint32_t>(p.sequences));
  if (one)
    balance_kernel<EPL, BF16, SIGMOID, true><<<grid, dim3(kSumsThreads), 0, stream>>>(p);
  else
    balance_kernel<EPL, BF16, SIGMOID, false><<<grid, dim3(kSumsThreads), 0, stream>>>(p);
  return hipGetLastError();
}
template <int EPL>
hipError_t run_forward(const BalanceArgs &p, bool one, bool bf16, bool sigmoid, hipStream_t stream) {
  if (bf16) return sigmoid ? run_forward<EPL, true, true>(p, one, stream) : run_forward<EPL, true, false>(p, one, stream);
  return sigmoid ? run_forward<EPL, false, true>(p, one, stream) : run_forward<EPL, false, false>(p, one, stream);
}
template <int EPL>
hipError_t run_backward(const BalanceBwdArgs &p, int64_t sequences, bool bf16, bool sigmoid, hipStream_t stream) {
  auto *kernel = bf16 ? (sigmoid ? balance_backward_kernel<EPL, true, true> : balance_backward_kernel<EPL, true, false>)
                      : (sigmoid ? balance_backward_kernel<EPL, false, true> : balance_backward_kernel<EPL, false, false>);
  kernel<<<dim3(static_cast<uint32_t>(p.blocks), static_cast<uint32_t>(sequences)), dim3(kThreads), 0, stream>>>(p);
  return hipGetLastError();
}

// Workgroups of a sequence's sums.
int64_t sum_groups(int64_t experts) { return (experts + kSumColumns - 1) / kSumColumns; }

bool one_block(int64_t tokens, int64_t sequences) { return sequences == 1 && tokens <= kOneBlockTokens; }

}  // namespace

size_t moe_balance_workspace_bytes(int64_t tokens, int64_t experts, int64_t sequences) {
  if (one_block(tokens, sequences)) return 0;
  const int64_t blocks = sequences * blocks_a_sequence(tokens / sequences, sequences, kSumsRows, kForwardBlocks);
  return static_cast<size_t>(blocks * (2 * experts + 1) + sequences * sum_groups(experts) + 1) * 4;
}

hipError_t launch_moe_balance(const MoeBalanceArgs &a) {
  BalanceArgs p{};
  const int es = a.dtype == 1 ? 2 : 4;
  p.logits = static_cast<const uint8_t *>(a.logits);
  p.row_bytes = a.ld * es;
  p.seq = a.tokens / a.sequences;
  p.E = static_cast<int>(a.experts);
  p.k = a.top_k;
  p.sequences = static_cast<int>(a.sequences);
  p.ids = a.ids;
  p.scale = a.coef / static_cast<float>(a.sequences);
  p.loss = a.loss;
  p.probs = a.probs;
  p.counts = a.counts;
  p.tokens = a.live;
  const bool one = one_block(a.tokens, a.sequences);
  p.blocks = one ? 1 : static_cast<int>(blocks_a_sequence(p.seq, a.sequences, kSumsRows, kForwardBlocks));
  const int64_t blocks = p.sequences * static_cast<int64_t>(p.blocks);
  if (!one) {
    p.part_probs = static_cast<float *>(a.workspace);
    p.part_counts = reinterpret_cast<int32_t *>(p.part_probs + blocks * p.E);
    p.part_tokens = p.part_counts + blocks * p.E;
    p.part_loss = reinterpret_cast<float *>(p.part_tokens + blocks);
    p.done = reinterpret_cast<uint32_t *>(p.part_loss + p.sequences * sum_groups(p.E));
  }
  const bool bf16 = a.dtype == 1;
  hipError_t e;
  switch (experts_per_lane(p.E)) {
    case 1: e = run_forward<1>(p, one, bf16, a.sigmoid, a.stream); break;
    case 2: e = run_forward<2>(p, one, bf16, a.sigmoid, a.stream); break;
    case 4: e = run_forward<4>(p, one, bf16, a.sigmoid, a.stream); break;
    case 8: e = run_forward<8>(p, one, bf16, a.sigmoid, a.stream); break;
    case 16: e = run_forward<16>(p, one, bf16, a.sigmoid, a.stream); break;
    default: e = run_forward<32>(p, one, bf16, a.sigmoid, a.stream); break;
  }
  if (e != hipSuccess || one) return e;
  const dim3 grid(static_cast<uint32_t>(sum_groups(p.E)), static_cast<uint32_t>(p.sequences));
  balance_sum_kernel<<<grid, dim3(kSumThreads), 0, a.stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_moe_balance_backward(const MoeBalanceArgs &a) {
  BalanceBwdArgs p{};
  const int es = a.dtype == 1 ? 2 : 4;
  p.logits = static_cast<const uint8_t *>(a.logits);
  p.din = static_cast<const uint8_t *>(a.dlogits_in);
  p.out = static_cast<uint8_t *>(a.dlogits);
  p.row_bytes = a.ld * es;
  p.din_row_bytes = a.ld_in * es;
  p.out_row_bytes = a.ldd * es;
  p.seq = a.tokens / a.sequences;
  p.E = static_cast<int>(a.experts);
  p.k = a.top_k;
  p.blocks = static_cast<int>(blocks_a_sequence(p.seq, a.sequences, kRows, kBackwardBlocks));
  p.ids = a.ids;
  p.counts = a.counts;
  p.tokens = a.live;
  p.dloss = a.dloss;
  p.factor = a.coef * static_cast<float>(a.experts) / (static_cast<float>(a.sequences) * static_cast<float>(a.top_k));
  const bool bf16 = a.dtype == 1;
  switch (experts_per_lane(p.E)) {
    case 1: return run_backward<1>(p, a.sequences, bf16, a.sigmoid, a.stream);
    case 2: return run_backward<2>(p, a.sequences, bf16, a.sigmoid, a.stream);
    case 4: return run_backward<4>(p, a.sequences, bf16, a.sigmoid, a.stream);
    case 8: return run_backward<8>(p, a.sequences, bf16, a.sigmoid, a.stream);
    case 16: return run_backward<16>(p, a.sequences, bf16, a.sigmoid, a.stream);
    default: return run_backward<32>(p, a.sequences, bf16, a.sigmoid, a.stream);
  }
}

}  // namespace nvfp4
