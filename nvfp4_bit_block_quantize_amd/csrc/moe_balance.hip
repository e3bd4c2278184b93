// moe_balance.hip -- the balance loss of a routing, the counts it needs, and its gradient with respect to the logits.
//
// Sixteen lanes (one DPP row) own a token, lane i the experts [i EPL, (i + 1) EPL): a token's maximum and sum are
// four DPP steps each, and a wave takes four tokens at once.  A lane adds its experts' probabilities over the
// workgroup's tokens in registers; rows, then waves, then workgroups meet in one fixed order.  Counts are integers
// (LDS atomics, whose order does not show).  A second kernel, a workgroup a sequence, adds the workgroups' parts and
// forms the sequence's loss; the last of them to finish, found with an integer counter that the first kernel clears,
// adds the sequences' losses in order.
//
// Gradient.  With counts n and c = coef dloss E / (S k N^2), N the sequence's tokens:
//   softmax  dl_e = c p_e (n_e - sum_j p_j n_j)
//   sigmoid  dl_e = c p_e (1 - s_e) (n_e - sum_j p_j n_j),  p = s / (sum s + 1e-20)
// Counts enter as differences (exact integers) from the count of the expert with the largest score: where one expert
// has nearly all of the score its small gradient comes from the others' terms, and nothing cancels.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "nvfp4_internal.h"
#include "vec_io.hpp"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256, kRows = kThreads / 16;  // tokens of a workgroup at once
constexpr int kMaxExperts = 512;
constexpr float kNegInf = -__builtin_huge_valf(), kMaxLogit = 3.402823466e38f;
constexpr float kTiny = 1e-20f;  // added to a sum of sigmoid scores

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

// A lane's EPL values of a row from element e0 on; `fill` beyond E.
template <int EPL, bool BF16>
__device__ __forceinline__ void load_row(const uint8_t *row, int e0, int E, bool vec, float fill, float (&l)[EPL]) {
  constexpr int BYTES = EPL * (BF16 ? 2 : 4);
  if constexpr (BYTES % 16 == 0) {
    if (vec && e0 + EPL <= E) {
      constexpr int V = BF16 ? 8 : 4;
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) {
        const uint4 v = *reinterpret_cast<const uint4 *>(row + e0 * (BF16 ? 2 : 4) + 16 * i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (BF16) {
            l[V * i + 2 * q] = __uint_as_float(w[q] << 16);
            l[V * i + 2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
          } else {
            l[V * i + q] = __uint_as_float(w[q]);
          }
        }
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    l[j] = fill;
    if (e0 + j < E)
      l[j] = BF16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[e0 + j]) << 16)
                  : reinterpret_cast<const float *>(row)[e0 + j];
  }
}
template <int EPL, bool BF16>
__device__ __forceinline__ void store_row(uint8_t *row, int e0, int E, bool vec, const float (&d)[EPL]) {
  constexpr int BYTES = EPL * (BF16 ? 2 : 4);
  if constexpr (BYTES % 16 == 0) {
    if (vec && e0 + EPL <= E) {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (BF16)
            w[q] = pack_bf16(d[8 * i + 2 * q], d[8 * i + 2 * q + 1]);
          else
            w[q] = __float_as_uint(d[4 * i + q]);
        }
        *reinterpret_cast<uint4 *>(row + e0 * (BF16 ? 2 : 4) + 16 * i) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j)
    if (e0 + j < E) {
      if constexpr (BF16)
        reinterpret_cast<uint16_t *>(row)[e0 + j] = static_cast<uint16_t>(pack_bf16(d[j], 0.0f));
      else
        reinterpret_cast<float *>(row)[e0 + j] = d[j];
    }
}

// Probabilities of a token from its logits (closed experts: -inf or NaN; others capped at FLT_MAX).  l is left as the
// logits in this form; `spare` is 1 - sum p (0 for a softmax).  Returns the largest logit.
template <int EPL, bool SIGMOID>
__device__ __forceinline__ float row_probs(float (&l)[EPL], float (&p)[EPL], float &spare) {
  float top = kNegInf;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    l[j] = l[j] > kNegInf ? fminf(l[j], kMaxLogit) : kNegInf;  // (NaN compares false)
    top = fmaxf(top, l[j]);
  }
  top = row_max(top);
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    if constexpr (SIGMOID) {
      const float e = expf(-fabsf(l[j]));
      p[j] = l[j] == kNegInf ? 0.0f : (l[j] > 0.0f ? 1.0f : e) / (1.0f + e);
    } else {
      p[j] = l[j] == kNegInf ? 0.0f : expf(l[j] - top);
    }
    sum += p[j];
  }
  sum = row_sum(sum);
  const float inv = SIGMOID ? 1.0f / (sum + kTiny) : (sum > 0.0f ? 1.0f / sum : 0.0f);
  spare = SIGMOID ? kTiny * inv : 0.0f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) p[j] *= inv;
  return top;
}

struct BalanceArgs {
  const uint8_t *logits;
  int64_t row_bytes;
  int64_t seq;  // tokens of a sequence
  int E, k, sequences, blocks;  // blocks: workgroups of a sequence
  bool vec;
  const int32_t *ids;
  float scale;  // coef / sequences
  float *part_probs;     // [sequences][blocks][E]
  int32_t *part_counts;  // the like
  int32_t *part_tokens;  // [sequences][blocks]
  float *part_loss;      // [sequences]
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
__global__ __launch_bounds__(kThreads) void balance_kernel(BalanceArgs p) {
  constexpr int P = 16 * EPL;
  __shared__ int32_t hist[P];
  __shared__ float sums[4][P];
  __shared__ int32_t live_count[4];
  __shared__ float loss_part[4];
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, e0 = l16 * EPL;
  const int64_t s = blockIdx.y, first = s * p.seq;
  for (int e = threadIdx.x; e < P; e += kThreads) hist[e] = 0;
  if (!ONE && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.done = 0;
  __syncthreads();
  float acc[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) acc[j] = 0.0f;
  int live = 0;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows; t0 < p.seq; t0 += static_cast<int64_t>(p.blocks) * kRows) {
    const int64_t i = t0 + (threadIdx.x >> 4);
    const bool exists = i < p.seq;
    const int64_t t = first + (exists ? i : p.seq - 1);
    float l[EPL], q[EPL], spare;
    load_row<EPL, BF16>(p.logits + t * p.row_bytes, e0, p.E, p.vec, kNegInf, l);
    const bool on = row_ids(p.ids, t, p.k, p.E, l16, exists, hist);
    row_probs<EPL, SIGMOID>(l, q, spare);
#pragma unroll
    for (int j = 0; j < EPL; ++j) acc[j] += on ? q[j] : 0.0f;
    live += on;
  }
  // the wave's four rows, then the waves
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    acc[j] += __shfl_xor(acc[j], 16);
    acc[j] += __shfl_xor(acc[j], 32);
    if (lane < 16) sums[wave][e0 + j] = acc[j];
  }
  live += __shfl_xor(live, 16);
  live += __shfl_xor(live, 32);
  if (lane == 0) live_count[wave] = live;
  __syncthreads();
  const int tokens = (live_count[0] + live_count[1]) + (live_count[2] + live_count[3]);
  const int64_t block = s * p.blocks + blockIdx.x;
  float loss = 0.0f;
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    const float sum = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
    if constexpr (ONE) {
      float prob;
      loss += seq_term(hist[e], sum, tokens, p.E, p.k, prob);
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
      *p.loss = ((loss_part[0] + loss_part[1]) + (loss_part[2] + loss_part[3])) * p.scale;
      *p.tokens = tokens;
    }
  } else if (threadIdx.x == 0) {
    p.part_tokens[block] = tokens;
  }
}

// A workgroup a sequence: 1024 / width threads an expert add the parts of every (1024 / width)-th workgroup.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void balance_sum_kernel(BalanceArgs p, int width) {
  __shared__ float sums[kSumThreads];
  __shared__ int32_t counts[kSumThreads];
  __shared__ float loss_part[16];
  __shared__ int32_t token_part[16];
  __shared__ uint32_t arrived;
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const int64_t s = blockIdx.x;
  const int e = threadIdx.x & (width - 1), step = kSumThreads / width;
  float sum = 0.0f;
  int count = 0, tokens = 0;
  if (e < p.E)
#pragma unroll 4
    for (int b = threadIdx.x / width; b < p.blocks; b += step) {
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
  float loss = 0.0f;
  if (static_cast<int>(threadIdx.x) < p.E) {
    for (int g = 1; g < step; ++g) {
      sum += sums[g * width + threadIdx.x];
      count += counts[g * width + threadIdx.x];
    }
    float prob;
    loss = seq_term(count, sum, tokens, p.E, p.k, prob);
    p.probs[s * p.E + threadIdx.x] = prob;
    p.counts[s * p.E + threadIdx.x] = count;
  }
  loss = wave_sum(loss);
  if (lane == 0) loss_part[wave] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    loss = 0.0f;
    for (int w = 0; w < 16; ++w) loss += loss_part[w];
    p.tokens[s] = tokens;
    if (p.sequences == 1) {
      *p.loss = loss * p.scale;
    } else {
      __hip_atomic_store(&p.part_loss[s], loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      arrived = __hip_atomic_fetch_add(p.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (p.sequences == 1) return;
  __syncthreads();
  if (arrived != static_cast<uint32_t>(p.sequences) - 1) return;
  // the last workgroup: every other one's loss is there
  loss = 0.0f;
  for (int64_t i = threadIdx.x; i < p.sequences; i += kSumThreads)
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
  bool vec, vec_din, vec_out;
  const int32_t *ids, *counts, *tokens;
  const float *dloss;  // NULL: 1
  float factor;        // coef E / (sequences k)
};

template <int EPL, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void balance_backward_kernel(BalanceBwdArgs p) {
  const int l16 = threadIdx.x & 15, e0 = l16 * EPL;
  const int64_t s = blockIdx.y, first = s * p.seq;
  int n[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) n[j] = e0 + j < p.E ? p.counts[s * p.E + e0 + j] : 0;
  const int tokens = p.tokens[s];
  // (in 64 bits: N^2 may pass what 32 hold well)
  double c = tokens > 0 ? static_cast<double>(p.factor) / tokens / tokens : 0.0;
  if (p.dloss) c *= static_cast<double>(*p.dloss);
  const float cf = static_cast<float>(c);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows; t0 < p.seq; t0 += static_cast<int64_t>(p.blocks) * kRows) {
    const int64_t i = t0 + (threadIdx.x >> 4);
    const bool exists = i < p.seq;
    const int64_t t = first + (exists ? i : p.seq - 1);
    float l[EPL], q[EPL], d[EPL], spare;
    load_row<EPL, BF16>(p.logits + t * p.row_bytes, e0, p.E, p.vec, kNegInf, l);
    if (p.din) {
      load_row<EPL, BF16>(p.din + t * p.din_row_bytes, e0, p.E, p.vec_din, 0.0f, d);
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) d[j] = 0.0f;
    }
    const bool on = row_ids(p.ids, t, p.k, p.E, l16, exists, nullptr);
    const float top = row_probs<EPL, SIGMOID>(l, q, spare);
    int ref = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) ref = max(ref, l[j] == top ? n[j] : 0);
    ref = row_max(ref);
    float mean = 0.0f;  // of the counts, less ref
#pragma unroll
    for (int j = 0; j < EPL; ++j) mean = fmaf(q[j], static_cast<float>(n[j] - ref), mean);
    mean = row_sum(mean);
    if (SIGMOID) mean = fmaf(-spare, static_cast<float>(ref), mean);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      float g = cf * q[j] * (static_cast<float>(n[j] - ref) - mean);
      if constexpr (SIGMOID) {
        const float e = expf(-fabsf(l[j]));
        g *= (l[j] > 0.0f ? e : 1.0f) / (1.0f + e);
      }
      if (on && l[j] != kNegInf) d[j] += g;
    }
    if (exists) store_row<EPL, BF16>(p.out + t * p.out_row_bytes, e0, p.E, p.vec_out, d);
  }
}

int experts_per_lane(int64_t E) {
  int epl = 1;
  while (16 * epl < E) epl *= 2;
  return epl;
}
bool rows_aligned16(const void *p, int64_t row_bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && row_bytes % 16 == 0;
}

// Tokens up to which one workgroup does all of it.
constexpr int64_t kOneBlockTokens = 64;
// Workgroups of a launch along the tokens, over all sequences.
constexpr int64_t kForwardBlocks = 256, kBackwardBlocks = 2048;
int64_t blocks_a_sequence(int64_t seq, int64_t sequences, int64_t most) {
  const int64_t need = (seq + kRows - 1) / kRows, share = most / sequences;
  const int64_t blocks = need < share ? need : share;
  return blocks > 1 ? blocks : 1;  // (without tokens a workgroup still writes zeros)
}
template <int EPL, bool BF16, bool SIGMOID>
hipError_t run_forward(const BalanceArgs &p, bool one, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(p.blocks), static_cast<uint32_t>(p.sequences));
  if (one)
    balance_kernel<EPL, BF16, SIGMOID, true><<<grid, dim3(kThreads), 0, stream>>>(p);
  else
    balance_kernel<EPL, BF16, SIGMOID, false><<<grid, dim3(kThreads), 0, stream>>>(p);
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

bool one_block(int64_t tokens, int64_t sequences) { return sequences == 1 && tokens <= kOneBlockTokens; }

}  // namespace

size_t moe_balance_workspace_bytes(int64_t tokens, int64_t experts, int64_t sequences) {
  if (one_block(tokens, sequences)) return 0;
  const int64_t blocks = sequences * blocks_a_sequence(tokens / sequences, sequences, kForwardBlocks);
  return static_cast<size_t>(blocks * (2 * experts + 1) + sequences + 1) * 4;
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
  p.vec = rows_aligned16(a.logits, p.row_bytes);
  p.ids = a.ids;
  p.scale = a.coef / static_cast<float>(a.sequences);
  p.loss = a.loss;
  p.probs = a.probs;
  p.counts = a.counts;
  p.tokens = a.live;
  const bool one = one_block(a.tokens, a.sequences);
  p.blocks = one ? 1 : static_cast<int>(blocks_a_sequence(p.seq, a.sequences, kForwardBlocks));
  const int64_t blocks = p.sequences * static_cast<int64_t>(p.blocks);
  if (!one) {
    p.part_probs = static_cast<float *>(a.workspace);
    p.part_counts = reinterpret_cast<int32_t *>(p.part_probs + blocks * p.E);
    p.part_tokens = p.part_counts + blocks * p.E;
    p.part_loss = reinterpret_cast<float *>(p.part_tokens + blocks);
    p.done = reinterpret_cast<uint32_t *>(p.part_loss + p.sequences);
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
  int width = 64;
  while (width < p.E) width *= 2;
  balance_sum_kernel<<<dim3(static_cast<uint32_t>(p.sequences)), dim3(kSumThreads), 0, a.stream>>>(p, width);
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
  p.blocks = static_cast<int>(blocks_a_sequence(p.seq, a.sequences, kBackwardBlocks));
  p.vec = rows_aligned16(a.logits, p.row_bytes);
  p.vec_din = rows_aligned16(a.dlogits_in, p.din_row_bytes);
  p.vec_out = rows_aligned16(a.dlogits, p.out_row_bytes);
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
