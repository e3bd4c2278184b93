// moe_route.hip -- routing of tokens to experts, its gradient, and the plan of a grouped product.
//
// Routing.  Sixteen lanes (one DPP row) own a token and hold its P = 16 EPL >= E experts, lane i the
// experts [i EPL, (i + 1) EPL): reductions over a token are four DPP steps, and a wave routes four
// tokens at once.  The softmax sum is one fixed order -- neighbours first -- which this layout gives
// for free (the lane's own EPL values pairwise, then lanes 1, 2, 4, 8 apart), so scores, and with them
// every choice, are the same bits in any implementation of that order.  top_k rounds then each take
// the largest key of the row (a DPP maximum, a ballot for the lowest lane that holds it).
//
// Plan.  A counting sort, stable in the slots: each chunk of tokens counts its experts (the routing
// kernel does so itself), and a second kernel gives every slot its row: the experts' totals and the
// counts of the chunks before it, then the slot's rank among its chunk's equal ids, found with ballots
// over the id's bits.  Up to 16 tokens (one chunk) the routing workgroup does all of it: one launch.
//
// What bounds them: the bytes are few (16384 tokens over 256 experts: 19 MB, 4 us).  The choice takes 1217 vector
// instructions a wave of four tokens; with four waves a SIMD these are issued in 57% of its cycles and scalar ones in
// 14%, while a wave by itself waits for 57% of its time (the rounds are a chain of exchanges, a ballot and a bit scan).
// 16384 tokens, 8 of 256 experts: 16.1 to 16.9 us with four of eight groups, sigmoid and bias, 12.2 without groups;
// 8192 tokens bf16, softmax 11.3 to 12.3, its gradient 6.2 to 6.5 (two waves a SIMD, vector instructions in 43% of the
// cycles); the sigmoid's gradient 9.1 us for 16384 tokens of 256 experts in fp32;
// one token over 64 experts with the plan 4.3 us, of which the work is less than half.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int kMaxExperts = 512;
constexpr int kPlanThreads = 1024;     // 16 waves
constexpr int kOneBlockSlots = 4096;   // planned from given ids by one workgroup
constexpr int64_t kMaxBlocks = int64_t(1) << 20;  // of a launch (2^32 threads or more do not launch)
// Tokens that one workgroup routes and plans (no workspace then): more would share its four SIMDs, and two
// launches are faster (64 tokens over 256 experts: 19 us in one launch, 13 in two).
constexpr int64_t kOneBlockTokens = 16;
constexpr float kNegInf = -__builtin_huge_valf();

// Value of the lane CTRL away in the DPP row of 16 lanes.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

// Over the 16 lanes of a row; every lane has the result.  (After the first two steps the lanes of a
// quad agree, so the mirrors are exchanges 4 and 8 apart: the sum's order is neighbours first.)
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  return v;
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<kXor1>(v));
  v = fmaxf(v, dpp<kXor2>(v));
  v = fmaxf(v, dpp<kHalfMirror>(v));
  v = fmaxf(v, dpp<kMirror>(v));
  return v;
}

template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ int row_max(int v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  v = max(v, dpp<kMirror>(v));
  return v;
}

// Keys as integers of the same order (no NaN arithmetic in the maxima); kClosed is below every key.
constexpr int kClosed = -2147483647 - 1;
__device__ __forceinline__ int order_of(float v) {
  const int b = __float_as_int(v);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float value_of(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }

// The lane's EPL logits from expert e0 on, as routing takes them: closed experts (-inf, NaN, beyond E)
// are -inf, others capped at FLT_MAX.  vec: the row is 16-byte aligned.
template <int EPL, bool BF16>
__device__ __forceinline__ void load_logits(const uint8_t *row, int e0, int E, bool vec, float (&l)[EPL]) {
  constexpr int ES = BF16 ? 2 : 4, BYTES = EPL * ES;
  if (vec && BYTES % 4 == 0 && e0 + EPL <= E) {
    uint32_t w[BYTES < 4 ? 1 : BYTES / 4];
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) {
        const uint4 v = *reinterpret_cast<const uint4 *>(row + e0 * ES + 16 * i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    } else if constexpr (BYTES == 8) {
      const uint2 v = *reinterpret_cast<const uint2 *>(row + e0 * ES);
      w[0] = v.x;
      w[1] = v.y;
    } else if constexpr (BYTES == 4) {
      w[0] = *reinterpret_cast<const uint32_t *>(row + e0 * ES);
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if constexpr (BF16)
        l[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
      else
        l[j] = __uint_as_float(w[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      l[j] = kNegInf;
      if (e0 + j < E) {
        if constexpr (BF16)
          l[j] = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[e0 + j]) << 16);
        else
          l[j] = reinterpret_cast<const float *>(row)[e0 + j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) l[j] = l[j] > kNegInf ? fminf(l[j], 3.402823466e+38f) : kNegInf;  // NaN -> -inf
}

// Correctly rounded 1 / x and e / total without the general division's range handling: the hardware's
// reciprocal and one Newton step, then (Markstein) one corrected quotient, each with a fused remainder.  For
// 1 <= x <= 2^125 and, in the quotient, 1 <= total <= 512 and e = 0 or 2^-100 <= e <= 1: no step under-
// or overflows there.  Elsewhere the general division, for a whole wave; the two give the same bits, so a token's
// choice does not depend on the tokens beside it.  (The Newton step is correctly rounded for every x if its start is,
// and for all but 32 significands if that is an ulp off.  The tests take those 32 through the keys: this chip's
// reciprocal is right there too.)
__device__ __forceinline__ float recip(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  return fmaf(fmaf(-x, r, 1.0f), r, r);
}
__device__ __forceinline__ float quotient(float e, float total, float r) {
  const float q = e * r;
  return fmaf(fmaf(-q, total, e), r, q);
}
constexpr float kPlainMost = 0x1p125f, kPlainLeast = 0x1p-100f;

// Scores (0 where closed: exp(-inf) = 0 and 1 / inf = 0).  (top, total): the row's softmax maximum and sum, 0
// and 1 for a row without an open expert.
__device__ __forceinline__ float softmax_score(float l, float top, float total) { return expf(l - top) / total; }
__device__ __forceinline__ float sigmoid_score(float l) { return 1.0f / (1.0f + expf(-l)); }
// s (1 - s).  For l >= 0 the complement is e s with e = exp(-l): 1 - s would lose it in the rounding of s (up to 1e-4 of
// it at l = 8, all of it from 17 on).
__device__ __forceinline__ float sigmoid_slope(float l) {
  const float e = expf(-l), s = 1.0f / (1.0f + e);
  return s * (l >= 0.0f ? e * s : 1.0f - s);
}

template <int EPL, bool SIGMOID>
__device__ __forceinline__ void row_scores(const float (&l)[EPL], float (&s)[EPL], float &top, float &total) {
  top = 0.0f;
  total = 1.0f;
  if constexpr (SIGMOID) {
    // (a closed expert has an infinite s, and so has a lane's padding, so with masks and with any number of experts but
    // 16, 32, .. 512 the wave takes the general division)
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      s[j] = 1.0f + expf(-l[j]);
      most = fmaxf(most, s[j]);
    }
    if (__ballot(most > kPlainMost)) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) s[j] = 1.0f / s[j];
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) s[j] = recip(s[j]);
    }
  } else {
    top = l[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) top = fmaxf(top, l[j]);
    top = row_max(top);
    top = top > kNegInf ? top : 0.0f;
    float t[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) t[j] = s[j] = expf(l[j] - top);
#pragma unroll
    for (int n = EPL; n > 1; n /= 2)
#pragma unroll
      for (int j = 0; j < n / 2; ++j) t[j] = t[2 * j] + t[2 * j + 1];
    total = row_sum(t[0]);
    total = total > 0.0f ? total : 1.0f;
    bool small = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) small |= s[j] < kPlainLeast && s[j] > 0.0f;
    if (__ballot(small)) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) s[j] = s[j] / total;
    } else {
      const float r = recip(total);
#pragma unroll
      for (int j = 0; j < EPL; ++j) s[j] = quotient(s[j], total, r);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const uint8_t *row, int e) {
  float v;
  if constexpr (BF16)
    v = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[e]) << 16);
  else
    v = reinterpret_cast<const float *>(row)[e];
  return v > kNegInf ? fminf(v, 3.402823466e+38f) : kNegInf;
}

// ---- plan ----------------------------------------------------------------------------------------
// Entries of a chunk's counts in the workspace: whole 16 bytes.
__host__ __device__ constexpr int count_pitch(int E) { return (E + 3) / 4 * 4; }

struct PlanLds {
  int32_t base[kMaxExperts];                // next row of each expert for this chunk
  alignas(16) int32_t wave_count[16][kMaxExperts];      // of the current tile of 1024 slots
  int32_t scan[16];
};

// Exclusive scan of v over the first 512 threads of a workgroup of 1024; total of all in *total.
__device__ __forceinline__ int32_t scan512(int32_t v, int32_t *scratch, int32_t *total) {
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  int32_t s = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int32_t o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  if (lane == 63) scratch[wave] = s;
  __syncthreads();
  int32_t before = 0, all = 0;
#pragma unroll
  for (uint32_t w = 0; w < 8; ++w) {
    const int32_t c = scratch[w];
    before += w < wave ? c : 0;
    all += c;
  }
  *total = all;
  return before + s - v;
}

// Rows of the slots [slot0, slot1) of one chunk, in order; lds.base holds each expert's next row.
// Called by a whole workgroup of 1024; base is complete and synchronised.
__device__ __forceinline__ void place_slots(PlanLds &lds, const int32_t *ids, int64_t slot0, int64_t slot1, int E,
                                            int bits, int64_t total, int32_t *rows, int32_t *pos, int32_t first_id) {
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
  for (int64_t s0 = slot0; s0 < slot1; s0 += kPlanThreads) {
    int4 *const clear = reinterpret_cast<int4 *>(&lds.wave_count[0][0]);
    for (int e = tid; e < 4 * kMaxExperts; e += kPlanThreads) clear[e] = make_int4(0, 0, 0, 0);
    __syncthreads();
    const int64_t slot = s0 + tid;
    const int32_t id = s0 == slot0 ? first_id : slot < slot1 ? ids[slot] : -1;
    const bool live = id >= 0 && id < E;
    // the lanes of this wave with the same id
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((id >> b) & 1);
      same &= ((id >> b) & 1) ? m : ~m;
    }
    const uint32_t rank = __popcll(same & ((1ull << lane) - 1));
    if (live && rank == 0) lds.wave_count[wave][id] = __popcll(same);
    __syncthreads();
    if (tid < kMaxExperts && static_cast<int>(tid) < E) {
      int32_t at = lds.base[tid];
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        const int32_t c = lds.wave_count[w][tid];
        lds.wave_count[w][tid] = at;
        at += c;
      }
      lds.base[tid] = at;
    }
    __syncthreads();
    if (slot < slot1) {
      int32_t p = -1;
      if (live) {
        p = lds.wave_count[wave][id] + static_cast<int32_t>(rank);
        rows[p] = static_cast<int32_t>(slot);
      }
      pos[slot] = p;
      if (slot >= total) rows[slot] = -1;  // rows beyond the last expert's (no slot is placed there)
    }
    __syncthreads();
  }
}

// counts: [chunks][count_pitch(E)] from the first kernel; chunk c has the slots [c * per, min((c + 1) * per, slots)).
__global__ __launch_bounds__(kPlanThreads) void place_kernel(const int32_t *ids, const int32_t *counts, int chunks,
                                                             int64_t per, int64_t slots, int E, int bits,
                                                             int32_t *offsets, int32_t *rows, int32_t *pos) {
  __shared__ PlanLds lds;
  const uint32_t tid = threadIdx.x;
  const int c = blockIdx.x;
  const int64_t slot0 = c * per, slot1 = min(slot0 + per, slots);
  const int32_t first_id = slot0 + tid < slot1 ? ids[slot0 + tid] : -1;
  // each expert's counts of all chunks and of those before this one: a thread takes four experts of every
  // parts-th chunk in loads of 16 bytes (16384 tokens, 8 of 256 experts: 9.0 us with loads of 4, 8.2 with these; 8 of
  // 64 experts 7.4 us, so what is left is the launch and the scattered rows)
  const int pitch = count_pitch(E), quads = pitch / 4;
  const int shift = bits < 8 ? 6 : bits - 2;  // threads to 4 << shift experts: 16 parts at most
  const int quad = tid & ((1 << shift) - 1), part = tid >> shift, parts = kPlanThreads >> shift;
  int4 before = make_int4(0, 0, 0, 0), all = before;
  if (quad < quads) {
    const int4 *column = reinterpret_cast<const int4 *>(counts) + quad;
#pragma unroll 8
    for (int i = part; i < chunks; i += parts) {
      const int4 n = column[static_cast<int64_t>(i) * quads];
      const int32_t m = i < c ? -1 : 0;
      all.x += n.x;
      all.y += n.y;
      all.z += n.z;
      all.w += n.w;
      before.x += n.x & m;
      before.y += n.y & m;
      before.z += n.z & m;
      before.w += n.w & m;
    }
  }
  int4 *const sums = reinterpret_cast<int4 *>(&lds.wave_count[0][0]);  // [2][1024]
  sums[tid] = all;
  sums[kPlanThreads + tid] = before;
  __syncthreads();
  int32_t total, n_all = 0, n_before = 0;
  if (tid < 4u << shift) {
    const int32_t *column = &lds.wave_count[0][0] + tid;
    for (int i = 0; i < parts; ++i) {
      n_all += column[i * (4 << shift)];
      n_before += column[(4 * kPlanThreads) + i * (4 << shift)];
    }
  }
  const int32_t first = scan512(n_all, lds.scan, &total);
  if (tid < kMaxExperts) lds.base[tid] = first + n_before;
  if (c == 0) {
    if (static_cast<int>(tid) < E) offsets[tid] = first;
    if (tid == 0) offsets[E] = total;
  }
  __syncthreads();
  place_slots(lds, ids, slot0, slot1, E, bits, total, rows, pos, first_id);
}

// The whole plan of at most 64 slots by one workgroup of 512 or more: each lane of the first wave compares its
// slot's id with all others bit by bit, and the offsets are found in the sorted ids.
__device__ __forceinline__ void plan_wave(PlanLds &lds, const int32_t *ids, int slots, int E, int bits,
                                          int32_t *offsets, int32_t *rows, int32_t *pos) {
  const uint32_t tid = threadIdx.x;
  if (tid < 64) {
    const int lane = tid;
    const int32_t id = lane < slots ? ids[lane] : -1;
    const bool live = id >= 0 && id < E;
    const uint64_t all = __ballot(live);
    uint64_t same = all, less = 0;  // slots whose id agrees with this one's so far; whose id is smaller
    for (int b = bits - 1; b >= 0; --b) {
      const bool one = (id >> b) & 1;
      const uint64_t ones = __ballot(one);
      less |= one ? same & ~ones : 0ull;
      same &= one ? ones : ~ones;
    }
    const int p = __popcll(less) + __popcll(same & ((1ull << lane) - 1));
    lds.base[lane] = E;  // (beyond the placed slots)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (live) {
      rows[p] = lane;
      lds.base[p] = id;
    }
    if (lane < slots) {
      pos[lane] = live ? p : -1;
      if (lane >= __popcll(all)) rows[lane] = -1;
    }
  }
  __syncthreads();
  for (int e = tid; e <= E; e += blockDim.x) {
    int lo = 0;  // slots with an id below e
#pragma unroll
    for (int n = 32; n > 0; n /= 2) lo += lds.base[lo + n - 1] < e ? n : 0;
    lo += lo < 64 && lds.base[lo < 64 ? lo : 63] < e ? 1 : 0;
    offsets[e] = lo;
  }
}

// The whole plan of at most kOneBlockSlots slots by one workgroup of 1024.
__device__ __forceinline__ void plan_block(PlanLds &lds, const int32_t *ids, int64_t slots, int E, int bits,
                                           int32_t *offsets, int32_t *rows, int32_t *pos) {
  const uint32_t tid = threadIdx.x;
  if (tid < kMaxExperts) lds.base[tid] = 0;
  __syncthreads();
  for (int64_t s = tid; s < slots; s += kPlanThreads) {
    const int32_t id = ids[s];
    if (id >= 0 && id < E) atomicAdd(&lds.base[id], 1);
  }
  __syncthreads();
  const int32_t n = tid < kMaxExperts ? lds.base[tid] : 0;
  int32_t total;
  const int32_t first = scan512(n, lds.scan, &total);
  if (tid < kMaxExperts) lds.base[tid] = first;
  if (static_cast<int>(tid) < E) offsets[tid] = first;
  if (tid == 0) offsets[E] = total;
  __syncthreads();
  place_slots(lds, ids, 0, slots, E, bits, total, rows, pos, tid < slots ? ids[tid] : -1);
}

__global__ __launch_bounds__(kPlanThreads) void plan_one_kernel(const int32_t *ids, int64_t slots, int E, int bits,
                                                                int32_t *offsets, int32_t *rows, int32_t *pos) {
  __shared__ PlanLds lds;
  plan_block(lds, ids, slots, E, bits, offsets, rows, pos);
}

// counts[c][e] of the slots of chunk c.
__global__ __launch_bounds__(256) void count_kernel(const int32_t *ids, int64_t per, int64_t slots, int E,
                                                    int32_t *counts) {
  __shared__ int32_t hist[kMaxExperts];
  for (int e = threadIdx.x; e < kMaxExperts; e += 256) hist[e] = 0;
  __syncthreads();
  const int64_t s0 = blockIdx.x * per, s1 = min(s0 + per, slots);
  for (int64_t s = s0 + threadIdx.x; s < s1; s += 256) {
    const int32_t id = ids[s];
    if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
  }
  __syncthreads();
  const int pitch = count_pitch(E);
  for (int e = threadIdx.x; e < pitch; e += 256) counts[static_cast<int64_t>(blockIdx.x) * pitch + e] = hist[e];
}

// ---- routing --------------------------------------------------------------------------------------
struct RouteArgs {
  const uint8_t *logits;
  int64_t row_bytes;
  int64_t tokens, per;  // tokens of a workgroup: [b * per, (b + 1) * per)
  int E, G, GS, group_k, k;
  int group_lanes;  // lanes of a group, where groups are whole lanes and a power of two of them (else 0)
  bool sum2, renorm, vec, vec_bias;
  float scale;
  const float *bias;
  int32_t *ids;
  float *weights;
  int32_t *counts;  // nullable [blocks][count_pitch(E)]
  int32_t *offsets, *rows, *pos;  // the whole plan (one workgroup of 1024), else NULL
  int bits;
};

// (m1, m2): the two largest of both pairs.
__device__ __forceinline__ void merge_two(int &m1, int &m2, int o1, int o2) {
  m2 = max(min(m1, o1), max(m2, o2));
  m1 = max(m1, o1);
}
template <int CTRL>
__device__ __forceinline__ void merge_two(int &m1, int &m2) {
  const int o1 = dpp<CTRL>(m1), o2 = dpp<CTRL>(m2);
  merge_two(m1, m2, o1, o2);
}

// Closes the experts of the groups that are not among the row's group_k best.  Where a group is 1, 2, 4, 8 or
// 16 whole lanes (group_lanes) its two best keys meet by lane exchanges; else through `keys`, the row's copy in
// LDS, which lane g reads for group g.
template <int EPL>
__device__ __forceinline__ void keep_groups(int (&key)[EPL], int *keys, const RouteArgs &p, uint32_t lane) {
  const int l16 = lane & 15, W = p.group_lanes;
  int m1 = kClosed, m2 = kClosed;
  int mine, stride;  // the group whose value this lane holds, lanes between the groups' values
  if (W > 0) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      m2 = max(min(m1, m2), min(max(m1, m2), key[j]));  // (the median of three: one instruction)
      m1 = max(m1, key[j]);
    }
    if (W > 1) merge_two<kXor1>(m1, m2);
    if (W > 2) merge_two<kXor2>(m1, m2);
    if (W > 4) merge_two<kHalfMirror>(m1, m2);
    if (W > 8) merge_two<kMirror>(m1, m2);
    mine = l16 / W;
    stride = W;
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) keys[l16 * EPL + j] = key[j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    mine = l16;
    stride = 1;
    if (l16 < p.G) {
      int at = l16 % p.GS;  // (each lane starts elsewhere in its group: other banks)
      for (int i = 0; i < p.GS; i += 4) {
        int v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[u] = i + u < p.GS ? keys[l16 * p.GS + at] : kClosed;
          at = at + 1 == p.GS ? 0 : at + 1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          m2 = max(m2, min(m1, v[u]));
          m1 = max(m1, v[u]);
        }
      }
    }
  }
  int value = m1;
  if (p.sum2 && m2 != kClosed) value = order_of((value_of(m1) + value_of(m2)) + 0.0f);
  if (mine >= p.G) value = kClosed;
  // the group's place: how many groups come before it
  int place = 0;
  for (int g0 = 0; g0 < p.G; g0 += 4) {
    int o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) o[u] = __shfl(value, (lane & 48) + min(g0 + u, p.G - 1) * stride);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (g0 + u < p.G) place += (o[u] > value || (o[u] == value && g0 + u < mine)) ? 1 : 0;
  }
  const bool stays = place < p.group_k;
  if (W > 0) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = stays ? key[j] : kClosed;
    return;
  }
  const uint32_t kept = static_cast<uint32_t>(__ballot(stays) >> (lane & 48)) & 0xFFFFu;
  int g = l16 * EPL / p.GS, left = (g + 1) * p.GS - l16 * EPL;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    if (!((kept >> g) & 1u)) key[j] = kClosed;
    if (--left == 0) {
      ++g;
      left = p.GS;
    }
  }
}

// The k best experts of the row in falling order, ties to the lower index: slot r to lane r mod 16, id_lo or id_hi.
// k rounds of: the row's best key, the lowest lane that holds it, that lane's first expert with it.
template <int EPL>
__device__ __forceinline__ void choose_by_rounds(int (&key)[EPL], int k, uint32_t lane, int &id_lo, int &id_hi) {
  const int l16 = lane & 15;
  int best = key[0];
#pragma unroll
  for (int j = 1; j < EPL; ++j) best = max(best, key[j]);
  for (int r = 0; r < k; ++r) {
    const int m = row_max(best);
    const uint32_t holds = static_cast<uint32_t>(__ballot(best == m) >> (lane & 48)) & 0xFFFFu;
    const int owner = __ffs(holds) - 1;
    // the lowest lane that holds the key closes it, and gets a bit for every expert of its that has it, the
    // first expert's the highest.  In integer arithmetic, since a lane mask for every compare costs wait
    // states: t is 0 for the key and -1 for a smaller one (other lanes want a key above all).
    const int want = l16 == owner ? m : 2147483647;
    int misses = 0;
    best = kClosed;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      int t = __builtin_elementwise_sub_sat(key[j], want) >> 31;
      asm("" : "+v"(t));  // (else the compiler goes back to compares)
      misses = (misses << 1) + t;
      key[j] = (key[j] & t) | (kClosed & ~t);
      best = max(best, key[j]);
    }
    const uint32_t hits = static_cast<uint32_t>(misses) + (EPL == 32 ? 0xFFFFFFFFu : (1u << (EPL & 31)) - 1u);
    const uint32_t others = hits & ((1u << (31 - __clz(hits | 1u))) - 1u);
    if (__ballot(others != 0 && m != kClosed)) {  // equal keys in one lane: all but the first come back
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if ((others >> (EPL - 1 - j)) & 1u) key[j] = m;
      best = others ? m : best;
    }
    const int at = __clz(hits) - (32 - EPL);
    const int id = m != kClosed ? owner * EPL + __shfl(at, (lane & 48) + owner) : -1;
    if (l16 == (r & 15)) {
      if (r < 16)
        id_lo = id;
      else
        id_hi = id;
    }
  }
}

// The same without closing keys: the owner's next best is its largest key below the one chosen, two instructions a
// key, and the experts behind the keys are looked up for all slots at once.  False, with nothing chosen, where a lane
// holds a chosen key twice (the rounds then start again): rare among fp32 scores, not among bf16 ones.
// 16384 tokens, 8 of 256 experts in four of eight groups 18.6 -> 16.3 us, without groups 15.5 -> 12.2; 512
// experts 28 -> 22.
template <int EPL>
__device__ __forceinline__ bool choose_unequal(const int (&key)[EPL], int k, uint32_t lane, int &id_lo, int &id_hi) {
  const int l16 = lane & 15;
  int best = key[0];
#pragma unroll
  for (int j = 1; j < EPL; ++j) best = max(best, key[j]);
  int m_lo = kClosed, m_hi = kClosed, from_lo = 0, from_hi = 0;
  for (int r = 0; r < k; ++r) {
    const int m = row_max(best);
    const uint32_t holds = static_cast<uint32_t>(__ballot(best == m) >> (lane & 48)) & 0xFFFFu;
    const int owner = __ffs(holds) - 1;
    // modulo 2^32, key - m is larger for every key below m than for the others, and rises with the key
    uint32_t next = static_cast<uint32_t>(kClosed) - static_cast<uint32_t>(m);
#pragma unroll
    for (int j = 0; j < EPL; ++j) next = max(next, static_cast<uint32_t>(key[j]) - static_cast<uint32_t>(m));
    best = l16 == owner && m != kClosed ? static_cast<int>(next + static_cast<uint32_t>(m)) : best;
    if (l16 == (r & 15)) {
      if (r < 16) {
        m_lo = m;
        from_lo = owner;
      } else {
        m_hi = m;
        from_hi = owner;
      }
    }
  }
  bool twice = false;
  const auto expert_of = [&](int m, int from) {
    uint32_t misses = 0;  // a bit for every expert of that lane with another key, the first expert's the highest
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      uint32_t other = min(static_cast<uint32_t>(__shfl(key[j], (lane & 48) + from) ^ m), 1u);
      asm("" : "+v"(other));
      misses = (misses << 1) + other;
    }
    const uint32_t hits = ~misses << (32 - EPL);
    twice |= m != kClosed && (hits & (hits - 1)) != 0;
    return m != kClosed ? from * EPL + __clz(hits) : -1;
  };
  id_lo = expert_of(m_lo, from_lo);
  if (k > 16) id_hi = expert_of(m_hi, from_hi);
  return __ballot(twice) == 0;
}

template <int EPL, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kPlanThreads) void route_kernel(RouteArgs p) {
  constexpr int P = 16 * EPL;
  __shared__ int32_t hist[kMaxExperts];
  // with groups that are not whole lanes: P keys a token; then, where this workgroup makes the plan, the plan's
  extern __shared__ __attribute__((aligned(16))) uint8_t area[];
  const uint32_t wave = threadIdx.x >> 6;
  if (p.counts) {
    for (int e = threadIdx.x; e < count_pitch(p.E); e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  const int64_t t1 = min(p.tokens, (blockIdx.x + 1) * p.per);
  const int step = blockDim.x / 16;
  for (int64_t tb = blockIdx.x * p.per; tb < t1; tb += step) {
    if (tb + 4 * wave >= t1) continue;  // (no workgroup barrier inside)
    // (an opaque copy: nothing that depends on the lane is computed ahead of the loop, for paths not taken)
    uint32_t lane = threadIdx.x & 63u;
    asm volatile("" : "+v"(lane));
    const int l16 = lane & 15;
    const int64_t t = tb + (threadIdx.x >> 4);
    const bool exists = t < t1;
    const uint8_t *row = p.logits + (exists ? t : t1 - 1) * p.row_bytes;
    float l[EPL], s[EPL], top, total;
    load_logits<EPL, BF16>(row, l16 * EPL, p.E, p.vec, l);
    row_scores<EPL, SIGMOID>(l, s, top, total);
    if (p.bias) {
      float b[EPL];
      if (EPL >= 4 && p.vec_bias && l16 * EPL + EPL <= p.E) {
#pragma unroll
        for (int j = 0; j + 4 <= EPL; j += 4) {
          const float4 v = *reinterpret_cast<const float4 *>(p.bias + l16 * EPL + j);
          b[j] = v.x;
          b[(j + 1) % EPL] = v.y;
          b[(j + 2) % EPL] = v.z;
          b[(j + 3) % EPL] = v.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) b[j] = p.bias[min(l16 * EPL + j, p.E - 1)];
      }
#pragma unroll
      for (int j = 0; j < EPL; ++j) s[j] += b[j];
    }
    // (a NaN key closes too; + 0 so that a key of -0 is +0)
    int key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const bool is_open = (l[j] > kNegInf) & (s[j] > kNegInf);
      key[j] = is_open ? order_of(s[j] + 0.0f) : kClosed;
    }
    if (p.group_k < p.G) keep_groups<EPL>(key, reinterpret_cast<int *>(area) + (threadIdx.x >> 4) * P, p, lane);

    int id_lo = -1, id_hi = -1;  // slots l16 and 16 + l16
    if constexpr (EPL >= 4 && !BF16) {
      if (!choose_unequal<EPL>(key, p.k, lane, id_lo, id_hi)) choose_by_rounds<EPL>(key, p.k, lane, id_lo, id_hi);
    } else {
      choose_by_rounds<EPL>(key, p.k, lane, id_lo, id_hi);
    }
    // the chosen experts' scores, formed again from their logits (the same operations, the same bits)
    auto score_of = [&](int id) {
      if (id < 0) return 0.0f;
      const float v = load_logit<BF16>(row, id);
      return SIGMOID ? sigmoid_score(v) : softmax_score(v, top, total);
    };
    float w_lo = score_of(id_lo), w_hi = p.k > 16 ? score_of(id_hi) : 0.0f;
    if (p.renorm) {
      const float sum = row_sum(w_lo + w_hi) + 1e-20f;
      w_lo /= sum;
      w_hi /= sum;
    }
    if (exists) {
      if (l16 < p.k) {
        p.ids[t * p.k + l16] = id_lo;
        p.weights[t * p.k + l16] = w_lo * p.scale;
        if (p.counts && id_lo >= 0) atomicAdd(&hist[id_lo], 1);
      }
      if (16 + l16 < p.k) {
        p.ids[t * p.k + 16 + l16] = id_hi;
        p.weights[t * p.k + 16 + l16] = w_hi * p.scale;
        if (p.counts && id_hi >= 0) atomicAdd(&hist[id_hi], 1);
      }
    }
  }
  if (p.counts) {
    __syncthreads();
    const int pitch = count_pitch(p.E);
    int32_t *const counts = p.counts + static_cast<int64_t>(blockIdx.x) * pitch;
    for (int e = threadIdx.x; e < pitch; e += blockDim.x) counts[e] = hist[e];
  }
  if (p.offsets) {
    __syncthreads();  // the ids are in global memory for the whole workgroup
    PlanLds &lds = *reinterpret_cast<PlanLds *>(area);
    if (p.tokens * p.k <= 64)
      plan_wave(lds, p.ids, static_cast<int>(p.tokens * p.k), p.E, p.bits, p.offsets, p.rows, p.pos);
    else
      plan_block(lds, p.ids, p.tokens * p.k, p.E, p.bits, p.offsets, p.rows, p.pos);
  }
}

// ---- gradient of the weights -------------------------------------------------------------------------
struct RouteBwdArgs {
  const uint8_t *logits;
  int64_t row_bytes;
  int64_t tokens;
  int E, k;
  bool renorm, vec, vec_out;
  float scale;
  const int32_t *ids;
  const float *dweights;
  uint8_t *dlogits;
  int64_t out_row_bytes;
  int64_t first_block;  // of this launch
};

__device__ __forceinline__ uint32_t bf16_of(float v) {
  return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(v)));
}

template <int EPL, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteBwdArgs p) {
  constexpr int P = 16 * EPL;
  __shared__ float ds_lds[16][P];  // gradient of each expert's score (sigmoid: of its logit), a row a token
  const uint32_t lane = threadIdx.x & 63u;
  const int l16 = lane & 15;
  const int64_t t = (p.first_block + blockIdx.x) * 16 + (threadIdx.x >> 4);
  const bool exists = t < p.tokens;
  const int64_t tr = exists ? t : p.tokens - 1;
  const uint8_t *row = p.logits + tr * p.row_bytes;
  float l[EPL], s[EPL], top = 0.0f, total = 1.0f;
  if constexpr (!SIGMOID) {
    load_logits<EPL, BF16>(row, l16 * EPL, p.E, p.vec, l);
    row_scores<EPL, false>(l, s, top, total);
  }

  // the row's slots l16 and 16 + l16: score, slope (sigmoid) and gradient
  float picked[2] = {0.0f, 0.0f}, slope[2] = {0.0f, 0.0f}, g[2] = {0.0f, 0.0f};
  int id[2] = {-1, -1};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = 16 * h + l16;
    if (j < p.k) {
      const int e = p.ids[tr * p.k + j];
      if (e >= 0 && e < p.E) {
        const float v = load_logit<BF16>(row, e);
        id[h] = e;
        picked[h] = SIGMOID ? sigmoid_score(v) : softmax_score(v, top, total);
        if (SIGMOID) slope[h] = sigmoid_slope(v);
        g[h] = p.dweights[tr * p.k + j] * p.scale;
      }
    }
  }
  // sum over the chosen of (gradient * score): the normaliser's own gradient, and the softmax's
  float gs = row_sum(fmaf(g[0], picked[0], g[1] * picked[1]));
  if (p.renorm) {
    const float sum = row_sum(picked[0] + picked[1]) + 1e-20f;
    const float mean = gs / sum;
    g[0] = (g[0] - mean) / sum;
    g[1] = (g[1] - mean) / sum;
    if (id[0] < 0) g[0] = 0.0f;
    if (id[1] < 0) g[1] = 0.0f;
    // The slot that has most of the sum: its weight's distance from the mean is lost in the mean's rounding.  What the
    // slots' g p add up to (mean 1e-20 / sum) gives it from the others.
    const bool leads[2] = {2.0f * picked[0] > sum, 2.0f * picked[1] > sum};
    if (__ballot(leads[0] || leads[1])) {
      const float others = row_sum(fmaf(leads[0] ? 0.0f : g[0], picked[0], leads[1] ? 0.0f : g[1] * picked[1]));
      const float left = fmaf(mean / sum, 1e-20f, -others);
      if (leads[0]) g[0] = left / picked[0];
      if (leads[1]) g[1] = left / picked[1];
    }
    if (!SIGMOID) gs = row_sum(fmaf(g[0], picked[0], g[1] * picked[1]));
  }
  // a sigmoid's gradient stays with its expert: it is formed here, and nothing is read for the others
  if (SIGMOID) {
    g[0] *= slope[0];
    g[1] *= slope[1];
  }
  float *ds = ds_lds[threadIdx.x >> 4];
#pragma unroll
  for (int j = 0; j < EPL; ++j) ds[l16 * EPL + j] = 0.0f;
  __syncthreads();
  // (an atomic add only so that an id given twice counts twice; distinct ids add to zero)
  if (id[0] >= 0) atomicAdd(&ds[id[0]], g[0]);
  if (id[1] >= 0) atomicAdd(&ds[id[1]], g[1]);
  __syncthreads();
  float d[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const float v = ds[l16 * EPL + j];
    if constexpr (SIGMOID)
      d[j] = v;
    else
      d[j] = s[j] * (v - gs);
  }
  // Likewise the expert with a softmax score above one half: a row's gradients add up to zero.
  if constexpr (!SIGMOID) {
    if (__ballot(total < 2.0f)) {
      float others = 0.0f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) others += s[j] > 0.5f ? 0.0f : d[j];
      others = row_sum(others);
#pragma unroll
      for (int j = 0; j < EPL; ++j) d[j] = s[j] > 0.5f ? -others : d[j];
    }
  }
  if (!exists) return;
  uint8_t *out = p.dlogits + t * p.out_row_bytes;
  constexpr int ES = BF16 ? 2 : 4, BYTES = EPL * ES;
  const int e0 = l16 * EPL;
  if (p.vec_out && BYTES % 16 == 0 && e0 + EPL <= p.E) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      uint4 v;
      uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = BF16 ? bf16_of(d[(8 * i + 2 * q) % EPL]) | bf16_of(d[(8 * i + 2 * q + 1) % EPL]) << 16
                    : __float_as_uint(d[(4 * i + q) % EPL]);
      *reinterpret_cast<uint4 *>(out + e0 * ES + 16 * i) = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (e0 + j < p.E) {
        if constexpr (BF16)
          reinterpret_cast<uint16_t *>(out)[e0 + j] = static_cast<uint16_t>(bf16_of(d[j]));
        else
          reinterpret_cast<float *>(out)[e0 + j] = d[j];
      }
  }
}

int id_bits(int64_t E) {
  int b = 0;
  while ((int64_t(1) << b) < E) ++b;
  return b;
}

// Experts a lane holds: the power of two that gives 16 lanes all of them.
int experts_per_lane(int64_t E) {
  int epl = 1;
  while (16 * epl < E) epl *= 2;
  return epl;
}

bool rows_aligned16(const void *p, int64_t row_bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && row_bytes % 16 == 0;
}

template <int EPL>
hipError_t run_route(const RouteArgs &p, bool bf16, bool sigmoid, int blocks, int threads, size_t lds,
                     hipStream_t stream) {
  auto *kernel = bf16 ? (sigmoid ? route_kernel<EPL, true, true> : route_kernel<EPL, true, false>)
                      : (sigmoid ? route_kernel<EPL, false, true> : route_kernel<EPL, false, false>);
  kernel<<<dim3(blocks), dim3(threads), lds, stream>>>(p);
  return hipGetLastError();
}

template <int EPL>
hipError_t run_route_backward(RouteBwdArgs p, bool bf16, bool sigmoid, hipStream_t stream) {
  auto *kernel = bf16 ? (sigmoid ? route_backward_kernel<EPL, true, true> : route_backward_kernel<EPL, true, false>)
                      : (sigmoid ? route_backward_kernel<EPL, false, true> : route_backward_kernel<EPL, false, false>);
  const int64_t blocks = (p.tokens + 15) / 16;
  for (p.first_block = 0; p.first_block < blocks; p.first_block += kMaxBlocks) {
    const int64_t n = blocks - p.first_block < kMaxBlocks ? blocks - p.first_block : kMaxBlocks;
    kernel<<<dim3(static_cast<uint32_t>(n)), dim3(256), 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t moe_workspace_bytes(int64_t tokens, int64_t experts) {
  if (tokens <= kOneBlockTokens) return 0;
  return static_cast<size_t>(kPlanChunks) * count_pitch(static_cast<int>(experts)) * sizeof(int32_t);
}

hipError_t launch_moe_plan(const int32_t *ids, int64_t slots, int64_t experts, int32_t *offsets, int32_t *rows,
                           int32_t *pos, int32_t *counts, hipStream_t stream) {
  const int E = static_cast<int>(experts), bits = id_bits(E);
  if (slots <= kOneBlockSlots) {
    plan_one_kernel<<<dim3(1), dim3(kPlanThreads), 0, stream>>>(ids, slots, E, bits, offsets, rows, pos);
    return hipGetLastError();
  }
  const int64_t per = ((slots + kPlanChunks - 1) / kPlanChunks + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
  const int chunks = static_cast<int>((slots + per - 1) / per);
  count_kernel<<<dim3(chunks), dim3(256), 0, stream>>>(ids, per, slots, E, counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  place_kernel<<<dim3(chunks), dim3(kPlanThreads), 0, stream>>>(ids, counts, chunks, per, slots, E, bits, offsets,
                                                                rows, pos);
  return hipGetLastError();
}

hipError_t launch_moe_route(const MoeRouteArgs &a) {
  RouteArgs p{};
  p.logits = static_cast<const uint8_t *>(a.logits);
  p.row_bytes = a.ld * (a.dtype == 1 ? 2 : 4);
  p.tokens = a.tokens;
  p.E = static_cast<int>(a.experts);
  p.G = a.num_groups;
  p.GS = p.E / p.G;
  p.group_k = a.group_top_k;
  p.k = a.top_k;
  p.sum2 = a.sum2;
  p.renorm = a.renorm;
  p.vec = rows_aligned16(a.logits, p.row_bytes);
  p.scale = a.scale;
  p.bias = a.bias;
  p.vec_bias = (reinterpret_cast<uintptr_t>(a.bias) & 15u) == 0;
  p.ids = a.ids;
  p.weights = a.weights;
  p.bits = id_bits(p.E);
  const bool plan = a.offsets != nullptr;
  if (a.tokens == 0)
    return plan ? launch_moe_plan(a.ids, 0, a.experts, a.offsets, a.rows, a.pos, a.workspace, a.stream) : hipSuccess;
  // keys of the tokens that a workgroup holds at once (whole waves of four), for the choice of groups
  const int epl = experts_per_lane(p.E);
  const int lanes = p.GS % epl == 0 ? p.GS / epl : 0;
  p.group_lanes = (lanes & (lanes - 1)) == 0 ? lanes : 0;
  const bool groups = p.group_k < p.G && p.group_lanes == 0;  // (through LDS)
  const bool one = plan && a.tokens <= kOneBlockTokens;
  size_t lds = 0;
  int blocks, threads;
  if (one) {
    p.offsets = a.offsets;
    p.rows = a.rows;
    p.pos = a.pos;
    p.per = a.tokens;
    blocks = 1;
    threads = a.tokens * a.top_k <= 64 ? 512 : kPlanThreads;
    lds = sizeof(PlanLds);
    if (groups && lds < static_cast<size_t>(kOneBlockTokens) * 16 * epl * sizeof(float))
      lds = static_cast<size_t>(kOneBlockTokens) * 16 * epl * sizeof(float);
  } else {
    // Chunks of whole workgroup steps, in at most kPlanChunks chunks where they are counted.  16 tokens a
    // workgroup (a wave a SIMD) as long as there are compute units for them, then 32 and 64: a wave's latency
    // is its instructions', so four waves a SIMD take four times as long.  With keys in LDS, at most 32 KB.
    const int64_t most = plan ? kPlanChunks : kMaxBlocks;
    threads = !plan || a.tokens <= 16 * most ? 256 : a.tokens <= 32 * most ? 512 : kPlanThreads;
    if (groups && threads * epl > 8192) threads = 8192 / epl;
    if (plan) p.counts = a.workspace;
    const int64_t at_once = threads / 16;
    p.per = ((a.tokens + most - 1) / most + at_once - 1) / at_once * at_once;
    lds = groups ? static_cast<size_t>(threads) * epl * sizeof(float) : 0;
    blocks = static_cast<int>((a.tokens + p.per - 1) / p.per);
  }
  hipError_t e;
  switch (epl) {
    case 1: e = run_route<1>(p, a.dtype == 1, a.sigmoid, blocks, threads, lds, a.stream); break;
    case 2: e = run_route<2>(p, a.dtype == 1, a.sigmoid, blocks, threads, lds, a.stream); break;
    case 4: e = run_route<4>(p, a.dtype == 1, a.sigmoid, blocks, threads, lds, a.stream); break;
    case 8: e = run_route<8>(p, a.dtype == 1, a.sigmoid, blocks, threads, lds, a.stream); break;
    case 16: e = run_route<16>(p, a.dtype == 1, a.sigmoid, blocks, threads, lds, a.stream); break;
    default: e = run_route<32>(p, a.dtype == 1, a.sigmoid, blocks, threads, lds, a.stream); break;
  }
  if (e != hipSuccess || !plan || one) return e;
  place_kernel<<<dim3(blocks), dim3(kPlanThreads), 0, a.stream>>>(a.ids, a.workspace, blocks, p.per * p.k,
                                                                  a.tokens * p.k, p.E, p.bits, a.offsets, a.rows, a.pos);
  return hipGetLastError();
}

hipError_t launch_moe_route_backward(const MoeRouteBackwardArgs &a) {
  RouteBwdArgs p{};
  const int es = a.dtype == 1 ? 2 : 4;
  p.logits = static_cast<const uint8_t *>(a.logits);
  p.row_bytes = a.ld * es;
  p.tokens = a.tokens;
  p.E = static_cast<int>(a.experts);
  p.k = a.top_k;
  p.renorm = a.renorm;
  p.vec = rows_aligned16(a.logits, p.row_bytes);
  p.vec_out = rows_aligned16(a.dlogits, a.ldd * es);
  p.scale = a.scale;
  p.ids = a.ids;
  p.dweights = a.dweights;
  p.dlogits = static_cast<uint8_t *>(a.dlogits);
  p.out_row_bytes = a.ldd * es;
  switch (experts_per_lane(p.E)) {
    case 1: return run_route_backward<1>(p, a.dtype == 1, a.sigmoid, a.stream);
    case 2: return run_route_backward<2>(p, a.dtype == 1, a.sigmoid, a.stream);
    case 4: return run_route_backward<4>(p, a.dtype == 1, a.sigmoid, a.stream);
    case 8: return run_route_backward<8>(p, a.dtype == 1, a.sigmoid, a.stream);
    case 16: return run_route_backward<16>(p, a.dtype == 1, a.sigmoid, a.stream);
    default: return run_route_backward<32>(p, a.dtype == 1, a.sigmoid, a.stream);
  }
}

}  // namespace nvfp4
