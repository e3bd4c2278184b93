// moe_rows.hip -- rows between tokens and experts: the gather into a plan's order, the weighted sum of
// the experts' rows, and its gradients.  All three move rows once (HBM-bound): a lane owns 16 bytes of
// a row's columns and walks the token's slots, so the k loads of a lane are independent and a token's
// own row (dout) is read once for all of its slots.  A token's sums run in the order of its slots.
// 4096 tokens of 8 rows of 4096 bf16: the sum 56 to 60 us (302 MB, 5.0 to 5.4 TB/s), its gradient 103 to
// 107 us (570 MB, 5.3 to 5.5 TB/s); a 1 GiB copy runs at 5.1 TB/s.  The gather 71 us (4.3 TB/s, nearly all writes).  16384 tokens of 8 rows of 512: gather 38
// us, sum 24; of 128 fp32 19 and 13 (59 and 20 with a workgroup a row).  One to a few tokens: 4 us, the launch.
#include "nvfp4_internal.h"
#include "vec_io.hpp"

namespace nvfp4 {
namespace {

constexpr int kRowThreads = 256;
// Workgroups along a launch's rows; each walks its share of a larger problem.
constexpr int64_t kMaxBlocks = 65535;

struct RowsArgs {
  const uint8_t *x;
  int64_t ldx;  // bytes
  const uint8_t *dout;
  int64_t ld_dout;  // bytes
  int64_t tokens;
  int pieces;  // 16-byte pieces of a row
  int lane_bits;  // gather, sum: 1 << lane_bits lanes a row (256 at most), so that short rows fill their workgroup
  const int32_t *pos, *rows;
  const float *weights;
  int k;
  uint8_t *out;
  int64_t ldo;  // bytes
  float *dweights;
};

template <bool ONCE>
__device__ __forceinline__ void store16(uint8_t *p, const uint4 &v) {
  if constexpr (ONCE)
    __builtin_nontemporal_store((vec_u32x4){v.x, v.y, v.z, v.w}, reinterpret_cast<vec_u32x4 *>(p));
  else
    *reinterpret_cast<uint4 *>(p) = v;
}

template <bool BF16>
__device__ __forceinline__ void unpack16(const uint4 &v, float (&f)[BF16 ? 8 : 4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (BF16) {
      f[2 * q] = __uint_as_float(w[q] << 16);
      f[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    } else {
      f[q] = __uint_as_float(w[q]);
    }
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack16(const float (&f)[BF16 ? 8 : 4]) {
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (BF16)
      w[q] = pack_bf16(f[2 * q], f[2 * q + 1]);
    else
      w[q] = __float_as_uint(f[q]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// y[r] = x[rows[r] / k]; the dtype does not matter.  A lane moves its piece of kGatherRows rows at once.
constexpr int kGatherRows = 4;
template <bool ONCE>
__global__ __launch_bounds__(kRowThreads) void gather_kernel(RowsArgs p) {
  const int c = blockIdx.x * kRowThreads + (threadIdx.x & ((1 << p.lane_bits) - 1));
  if (c >= p.pieces) return;
  const int64_t slots = p.tokens * p.k;
  const int rows_at_once = kRowThreads >> p.lane_bits;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows_at_once * kGatherRows + (threadIdx.x >> p.lane_bits); r0 < slots;
       r0 += static_cast<int64_t>(gridDim.y) * rows_at_once * kGatherRows) {
    uint4 v[kGatherRows];
#pragma unroll
    for (int u = 0; u < kGatherRows; ++u) {
      const int64_t r = r0 + u * rows_at_once;
      const uint32_t slot = r < slots ? static_cast<uint32_t>(p.rows[r]) : 0xFFFFFFFFu;
      v[u] = make_uint4(0, 0, 0, 0);
      if (slot < static_cast<uint64_t>(slots))
        v[u] = *reinterpret_cast<const uint4 *>(p.x + slot / static_cast<uint32_t>(p.k) * p.ldx + 16ll * c);
    }
#pragma unroll
    for (int u = 0; u < kGatherRows; ++u) {
      const int64_t r = r0 + u * rows_at_once;
      if (r < slots) store16<ONCE>(p.out + r * p.ldo + 16ll * c, v[u]);
    }
  }
}

template <bool BF16, bool ONCE>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(RowsArgs p) {
  constexpr int V = BF16 ? 8 : 4;
  const int c = blockIdx.x * kRowThreads + (threadIdx.x & ((1 << p.lane_bits) - 1));
  if (c >= p.pieces) return;
  const uint32_t slots = static_cast<uint32_t>(p.tokens * p.k);
  const int rows_at_once = kRowThreads >> p.lane_bits;
  for (int64_t t = static_cast<int64_t>(blockIdx.y) * rows_at_once + (threadIdx.x >> p.lane_bits); t < p.tokens;
       t += static_cast<int64_t>(gridDim.y) * rows_at_once) {
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += 8) {
      uint4 v[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = make_uint4(0, 0, 0, 0);
        w[j] = 0.0f;
        if (j0 + j < p.k) {
          const uint32_t row = static_cast<uint32_t>(p.pos[t * p.k + j0 + j]);
          if (row < slots) {  // (-1 is beyond)
            v[j] = load16<ONCE>(p.x + row * p.ldx + 16ll * c);
            w[j] = p.weights ? p.weights[t * p.k + j0 + j] : 1.0f;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j0 + j >= p.k) break;
        float f[V];
        unpack16<BF16>(v[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(w[j], f[i], acc[i]);
      }
    }
    *reinterpret_cast<uint4 *>(p.out + t * p.ldo + 16ll * c) = pack16<BF16>(acc);
  }
}

// LANES lanes a token, a wave or a workgroup; a workgroup's partial dot products of eight slots at a time meet in LDS.
template <bool BF16, bool ONCE, int LANES>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(RowsArgs p) {
  constexpr int V = BF16 ? 8 : 4, kTokens = kRowThreads / LANES;
  __shared__ float part[4][8];
  const int64_t slots = p.tokens * p.k;
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const int first = threadIdx.x % LANES;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + threadIdx.x / LANES; t < p.tokens;
       t += static_cast<int64_t>(gridDim.x) * kTokens) {
    const uint8_t *dout = p.dout + t * p.ld_dout;
    for (int j0 = 0; j0 < p.k; j0 += 8) {
      float dot[8], w[8];
      int64_t row[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dot[j] = 0.0f;
        w[j] = 0.0f;
        row[j] = -1;
        if (j0 + j < p.k) {
          const int64_t r = p.pos[t * p.k + j0 + j];
          row[j] = r < slots ? r : -1;
          w[j] = p.weights[t * p.k + j0 + j];
        }
      }
      for (int c = first; c < p.pieces; c += LANES) {
        uint4 v[8];
        const uint4 dv = *reinterpret_cast<const uint4 *>(dout + 16ll * c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = make_uint4(0, 0, 0, 0);
          if (row[j] >= 0) v[j] = load16<ONCE>(p.x + row[j] * p.ldx + 16ll * c);
        }
        float d[V];
        unpack16<BF16>(dv, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (row[j] < 0) continue;
          float f[V], g[V];
          unpack16<BF16>(v[j], f);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            dot[j] = fmaf(d[i], f[i], dot[j]);
            g[i] = w[j] * d[i];
          }
          *reinterpret_cast<uint4 *>(p.out + row[j] * p.ldo + 16ll * c) = pack16<BF16>(g);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) dot[j] = wave_sum(dot[j]);
      if constexpr (LANES == 64) {
        float mine = dot[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) mine = lane == static_cast<uint32_t>(j) ? dot[j] : mine;
        if (lane < 8 && j0 + static_cast<int>(lane) < p.k) p.dweights[t * p.k + j0 + lane] = mine;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (lane == 0) part[wave][j] = dot[j];
        __syncthreads();
        if (threadIdx.x < 8 && j0 + static_cast<int>(threadIdx.x) < p.k)
          p.dweights[t * p.k + j0 + threadIdx.x] =
              (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
        __syncthreads();
      }
    }
    // rows that no slot has: these lanes look after rows [t k, (t + 1) k)
    for (int j = 0; j < p.k; ++j) {
      const int64_t r = t * p.k + j;
      if (p.rows[r] < 0)
        for (int c = first; c < p.pieces; c += LANES)
          *reinterpret_cast<uint4 *>(p.out + r * p.ldo + 16ll * c) = make_uint4(0, 0, 0, 0);
    }
  }
}

RowsArgs rows_args(const MoeRowsArgs &a) {
  const int es = a.dtype == 1 ? 2 : 4;
  RowsArgs p{};
  p.x = static_cast<const uint8_t *>(a.x);
  p.ldx = a.ldx * es;
  p.dout = static_cast<const uint8_t *>(a.dout);
  p.ld_dout = a.ld_dout * es;
  p.tokens = a.tokens;
  p.pieces = static_cast<int>(a.d * es / 16);
  while (p.lane_bits < 8 && (1 << p.lane_bits) < p.pieces) ++p.lane_bits;
  p.pos = a.pos;
  p.rows = a.rows;
  p.weights = a.weights;
  p.k = a.top_k;
  p.out = static_cast<uint8_t *>(a.out);
  p.ldo = a.ldo * es;
  p.dweights = a.dweights;
  return p;
}

// Whether the experts' rows are too many for the cache.  4096 tokens of 8 rows of 4096: the sum bf16 59 -> 55 us, fp32
// 119 -> 105, its gradient bf16 122 -> 101, fp32 252 -> 250 (non-temporal stores of dy besides: 110 and 235).
bool rows_once(const MoeRowsArgs &a) {
  return a.tokens * a.top_k * a.d * (a.dtype == 1 ? 2 : 4) >= kStreamBytes;
}

// A workgroup for every 256 columns and `rows` rows.
dim3 grid_of(const RowsArgs &p, int64_t rows, int rows_a_group) {
  const int64_t groups = (rows + rows_a_group - 1) / rows_a_group;
  return dim3((p.pieces + kRowThreads - 1) / kRowThreads, static_cast<uint32_t>(groups < kMaxBlocks ? groups : kMaxBlocks));
}

// A wave a token up to 128 pieces, without barriers (16384 x 8 x 512 bf16 97 -> 55 us, 5.2 TB/s); at 512 pieces a workgroup
// is faster (100 us against 109).
template <bool BF16, bool ONCE>
hipError_t run_backward(const RowsArgs &p, hipStream_t stream) {
  const int64_t groups = p.pieces <= 128 ? (p.tokens + 3) / 4 : p.tokens;
  const dim3 grid(static_cast<uint32_t>(groups < (1 << 20) ? groups : 1 << 20));
  if (p.pieces <= 128)
    combine_backward_kernel<BF16, ONCE, 64><<<grid, dim3(kRowThreads), 0, stream>>>(p);
  else
    combine_backward_kernel<BF16, ONCE, 256><<<grid, dim3(kRowThreads), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_gather(const MoeRowsArgs &a) {
  const RowsArgs p = rows_args(a);
  auto *kernel = rows_once(a) ? gather_kernel<true> : gather_kernel<false>;
  kernel<<<grid_of(p, a.tokens * a.top_k, (kRowThreads >> p.lane_bits) * kGatherRows), dim3(kRowThreads), 0, a.stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeRowsArgs &a) {
  const RowsArgs p = rows_args(a);
  const bool once = rows_once(a);
  auto *kernel = a.dtype == 1 ? (once ? combine_kernel<true, true> : combine_kernel<true, false>)
                              : (once ? combine_kernel<false, true> : combine_kernel<false, false>);
  kernel<<<grid_of(p, a.tokens, kRowThreads >> p.lane_bits), dim3(kRowThreads), 0, a.stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const MoeRowsArgs &a) {
  const RowsArgs p = rows_args(a);
  if (rows_once(a)) return a.dtype == 1 ? run_backward<true, true>(p, a.stream) : run_backward<false, true>(p, a.stream);
  return a.dtype == 1 ? run_backward<true, false>(p, a.stream) : run_backward<false, false>(p, a.stream);
}

}  // namespace nvfp4
