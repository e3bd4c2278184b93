// adapter.hip -- low-rank adapters of many requests (or experts) at once, beside a shared projection:
//   h_r = A_g x_r,   c_r = base_r + s_g B_g h_r     (g: the adapter of row r)
// and the gradients of x, A and B.  A [R x K] and B [N x R] of an adapter are bf16, R at most 128: all products run on
// the bf16 matrix cores (v_mfma_f32_16x16x32_bf16: lane l holds row l & 15, elements 8 (l >> 4) .. + 7 of either operand,
// and column l & 15, rows 4 (l >> 4) .. + 3 of the result).
//
// The long sums (h over K, dA and dB over the rows) stay in fp32.  Where h or its gradient g is an operand again, it is
// taken as a sum of bf16 numbers, v = v0 + v1 (+ v2), each the rounding of what the ones before leave: to 2^-16 of it for a
// bf16 result, whose own rounding is 2^-8, and to 2^-24, all that fp32 has, for fp32 results (with two pieces their error
// was 1.2e-6 of the result, with three it is the sums' own 1e-7).  Such rows are kept as [M][3 R] bf16.
//
// Rows.  A plan's offsets live on the device: the launch has as many workgroups as any offsets could need (a partial
// tile more for every adapter), and each finds its tile by a scan over the adapters' tile counts.
//
// What bounds it.  Ranks are small, so the rows of x, base, c and dc are nearly all of the bytes, and the products (two to
// six R operations a byte) run under their loads up to a rank of 64.  8192 x 4096 x 14336 of rank 16, bf16: h 17.6 to
// 21 us (67 MB), c 84 to 87 us (470 MB, 5.4 to 5.6 TB/s; a 1 GiB copy runs at 5.1 to 5.2, an elementwise pass over as much at
// 6.2); gradients 153 us (dc read once 81, dx 30, x 20, the rest small).  Whole calls against the bytes at 6.2 TB/s: forward
// 118 us (87), step 248 (157).
#include "gemm_common.hpp"
#include "nvfp4_internal.h"
#include "vec_io.hpp"

namespace nvfp4 {
namespace {

using namespace gemm;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));

// Where rows come from and go to (see MoEPlan): row r of the plan's order is row x_row(r) of x and row c_row(r) of c.
struct Rows {
  const int32_t *offsets;  // NULL: one adapter for all M rows
  const int32_t *rows;     // NULL: row r itself
  int32_t groups;
  int32_t x_div;           // 0: x has rows in the plan's order; else x row = rows[r] / x_div
  int32_t x_shift;         // of a power of two x_div, else -1 (a division takes some thirty instructions)
  int32_t by_rows;         // c row = rows[r]
  int64_t M, x_rows;
};

// What rows or columns that do not exist read.
__device__ const uint4 kZeros = {0u, 0u, 0u, 0u};

__device__ __forceinline__ int64_t x_row(const Rows &p, int64_t r) {
  if (p.x_div == 0) return r;
  const int32_t slot = p.rows[r];
  const int64_t s = p.x_shift >= 0 ? slot >> p.x_shift : slot / p.x_div;
  return slot >= 0 && s < p.x_rows ? s : -1;
}
__device__ __forceinline__ int64_t c_row(const Rows &p, int64_t r) {
  if (!p.by_rows) return r;
  const int64_t s = p.rows[r];
  return s >= 0 && s < p.M ? s : -1;
}

// Tile `tm` of `size` rows among all adapters' tiles: its adapter and rows [m0, m_end), and how many tiles the adapter
// has.  False beyond the last.  Every lane of the wave takes part and has the result.
struct Tile {
  int32_t group, tiles;
  int64_t m0, m_end;
};
__device__ __forceinline__ bool find_tile(const Rows &p, int32_t size, int32_t tm, Tile &t) {
  if (!p.offsets) {
    t.group = 0;
    t.tiles = static_cast<int32_t>((p.M + size - 1) / size);
    t.m0 = static_cast<int64_t>(tm) * size;
    t.m_end = min(t.m0 + size, p.M);
    return t.m0 < p.M;
  }
  const int lane = threadIdx.x & 63;
  int32_t before = 0;
  for (int g0 = 0; g0 < p.groups; g0 += 64) {
    const int g = g0 + lane;
    const int32_t lo = g < p.groups ? p.offsets[g] : 0, hi = g < p.groups ? p.offsets[g + 1] : 0;
    const int32_t n = hi > lo ? (hi - lo - 1) / size + 1 : 0;
    int32_t s = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int32_t o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    const uint64_t past = __ballot(before + s > tm);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int32_t first = __builtin_amdgcn_readfirstlane(before + __shfl(s - n, at));
      const int32_t m_lo = __builtin_amdgcn_readfirstlane(__shfl(lo, at)), m_hi = __builtin_amdgcn_readfirstlane(__shfl(hi, at));
      t.group = g0 + at;
      t.tiles = __builtin_amdgcn_readfirstlane(__shfl(n, at));
      t.m0 = m_lo + static_cast<int64_t>(tm - first) * size;
      t.m_end = min(min(t.m0 + size, static_cast<int64_t>(m_hi)), p.M);
      return t.m0 >= 0 && t.m0 < t.m_end;
    }
    before += __builtin_amdgcn_readfirstlane(__shfl(s, 63));
  }
  return false;
}

__device__ __forceinline__ bf16x8 frag(const void *p) { return __builtin_bit_cast(bf16x8, *static_cast<const uint4 *>(p)); }
__device__ __forceinline__ floatx4 mfma(const bf16x8 &a, const bf16x8 &b, const floatx4 &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Eight values as PARTS bf16 pieces each of which takes what the ones before leave.  An infinity is its first piece alone
// (what it leaves would be NaN), and the first piece of a finite value that would round to one is the largest bf16 number.
constexpr float kBf16Max = 0x1.FEp127f;
template <int PARTS>
__device__ __forceinline__ void split8(float (&v)[8], uint4 (&out)[PARTS]) {
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
  const bool over = top > kBf16Max;
#pragma unroll
  for (int s = 0; s < PARTS; ++s) {
    float piece[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) piece[e] = v[e];
    if (s == 0 && over) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (fabsf(v[e]) > kBf16Max && !isinf(v[e])) piece[e] = copysignf(kBf16Max, v[e]);
    }
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      w[q] = pack_bf16(piece[2 * q], piece[2 * q + 1]);
      v[2 * q] -= __uint_as_float(w[q] << 16);
      v[2 * q + 1] -= __uint_as_float(w[q] & 0xFFFF0000u);
    }
    if (s == 0 && over) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (isinf(piece[e])) v[e] = 0.0f;
    }
    out[s] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Four rows of 16 columns (bf16, LDS), transposed: lane l16 of a group of 16 gives the address of elements 4 (l16 & 3) .. + 3
// of row l16 >> 2 and gets column l16 of the four rows.  Two of them are a fragment.
__device__ __forceinline__ short4v tr(const uint8_t *at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4v *)(at));
}
__device__ __forceinline__ bf16x8 pair(const short4v &lo, const short4v &hi) {
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// ---- rows x factor: part[split][r][q] = sum over the split's k of y[row(r)][k] f[g][q][k] --------------------
struct ShrinkArgs {
  Rows rows;
  const uint8_t *y;
  int64_t ldy;           // bytes
  const uint8_t *f;      // [groups][R][K] bf16
  int64_t K;
  int32_t R;
  int32_t splits, split_k;  // elements of K a split, a multiple of the step
  float *part;           // [splits][M][R]
};

// Few rows an adapter: a workgroup has 16 rows and kFewK elements of K, a wave an eighth of these, all its loads in
// flight at once; the waves' sums meet in LDS.  Latency: 48 rows of 4096, each with an adapter of rank 16, 5.2 us (6.7 MB);
// 37 rows of 14336 and 16 adapters of rank 64 8.7 us (30 MB).
constexpr int kFewWaveK = 128, kFewWaves = 8, kFewK = kFewWaves * kFewWaveK;
template <int RF>
__global__ __launch_bounds__(64 * kFewWaves) void shrink_few_kernel(ShrinkArgs p) {
  __shared__ floatx4 sums[kFewWaves][RF][64];
  const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, j = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t tm = blockIdx.x / p.splits, split = blockIdx.x - tm * p.splits;
  Tile t;
  if (!find_tile(p.rows, 16, tm, t)) return;
  const int64_t k0 = static_cast<int64_t>(split) * kFewK + wave * kFewWaveK + 8 * j;
  const uint8_t *f = p.f + (static_cast<int64_t>(t.group) * p.R * p.K + k0) * 2;
  uint4 a[RF][4], b[4];
#pragma unroll
  for (int u = 0; u < RF; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[u][i] = make_uint4(0, 0, 0, 0);
      const int q = 16 * u + l16;
      if (q < p.R && k0 + 32 * i < p.K) a[u][i] = *reinterpret_cast<const uint4 *>(f + (q * p.K + 32 * i) * 2);
    }
  const int64_t r = t.m0 + l16, y = r < t.m_end ? x_row(p.rows, r) : -1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    b[i] = make_uint4(0, 0, 0, 0);
    if (y >= 0 && k0 + 32 * i < p.K) b[i] = *reinterpret_cast<const uint4 *>(p.y + y * p.ldy + (k0 + 32 * i) * 2);
  }
  floatx4 acc[RF];
#pragma unroll
  for (int u = 0; u < RF; ++u) acc[u] = (floatx4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < RF; ++u) acc[u] = mfma(__builtin_bit_cast(bf16x8, a[u][i]), __builtin_bit_cast(bf16x8, b[i]), acc[u]);
#pragma unroll
  for (int u = 0; u < RF; ++u) sums[wave][u][lane] = acc[u];
  __syncthreads();
  for (int u = wave; u < RF; u += kFewWaves) {
    floatx4 v = sums[0][u][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += sums[w][u][lane];
    const int q = 16 * u + 4 * j;
    if (r < t.m_end && q < p.R)
      *reinterpret_cast<floatx4 *>(p.part + (static_cast<int64_t>(split) * p.rows.M + r) * p.R + q) = v;
  }
}

// Many rows: a workgroup has 64 rows (a wave 16) and walks its split of K 64 elements (128 bytes of a row) a step through
// a ring of LDS stages filled by direct loads.  16-byte chunk c of row r sits at c ^ ((r >> 1) & 7): the reads of a
// fragment then cover all banks.  Two, three and four stages leave eight, five and four workgroups a compute unit at rank 16:
// 32768 gathered rows of 4096 take 32.2, 33.6 and 35.5 us, 8192 rows 22.3, 21.3 and 21.3, 2047 of 14336 at rank 64 27.4,
// 26.1 and 25.7.  The gathered rows (268 MB from the L2, 72% hits) take vector instructions for half of that time.
constexpr int kManyRows = 64, kManyStep = 64, kManyStages = 3;
__device__ __forceinline__ uint32_t swz(uint32_t r) { return (r >> 1) & 7u; }
template <int RF>
__global__ __launch_bounds__(256) void shrink_many_kernel(ShrinkArgs p) {
  constexpr int kF = kManyRows * 128, kStage = kF + RF * 16 * 128;
  constexpr int NF = (2 * RF + 3) / 4;  // loads of the factor a wave and step, eight rows each
  constexpr bool all = 2 * RF >= 4;     // (of a rank of 16 there are two, and two waves have one)
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kManyStages * kStage];
  const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, j = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t tm = blockIdx.x / p.splits, split = blockIdx.x - tm * p.splits;
  Tile t;
  if (!find_tile(p.rows, kManyRows, tm, t)) return;
  const uint8_t *const zeros = reinterpret_cast<const uint8_t *>(&kZeros);
  const int64_t k_lo = static_cast<int64_t>(split) * p.split_k, k_hi = min(k_lo + p.split_k, p.K);
  const int32_t steps = static_cast<int32_t>((k_hi - k_lo + kManyStep - 1) / kManyStep);
  // where the lane's next piece of each load lies, and what a step adds: rows that do not exist stay at the zeros
  const uint8_t *srcY[2], *srcF[NF];
  uint32_t stepY[2], stepF[NF], chunkY[2], chunkF[NF];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t R = 16 * wave + 8 * i + (lane >> 3);
    chunkY[i] = ((lane & 7u) ^ swz(R)) * 8;
    const int64_t r = t.m0 + R, y = r < t.m_end ? x_row(p.rows, r) : -1;
    srcY[i] = y >= 0 ? p.y + y * p.ldy + (k_lo + chunkY[i]) * 2 : zeros;
    stepY[i] = y >= 0 ? 2 * kManyStep : 0;
  }
#pragma unroll
  for (int i = 0; i < NF; ++i) {
    const uint32_t R = 8 * (wave + 4 * i) + (lane >> 3);
    chunkF[i] = ((lane & 7u) ^ swz(R)) * 8;
    const bool real = R < static_cast<uint32_t>(p.R);
    srcF[i] = real ? p.f + ((static_cast<int64_t>(t.group) * p.R + R) * p.K + k_lo + chunkF[i]) * 2 : zeros;
    stepF[i] = real ? 2 * kManyStep : 0;
  }
  // loads of steps 0, 1, ... in turn; from the last on, whatever lies beyond the split reads zeros
  const int32_t whole = static_cast<int32_t>((k_hi - k_lo) / kManyStep);
  auto load = [&](int32_t kt) {
    uint8_t *st = smem + (kt % kManyStages) * kStage;
    const int64_t left = k_hi - k_lo - static_cast<int64_t>(kt) * kManyStep;
    const bool cut = kt >= whole;  // (the same in every lane)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lds_load16(cut && static_cast<int64_t>(chunkY[i]) >= left ? zeros : srcY[i], st + (16 * wave + 8 * i) * 128);
      srcY[i] += stepY[i];
    }
    if (!all && wave >= 2) return;
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      lds_load16(cut && static_cast<int64_t>(chunkF[i]) >= left ? zeros : srcF[i], st + kF + 8 * (wave + 4 * i) * 128);
      srcF[i] += stepF[i];
    }
  };
  constexpr int LPS = 2 + NF;
#pragma unroll
  for (int s = 0; s < kManyStages - 1; ++s) load(s);
  floatx4 acc[RF];
#pragma unroll
  for (int u = 0; u < RF; ++u) acc[u] = (floatx4){0.0f, 0.0f, 0.0f, 0.0f};
  for (int32_t kt = 0; kt < steps; ++kt) {
    if (!all && wave >= 2)
      wait_vmcnt<(kManyStages - 2) * 2>();
    else
      wait_vmcnt<(kManyStages - 2) * LPS>();
    wait_lgkmcnt0();  // (this wave's reads of the stage that is filled next)
    lds_barrier();
    load(kt + kManyStages - 1);  // (beyond the last step: zeros, into a stage that nobody reads)
    const uint8_t *st = smem + (kt % kManyStages) * kStage;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t R = 16 * wave + l16;
      const bf16x8 b = frag(st + R * 128 + ((4 * s + j) ^ swz(R)) * 16);
#pragma unroll
      for (int u = 0; u < RF; ++u) {
        const uint32_t Q = 16 * u + l16;
        acc[u] = mfma(frag(st + kF + Q * 128 + ((4 * s + j) ^ swz(Q)) * 16), b, acc[u]);
      }
    }
  }
  wait_vmcnt<0>();
  const int64_t r = t.m0 + 16 * wave + l16;
#pragma unroll
  for (int u = 0; u < RF; ++u) {
    const int q = 16 * u + 4 * j;
    if (r < t.m_end && q < p.R)
      *reinterpret_cast<floatx4 *>(p.part + (static_cast<int64_t>(split) * p.rows.M + r) * p.R + q) = acc[u];
  }
}

// ---- sums of the splits -----------------------------------------------------------------------------------------
// Eight columns of row r.
__device__ __forceinline__ void sum_splits(const float *part, int64_t M, int32_t R, int32_t splits, int64_t r, int32_t q,
                                           float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const floatx4 *at = reinterpret_cast<const floatx4 *>(part + (s * M + r) * R + q);
    const floatx4 lo = at[0], hi = at[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] += lo[i];
      v[4 + i] += hi[i];
    }
  }
}
__device__ __forceinline__ void store_h(float *h, int32_t R, int64_t r, int32_t q, const float (&v)[8]) {
  floatx4 *at = reinterpret_cast<floatx4 *>(h + r * R + q);
  at[0] = (floatx4){v[0], v[1], v[2], v[3]};
  at[1] = (floatx4){v[4], v[5], v[6], v[7]};
}
// part[0] = the splits' sum, four values a thread.
__global__ __launch_bounds__(256) void split_sum_kernel(float *part, int64_t size, int32_t splits) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= size) return;
  floatx4 v = *reinterpret_cast<const floatx4 *>(part + i);
#pragma unroll 8
  for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const floatx4 *>(part + s * size + i);
  *reinterpret_cast<floatx4 *>(part + i) = v;
}
// ---- rows + pieces x factor: c[row(r)][n] = base[row(r)][n] + sum_q piece[r][q] f[g][n][q] --------------------
struct ExpandArgs {
  Rows rows;
  const int32_t *pos;     // by_rows: the row of each token (-1: none)
  const uint8_t *f;       // [groups][N][R] bf16
  int64_t N;
  int32_t R;
  const float *part;      // [splits][M][R]
  int32_t splits;
  const uint8_t *x;       // OWN: as ShrinkArgs' y, f and K
  int64_t ldx;            // bytes
  const uint8_t *a;
  int64_t K;
  const float *scales;
  float *h;               // nullable [M][R]: the splits' sums
  uint8_t *pieces;        // nullable [M][3 R] bf16: of scale * sum
  const uint8_t *base;    // NULL: zeros
  int64_t ldb;            // bytes
  uint8_t *c;
  int64_t ldc;            // bytes
  int32_t columns;        // of a workgroup, a multiple of 256
  int32_t tiles_n, tiles_m;  // a launch has tiles_n * (tiles_m + copy tiles) workgroups
};

template <bool BF16>
__device__ __forceinline__ float element(const uint8_t *p, int64_t i) {
  return BF16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i]) << 16)
              : reinterpret_cast<const float *>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void set_element(uint8_t *p, int64_t i, float v) {
  if constexpr (BF16)
    reinterpret_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(pack_bf16(v, 0.0f));
  else
    reinterpret_cast<float *>(p)[i] = v;
}

// How a wave meets rows of c, 64 columns (128 or 256 bytes) of each at a time: an instruction moves whole segments of
// kRows rows, lane l the piece l % kPieces of row l / kPieces.  (Rows of 8192 x 14336 bf16 added to in 128-byte segments
// run at 6.4 to 6.6 TB/s with non-temporal loads, in 64-byte ones, as the products' registers hold them, at 4.8.)
template <bool BF16>
struct Segment {
  static constexpr int ES = BF16 ? 2 : 4, kValues = 16 / ES, kPieces = 64 / kValues, kRows = 64 / kPieces;
};

// A piece of a row of base or c; rows whose pieces lie at any element unless VEC.
template <bool ONCE, bool VEC>
__device__ __forceinline__ uint4 load_piece(const uint8_t *at) {
  if constexpr (VEC) return load16<ONCE>(at);
  const any_u32x4 v = *reinterpret_cast<const any_u32x4 *>(at);
  return make_uint4(v.x, v.y, v.z, v.w);
}
template <bool VEC>
__device__ __forceinline__ void store_piece(uint8_t *at, const uint4 &v) {
  if constexpr (VEC)
    *reinterpret_cast<uint4 *>(at) = v;
  else
    *reinterpret_cast<any_u32x4 *>(at) = (any_u32x4){v.x, v.y, v.z, v.w};
}

// Rows without an adapter: c = base (or zeros), 64 rows of a workgroup's columns.
template <bool BF16, bool ONCE, bool VEC>
__device__ void copy_rows(const ExpandArgs &p, int32_t tile, int64_t n0) {
  using S = Segment<BF16>;
  constexpr int ES = S::ES, NI = 64 / S::kRows;
  const int32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n1 = min(n0 + p.columns, p.N);
  const int64_t mine = static_cast<int64_t>(tile) * 64 + lane;
  const bool bare = mine < p.rows.M && (p.rows.by_rows ? p.pos[mine] < 0 : mine >= p.rows.offsets[p.rows.groups]);
  const uint64_t rows = __ballot(bare);
  if (rows == 0) return;
  const int32_t first = lane / S::kPieces, col = lane % S::kPieces * S::kValues;
  for (int64_t n = n0 + 64 * wave + col; n < n1; n += 256) {
    if (n + S::kValues <= p.N) {
#pragma clang loop unroll(disable)
      for (int i0 = 0; i0 < NI; i0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int32_t r = S::kRows * (i0 + i) + first;
          v[i] = make_uint4(0, 0, 0, 0);
          const int64_t row = static_cast<int64_t>(tile) * 64 + r;
          if (p.base && (rows >> r & 1)) v[i] = load_piece<ONCE, VEC>(p.base + row * p.ldb + n * ES);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int32_t r = S::kRows * (i0 + i) + first;
          if (rows >> r & 1) store_piece<VEC>(p.c + (static_cast<int64_t>(tile) * 64 + r) * p.ldc + n * ES, v[i]);
        }
      }
    } else if constexpr (!VEC) {
#pragma clang loop unroll(disable)
      for (int i = 0; i < NI; ++i) {
        const int32_t r = S::kRows * i + first;
        const int64_t row = static_cast<int64_t>(tile) * 64 + r;
        if (rows >> r & 1)
          for (int64_t e = n; e < p.N; ++e)
            set_element<BF16>(p.c + row * p.ldc, e, p.base ? element<BF16>(p.base + row * p.ldb, e) : 0.0f);
      }
    }
  }
}

// A workgroup has 16 TF rows and walks its columns 256 at a time, a wave 64 of these in four fragments of the factor's
// rows.  The rows' pieces are formed once, in LDS, from the splits' sums: part s of eight columns rc of a row is its chunk
// s RCP + rc, RCP the power of two that holds R / 8, and NM products of 32 cover a row.  As RCP is a power of two, these take UF
// different fragments of the factor, again and again for each part.  Sums leave through the wave's own LDS, 16 rows at a time, in
// whole segments (see Segment).
// OWN (16 rows): there are no splits; each workgroup forms its rows' h itself, a wave a quarter of K.  One row of 4096 x 14336,
// rank 16: 9.6 us and 13.4 to 13.8 from Python, where two launches take 4.0 + 4.5 us and 17.2.
// HBM-bound for many rows: see the top of the file for rank 16; 2047 x 14336 of rank 64 33 us (117 MB).  48 rows of 14336 with 48
// adapters 8.8 us (25 MB).
template <int RCP, int TF, bool BF16, bool ONCE, bool VEC, bool OWN>
__global__ __launch_bounds__(256, OWN || RCP > 8 ? 2 : VEC || TF == 1 ? 4 : 3) void expand_kernel(ExpandArgs p) {
  using S = Segment<BF16>;
  constexpr int ES = S::ES, PARTS = BF16 ? 2 : 3, NI = 16 * TF / S::kRows;
  constexpr int NM = (PARTS * RCP + 3) / 4, UF = RCP <= 4 ? 1 : RCP / 4;
  constexpr int kPitch = NM * 64 + 16;  // of a row of pieces in LDS (with the pad, rows start in different banks)
  __shared__ __attribute__((aligned(16))) uint8_t staged[16 * TF * kPitch];
  __shared__ floatx4 turned[4][16 * 16];
  __shared__ int32_t c_rows[16 * TF];  // -1: none
  constexpr int RF = OWN ? (RCP + 1) / 2 : 1;
  __shared__ floatx4 own[OWN ? 4 * 16 * 4 * RF : 1];  // [wave][row][16 RF values]
  const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, j = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t tm = blockIdx.x / p.tiles_n, tn = blockIdx.x - tm * p.tiles_n;
  const int64_t n_lo = static_cast<int64_t>(tn) * p.columns, n_hi = min(n_lo + p.columns, p.N);
  if (tm >= p.tiles_m) return copy_rows<BF16, ONCE, VEC>(p, tm - p.tiles_m, n_lo);
  Tile t;
  if (!find_tile(p.rows, 16 * TF, tm, t)) return;
  const int32_t RC = p.R / 8;
  if (threadIdx.x < 16 * TF) {
    const int64_t r = t.m0 + threadIdx.x;
    c_rows[threadIdx.x] = static_cast<int32_t>(r < t.m_end ? c_row(p.rows, r) : -1);
  }
  const uint32_t first = lane / S::kPieces, col = lane % S::kPieces * S::kValues;
  uint4 f[4][UF], b[NI];
  auto load = [&](int64_t n0) {
    const int64_t n = n0 + col;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t row = c_rows[S::kRows * i + first];
      b[i] = make_uint4(0, 0, 0, 0);
      if (p.base && row >= 0 && n + S::kValues <= p.N) b[i] = load_piece<ONCE, VEC>(p.base + row * p.ldb + n * ES);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint8_t *from = p.f + (static_cast<int64_t>(t.group) * p.N + min(n0 + 16 * u + l16, p.N - 1)) * p.R * 2;
#pragma unroll
      for (int i = 0; i < UF; ++i) {
        const int32_t rc = (4 * i + j) % RCP;
        f[u][i] = make_uint4(0, 0, 0, 0);
        if (rc < RC) f[u][i] = *reinterpret_cast<const uint4 *>(from + rc * 16);
      }
    }
  };
  const float scale = p.scales[t.group];
  __syncthreads();  // c_rows
  int64_t n0 = n_lo + 64 * wave;
  if (TF == 1 && n0 < n_hi) load(n0);
  if constexpr (OWN) {
    const int64_t r = t.m0 + l16, y = r < t.m_end ? x_row(p.rows, r) : -1;
    const uint8_t *a = p.a + static_cast<int64_t>(t.group) * p.R * p.K * 2;
    floatx4 acc[RF];
#pragma unroll
    for (int u = 0; u < RF; ++u) acc[u] = (floatx4){0.0f, 0.0f, 0.0f, 0.0f};
    // kBatch steps' loads in flight at once (steps are the same for every lane: matrix instructions want all)
    constexpr int kBatch = 16 / RF;
    const uint8_t *const zeros = reinterpret_cast<const uint8_t *>(&kZeros), *const x = p.x + (y >= 0 ? y : 0) * p.ldx;
    for (int64_t k0 = 32 * wave; k0 < p.K; k0 += 128 * kBatch) {
      uint4 v[kBatch], w[RF][kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t k = k0 + 128 * i + 8 * j;
        v[i] = *reinterpret_cast<const uint4 *>(y >= 0 && k < p.K ? x + k * 2 : zeros);
#pragma unroll
        for (int u = 0; u < RF; ++u)
          w[u][i] = *reinterpret_cast<const uint4 *>(
              16 * u + static_cast<int>(l16) < p.R && k < p.K ? a + ((16 * u + l16) * p.K + k) * 2 : zeros);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int u = 0; u < RF; ++u) acc[u] = mfma(__builtin_bit_cast(bf16x8, w[u][i]), __builtin_bit_cast(bf16x8, v[i]), acc[u]);
    }
#pragma unroll
    for (int u = 0; u < RF; ++u) own[((wave * 16 + l16) * RF + u) * 4 + j] = acc[u];
    __syncthreads();
  }
  for (int i = threadIdx.x; i < 16 * TF * RCP; i += 256) {
    const int32_t m = i / RCP, rc = i % RCP;
    const int64_t r = t.m0 + m;
    const bool real = r < t.m_end && rc < RC;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    if (real) {
      if constexpr (OWN) {
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += own[(w * 16 + m) * RF * 4 + 2 * rc + e / 4][e % 4];
      } else {
        sum_splits(p.part, p.rows.M, p.R, p.splits, r, 8 * rc, v);
      }
      if (p.h && tn == 0) store_h(p.h, p.R, r, 8 * rc, v);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= scale;
    uint4 w[3];
    split8(v, w);
#pragma unroll
    for (int s = 0; s < PARTS; ++s) *reinterpret_cast<uint4 *>(staged + m * kPitch + (s * RCP + rc) * 16) = w[s];
    if (p.pieces && tn == 0 && real) {
      uint4 *out = reinterpret_cast<uint4 *>(p.pieces + r * (6 * p.R)) + rc;
      out[0] = w[0];
      out[RC] = w[1];
      out[2 * RC] = w[2];
    }
  }
  __syncthreads();

  floatx4 *const mine = turned[wave];
  for (; n0 < n_hi; n0 += 256) {
    const int64_t n = n0 + col;
    if (TF > 1) load(n0);
#pragma unroll
    for (int tf = 0; tf < TF; ++tf) {
      if constexpr (RCP >= 4) asm volatile("" ::: "memory");  // (16 rows at a time: all rows' pieces in registers would spill)
      bf16x8 x[NM];
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (PARTS * RCP == 4 * NM || 4 * i + static_cast<int32_t>(j) < PARTS * RCP)
          v = *reinterpret_cast<const uint4 *>(staged + (16 * tf + l16) * kPitch + (4 * i + j) * 16);
        x[i] = __builtin_bit_cast(bf16x8, v);
      }
      // column 16 u + 4 j of row l16 on: chunk 4 u + j of the row, at (4 u + j) ^ row
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NM; ++i) acc = mfma(__builtin_bit_cast(bf16x8, f[u][i % UF]), x[i], acc);
        mine[16 * l16 + ((4 * u + j) ^ l16)] = acc;
      }
      // the wave reads back its own rows (LDS accesses of one wave complete in order)
#pragma unroll
      for (int k = 0; k < 16 / S::kRows; ++k) {
        const int i = tf * (16 / S::kRows) + k;
        const uint32_t m = S::kRows * k + first;
        const int64_t row = c_rows[16 * tf + m];
        float v[S::kValues];
#pragma unroll
        for (int q = 0; q < S::kValues / 4; ++q) {
          const floatx4 four = mine[16 * m + ((col / 4 + q) ^ m)];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * q + e] = four[e];
        }
        if (row >= 0 && n + S::kValues <= p.N) {
          uint32_t w[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (BF16)
              w[e] = pack_bf16(__uint_as_float(w[e] << 16) + v[2 * e], __uint_as_float(w[e] & 0xFFFF0000u) + v[2 * e + 1]);
            else
              w[e] = __float_as_uint(__uint_as_float(w[e]) + v[e]);
          }
          store_piece<VEC>(p.c + row * p.ldc + n * ES, make_uint4(w[0], w[1], w[2], w[3]));
        } else if (!VEC && row >= 0) {
          // the last columns of a row (a loop, to keep this path's code short)
#pragma clang loop unroll(disable)
          for (int e = 0; e < S::kValues && n + e < p.N; ++e) {
            const float was = p.base ? element<BF16>(p.base + row * p.ldb, n + e) : 0.0f;
            float d = v[0];
#pragma unroll
            for (int q = 1; q < S::kValues; ++q) d = e == q ? v[q] : d;
            set_element<BF16>(p.c + row * p.ldc, n + e, was + d);
          }
        }
      }
    }
    if (TF == 1 && n0 + 256 < n_hi) load(n0 + 256);
  }
}

// ---- the factors' gradients: out[g][q][n] or out[g][n][q] = sum_r piece[r][q] y[row(r)][n] -----------------------
// and with a factor f in the same pass over y:  g_part[column tile][r][q] = sum over the tile's n of y[row(r)][n] f[g][n][q]
struct OuterArgs {
  Rows rows;
  const uint8_t *y;
  int64_t ldy;            // bytes
  int64_t N;              // a multiple of 8
  int32_t R;
  const uint8_t *pieces;  // [M][3 R] bf16
  bool n_major;           // out is [N][R], not [R][N]
  int32_t chunk;          // rows of a workgroup, a multiple of 32
  int32_t tiles_n;
  float *part;            // [chunks][N R]
  float *out;             // [groups][N R]
  const uint8_t *f;       // [groups][N][R] bf16
  float *g_part;          // [tiles_n][M][R]
};

// A workgroup of eight waves has `chunk` rows of one adapter and 256 columns of y, a wave 32 of these; 32 rows a step through a
// ring in LDS.  Both operands lie with their rows (the contraction) outermost: fragments come from ds_read_b64_tr_b16, which
// gives a lane four rows of one column.  32-byte unit u of row t of y sits at u ^ ((t & 3) | (t >> 1) & 4): the sixteen rows
// that one read touches lie in different banks.
// The second product contracts over columns: f's fragments (again by transposed reads, from LDS before the rows' loop)
// stay in registers, and each step the waves share out rows 0 to 15 and 16 to 31 with each fragment of f (of a rank of 16
// there is one, and two waves take it).  Reading dc once for both costs 82 us where two passes took 130 (8192 x 14336, rank 16:
// 235 MB, and 58 MB of g's parts written and read again); what of c the launch before left in the cache is written back
// meanwhile.  x, 8192 x 4096: 20 us (3.4 TB/s).  From rank 64 on LDS reads and matrix instructions count: 2047 x 14336 28 us.
constexpr int kOuterStep = 32, kMaxChunk = 960, kOuterThreads = 512;
// The ring's stages: two workgroups a compute unit share its 160 KB of LDS up to a rank of 64, above it one has them.
template <int RF>
constexpr int kOuterStages = RF == 1 ? 4 : RF == 4 ? 2 : 3;
template <int RF, bool G>
__global__ __launch_bounds__(kOuterThreads, RF <= 4 ? 4 : 2) void outer_kernel(OuterArgs p) {
  constexpr int S = kOuterStages<RF>;
  constexpr int kY = kOuterStep * 512, kStage = kY + kOuterStep * 96 * RF;
  // loads of pieces a step: 3 RF of 1 KB (R = 16 RF at most), NP for every wave and one more for the first `rest` waves
  constexpr int NP = 3 * RF / 8;
  constexpr uint32_t rest = 3 * RF % 8;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * kStage + 64];
  __shared__ int32_t y_rows[kMaxChunk];  // the chunk's rows of y; -1 beyond the last
  const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, j = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t tm = blockIdx.x / p.tiles_n, tn = blockIdx.x - tm * p.tiles_n;
  Tile t;
  if (!find_tile(p.rows, p.chunk, tm, t)) return;
  const uint8_t *const zeros = reinterpret_cast<const uint8_t *>(&kZeros);
  const int64_t n_wg = static_cast<int64_t>(tn) * 256;
  for (int i = threadIdx.x; i < p.chunk; i += kOuterThreads) {
    const int64_t r = t.m0 + i;
    y_rows[i] = static_cast<int32_t>(r < t.m_end ? x_row(p.rows, r) : -1);
  }
  constexpr int GF = G ? (RF + 3) / 4 : 1;  // fragments of f a wave
  bf16x8 f[GF][8];
  if constexpr (G) {
    static_assert(256 * 32 * RF <= S * kStage, "f fits the ring");
    const int32_t fp = p.R * 2, pieces = 256 * fp / 16;
    const uint8_t *from = p.f + (static_cast<int64_t>(t.group) * p.N + n_wg) * fp;
    const int32_t real = static_cast<int32_t>(min(static_cast<int64_t>(256), p.N - n_wg)) * fp / 16;
    for (int32_t i = threadIdx.x; i < pieces; i += kOuterThreads)
      *reinterpret_cast<uint4 *>(smem + i * 16) =
          i < real ? *reinterpret_cast<const uint4 *>(from + i * 16) : make_uint4(0, 0, 0, 0);
    __syncthreads();
#pragma unroll
    for (int v = 0; v < GF; ++v)
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const int u = (4 * v + (wave >> 1)) % RF;
        const uint8_t *at = smem + (32 * ks + 8 * j + (l16 >> 2)) * fp + (16 * u + 4 * (l16 & 3u)) * 2;
        f[v][ks] = pair(tr(at), tr(at + 4 * fp));
      }
    wait_lgkmcnt0();
  }
  __syncthreads();  // (the ring takes f's place; y_rows are there)
  const int32_t RC3 = 3 * p.R / 8;                 // 16-byte chunks of a row of pieces
  const int32_t pitch = RC3 * 16;
  // 32-byte unit u of row t of the pieces sits at u + turn(t) modulo their number, where a row is whole units
  const int32_t units = p.R % 16 == 0 ? 3 * p.R / 16 : 0;
  auto turn = [](uint32_t row) { return static_cast<int32_t>(((row & 3u) >> 1) + ((row >> 3) & 1u) * 2u); };
  const int32_t steps = static_cast<int32_t>((t.m_end - t.m0 + kOuterStep - 1) / kOuterStep);
  // y: wave w loads rows [4 w, 4 w + 4), two a load; lane: row lane >> 5, position lane & 31
  uint32_t col[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t T = 4 * wave + 2 * i + (lane >> 5);
    const uint32_t u = ((lane & 31u) >> 1) ^ ((T & 3u) | ((T >> 1) & 4u));
    col[i] = u * 16 + (lane & 1u) * 8;
  }
  int32_t prow[NP + 1], pchunk[NP + 1];
#pragma unroll
  for (int i = 0; i < NP + 1; ++i) {
    const int32_t at = (8 * i + wave) * 64 + lane;
    prow[i] = at / RC3;
    pchunk[i] = at - prow[i] * RC3;
    if (units) {
      int32_t u = (pchunk[i] >> 1) - turn(prow[i]);
      if (u < 0) u += units;
      pchunk[i] = 2 * u + (pchunk[i] & 1);
    }
  }
  auto load = [&](int32_t kt) {
    uint8_t *st = smem + (kt % S) * kStage;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int32_t at = kt * kOuterStep + 4 * wave + 2 * i + (lane >> 5), y = at < p.chunk ? y_rows[at] : -1;
      const int64_t n = n_wg + col[i];
      lds_load16(y >= 0 && n < p.N ? p.y + y * p.ldy + n * 2 : zeros, st + (4 * wave + 2 * i) * 512);
    }
    const int64_t r0 = t.m0 + static_cast<int64_t>(kt) * kOuterStep;
    auto piece = [&](int i) {
      const int64_t r = r0 + prow[i];
      lds_load16(prow[i] < kOuterStep && r < t.m_end ? p.pieces + r * pitch + pchunk[i] * 16 : zeros,
                 st + kY + (8 * i + wave) * 1024);
    };
#pragma unroll
    for (int i = 0; i < NP; ++i) piece(i);
    if (rest > 0 && wave < rest) piece(NP);
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) load(s);
  floatx4 acc[RF][2];
#pragma unroll
  for (int u = 0; u < RF; ++u)
#pragma unroll
    for (int v = 0; v < 2; ++v) acc[u][v] = (floatx4){0.0f, 0.0f, 0.0f, 0.0f};
  for (int32_t kt = 0; kt < steps; ++kt) {
    // (stores of the second product count too, and then a few of the later steps' loads are waited for)
    if (rest > 0 && wave < rest)
      wait_vmcnt<(S - 2) * (3 + NP)>();
    else
      wait_vmcnt<(S - 2) * (2 + NP)>();
    wait_lgkmcnt0();
    lds_barrier();
    load(kt + S - 1);
    uint8_t *st = smem + (kt % S) * kStage;
    bf16x8 y[2];
    const uint32_t T = 8 * j + (l16 >> 2);  // (row T + 4 has the same swizzle and turn)
    const int32_t mine = turn(T);
    const uint32_t sw = (T & 3u) | ((T >> 1) & 4u);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const uint8_t *at = st + T * 512 + ((2 * wave + v) ^ sw) * 32 + (l16 & 3u) * 8;
      y[v] = pair(tr(at), tr(at + 4 * 512));
    }
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int u = 0; u < RF; ++u) {
        int32_t unit = s * (p.R / 16) + u + mine;
        unit = unit >= units ? unit - units : unit;
        const uint8_t *at = st + kY + T * pitch + (units ? unit * 32 : (s * p.R + 16 * u) * 2) + (l16 & 3u) * 8;
        const bf16x8 a = pair(tr(at), tr(at + 4 * pitch));
#pragma unroll
        for (int v = 0; v < 2; ++v) acc[u][v] = mfma(a, y[v], acc[u][v]);
      }
    if (G && (RF >= 4 || wave < 2 * RF)) {
      const uint32_t tr_row = 16 * (wave & 1) + l16, sw2 = (tr_row & 3u) | ((tr_row >> 1) & 4u);
      floatx4 g[GF];
#pragma unroll
      for (int v = 0; v < GF; ++v) g[v] = (floatx4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const bf16x8 b = frag(st + tr_row * 512 + ((2 * ks + (j >> 1)) ^ sw2) * 32 + (j & 1u) * 16);
#pragma unroll
        for (int v = 0; v < GF; ++v) g[v] = mfma(f[v][ks], b, g[v]);
      }
      const int64_t r = t.m0 + static_cast<int64_t>(kt) * kOuterStep + tr_row;
#pragma unroll
      for (int v = 0; v < GF; ++v) {
        const int q = 16 * ((4 * v + (wave >> 1)) % RF) + 4 * j;
        if (r < t.m_end && q < p.R)
          *reinterpret_cast<floatx4 *>(p.g_part + (static_cast<int64_t>(tn) * p.rows.M + r) * p.R + q) = g[v];
      }
    }
  }
  wait_vmcnt<0>();
  float *out = t.tiles == 1 ? p.out + static_cast<int64_t>(t.group) * p.N * p.R : p.part + static_cast<int64_t>(tm) * p.N * p.R;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const int64_t n = n_wg + 32 * wave + 16 * v + l16;
    if (n >= p.N) continue;
#pragma unroll
    for (int u = 0; u < RF; ++u) {
      const int q = 16 * u + 4 * j;
      if (q >= p.R) continue;
      if (p.n_major) {
        *reinterpret_cast<floatx4 *>(out + n * p.R + q) = acc[u][v];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) out[(q + e) * p.N + n] = acc[u][v][e];
      }
    }
  }
}

// Sums of an adapter's chunks in order; zeros for an adapter without rows.  Only chunks that a workgroup of the launch before
// had are read, whatever the offsets are: those among its tiles that start at one of the M rows.
struct OuterSumArgs {
  Rows rows;
  int32_t chunk;
  int64_t tiles;  // of the launch before
  int64_t size;  // N R
  int32_t blocks;  // workgroups an adapter
  const float *part;
  float *out;
};
constexpr int kOuterSumSize = 1024;
__device__ __forceinline__ void outer_sum(const OuterSumArgs &p, int64_t id) {
  const int32_t g = static_cast<int32_t>(id / p.blocks), lane = threadIdx.x & 63;
  int64_t first = 0, lo = 0, n;
  if (p.rows.offsets) {
    int32_t before = 0;
    for (int i = lane; i < g; i += 64) {
      const int32_t rows = p.rows.offsets[i + 1] - p.rows.offsets[i];
      before += rows > 0 ? (rows - 1) / p.chunk + 1 : 0;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) before += __shfl_xor(before, d);
    first = before;
    lo = p.rows.offsets[g];
    const int32_t rows = p.rows.offsets[g + 1] - p.rows.offsets[g];
    n = rows > 0 ? (rows - 1) / p.chunk + 1 : 0;
  } else {
    n = (p.rows.M + p.chunk - 1) / p.chunk;
  }
  // chunk c starts at row lo + c chunk and is tile first + c
  const bool direct = n == 1;  // the result itself
  int64_t c0 = lo < 0 ? (p.chunk - 1 - lo) / p.chunk : 0;
  if (first < 0) n = 0;
  n = min(n, min(p.tiles - first, (p.rows.M - lo + p.chunk - 1) / p.chunk));
  if (direct && c0 == 0 && n == 1) return;
  const int64_t i = (id - static_cast<int64_t>(g) * p.blocks) * kOuterSumSize + threadIdx.x * 4;
  if (i >= p.size) return;
  floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (!direct)
#pragma unroll 4
    for (int64_t c = c0; c < n; ++c) v += *reinterpret_cast<const floatx4 *>(p.part + (first + c) * p.size + i);
  *reinterpret_cast<floatx4 *>(p.out + g * p.size + i) = v;
}
__global__ __launch_bounds__(256) void outer_sum_kernel(OuterSumArgs a, OuterSumArgs b, int64_t blocks_a) {
  if (blockIdx.x < blocks_a)
    outer_sum(a, blockIdx.x);
  else
    outer_sum(b, blockIdx.x - blocks_a);
}

// ---- before a backward pass: a transposed factor, and the pieces of h -------------------------------------------
// out[g][c][r] = in[g][r][c], [rows x cols] bf16 with rows and cols multiples of 8; 64 x 64 tiles, 16 bytes a thread both ways.
struct TransposeArgs {
  const uint16_t *in;
  uint16_t *out;
  int64_t rows, cols;
  int32_t tiles_r, tiles_c;
};
constexpr int kTurnPitch = 66;  // elements of a row in LDS: eight rows of one column lie in different banks
__device__ void transpose_tile(const TransposeArgs &p, int64_t id, uint16_t (&lds)[64 * kTurnPitch]) {
  const int64_t per = static_cast<int64_t>(p.tiles_r) * p.tiles_c, g = id / per;
  const int32_t in_g = static_cast<int32_t>(id - g * per), tr = in_g / p.tiles_c, tc = in_g - tr * p.tiles_c;
  const int64_t r0 = tr * 64ll, c0 = tc * 64ll;
  const uint16_t *in = p.in + g * p.rows * p.cols;
  uint16_t *out = p.out + g * p.rows * p.cols;
#pragma unroll
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int r = i / 8, c = i % 8 * 8;
    if (r0 + r >= p.rows || c0 + c >= p.cols) continue;
    const uint4 v = *reinterpret_cast<const uint4 *>(in + (r0 + r) * p.cols + c0 + c);
    uint32_t *at = reinterpret_cast<uint32_t *>(&lds[r * kTurnPitch + c]);
    at[0] = v.x;
    at[1] = v.y;
    at[2] = v.z;
    at[3] = v.w;
  }
  __syncthreads();
#pragma unroll
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int c = i / 8, r = i % 8 * 8;
    if (r0 + r >= p.rows || c0 + c >= p.cols) continue;
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = lds[(r + 2 * q) * kTurnPitch + c] | static_cast<uint32_t>(lds[(r + 2 * q + 1) * kTurnPitch + c]) << 16;
    *reinterpret_cast<uint4 *>(out + (c0 + c) * p.rows + r0 + r) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// The pieces of scale * h, 64 rows a workgroup.
struct PiecesArgs {
  Rows rows;
  const float *h;  // [M][R]
  int32_t R;
  const float *scales;
  uint8_t *pieces;  // [M][3 R] bf16
};
constexpr int kPiecesRows = 64;
__device__ __forceinline__ void pieces_tile(const PiecesArgs &p, int32_t tm) {
  Tile t;
  if (!find_tile(p.rows, kPiecesRows, tm, t)) return;
  const int32_t RC = p.R / 8;
  const float scale = p.scales[t.group];
  for (int i = threadIdx.x; i < kPiecesRows * RC; i += 256) {
    const int64_t r = t.m0 + i / RC;
    const int32_t rc = i % RC;
    if (r >= t.m_end) break;
    const floatx4 *at = reinterpret_cast<const floatx4 *>(p.h + r * p.R + 8 * rc);
    const floatx4 lo = at[0], hi = at[1];
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (e < 4 ? lo[e] : hi[e - 4]) * scale;
    uint4 w[3];
    split8(v, w);
    uint4 *out = reinterpret_cast<uint4 *>(p.pieces + r * (6 * p.R)) + rc;
    out[0] = w[0];
    out[RC] = w[1];
    out[2 * RC] = w[2];
  }
}
__global__ __launch_bounds__(256) void adapter_prep_kernel(TransposeArgs a, int64_t blocks_a, PiecesArgs h) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[64 * kTurnPitch];
  if (blockIdx.x < blocks_a)
    transpose_tile(a, blockIdx.x, lds);
  else
    pieces_tile(h, static_cast<int32_t>(blockIdx.x - blocks_a));
}

// ---- launches ----------------------------------------------------------------------------------------------------
Rows rows_of(const AdapterArgs &a) {
  Rows p{};
  p.offsets = a.offsets;
  p.rows = a.rows;
  p.groups = a.adapters;
  p.x_div = a.by_token ? 1 : (a.gather ? a.row_div : 0);
  p.x_shift = p.x_div > 0 && (p.x_div & (p.x_div - 1)) == 0 ? __builtin_ctz(p.x_div) : -1;
  p.by_rows = a.by_token;
  p.M = a.M;
  p.x_rows = a.x_rows;
  return p;
}
// Tiles of `size` rows that any offsets could need.
int64_t tiles_for(const AdapterArgs &a, int64_t size) {
  if (!a.offsets) return (a.M + size - 1) / size;
  return a.M / size + (a.adapters < a.M ? a.adapters : a.M);
}

// Rows of a workgroup that adds to many rows of c: what a lane holds of base's rows is then the same for both types.
template <bool BF16>
constexpr int kExpandRows = BF16 ? 64 : 32;
// Workgroups of the launch that adds to c, at least, where there is work for them.  Whole calls of 8192 x 4096 x 14336, eight
// adapters, replayed from a graph: rank 16 at 903 workgroups 131 us, 1806 113, 7224 107; rank 64 156, 139 and 135.
constexpr int64_t kExpandGroups = 1536, kFewGroups = 1024;

// A few rows of low rank: one launch, in which each workgroup forms its rows' h by itself, as long as every workgroup has a
// compute unit and A is small.  From Python, where a call's own time counts, a token of 4096 x 14336 and rank 16 takes 13.4 us
// so and 17.2 in two launches.  Replayed from a graph one launch gains up to a K of 1024 or so and loses from there on: 64 rows
// of 1024 x 1024 6.5 us against 7.9, 256 of 512 x 512 6.3 against 7.8, 16 of 4096 x 4096 8.0 either way, the token above 9.2
// against 7.8, one of 4096 x 4096 and rank 32 12.5 against 8.6, one of 14336 x 4096 and rank 8 16.6 against 8.5.
constexpr int32_t kOwnRank = 32;
bool own_h(int64_t M, int64_t N, int64_t K, int32_t rank, int32_t adapters) {
  const int64_t tiles = adapters == 1 ? (M + 15) / 16 : (M < adapters ? M : adapters) + M / 16;
  return rank <= kOwnRank && rank * K <= (1 << 17) && tiles * ((N + 255) / 256) <= 256;
}

// Few rows an adapter: 16 rows a tile.  (K 4096, replayed from a graph, in tiles of 16 and of 64 rows: 512 rows of 32 adapters of
// rank 16 18 and 24 us, 2048 of 128 39 and 55, 8000 of 512 182 and 182, of rank 64 170 and 184.  The rule counts the adapters
// that there are; where a few of them have all rows, 1024 of 64 take 21 and 26 us, 8000 of 512 138 and 136, and of rank 64
// 105 and 103; 2048 rows of 2 in 128 of rank 64 32 and 26.)
bool few_rows(int64_t M, int64_t adapters) { return M <= 256 || M <= 16 * adapters; }

// Splits of K for many rows: workgroups for every compute unit, each with at least four steps.  Gathered rows come up
// again for each of a token's experts: in eight splits, each XCD (workgroup i runs on XCD i mod 8) meets only its own
// eighth of every row, which its L2 holds.
void many_splits(int64_t M, int64_t K, bool gather, int32_t &splits, int32_t &split_k) {
  const int64_t tiles = (M + kManyRows - 1) / kManyRows, steps = (K + kManyStep - 1) / kManyStep;
  int64_t n = gather ? 8 : (768 + tiles - 1) / tiles;
  if (n > steps / 4) n = steps / 4;
  if (n > 8) n = 8;
  if (n < 1) n = 1;
  const int64_t per = (steps + n - 1) / n;
  split_k = static_cast<int32_t>(per * kManyStep);
  splits = static_cast<int32_t>((steps + per - 1) / per);
}
int32_t splits_for(int64_t M, int64_t adapters, int64_t K, bool gather) {
  if (few_rows(M, adapters)) return static_cast<int32_t>((K + kFewK - 1) / kFewK);
  int32_t n, k;
  many_splits(M, K, gather, n, k);
  return n;
}

template <int RF>
hipError_t run_shrink(const ShrinkArgs &p, bool few, int64_t tiles, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(tiles * p.splits));
  if (few)
    shrink_few_kernel<RF><<<grid, dim3(64 * kFewWaves), 0, stream>>>(p);
  else
    shrink_many_kernel<RF><<<grid, dim3(256), 0, stream>>>(p);
  return hipGetLastError();
}
hipError_t run_shrink(const AdapterArgs &a, float *part, int32_t &splits) {
  ShrinkArgs p{};
  p.rows = rows_of(a);
  p.y = static_cast<const uint8_t *>(a.x);
  p.ldy = a.ldx * 2;
  p.f = static_cast<const uint8_t *>(a.a);
  p.K = a.K;
  p.R = a.rank;
  p.part = part;
  const bool few = few_rows(a.M, a.adapters);
  if (few) {
    p.splits = static_cast<int32_t>((a.K + kFewK - 1) / kFewK);
    p.split_k = kFewK;
  } else {
    many_splits(a.M, a.K, a.gather, p.splits, p.split_k);
  }
  splits = p.splits;
  const int64_t tiles = tiles_for(a, few ? 16 : kManyRows);
  if (a.rank <= 16) return run_shrink<1>(p, few, tiles, a.stream);
  if (a.rank <= 32) return run_shrink<2>(p, few, tiles, a.stream);
  if (a.rank <= 64) return run_shrink<4>(p, few, tiles, a.stream);
  return run_shrink<8>(p, few, tiles, a.stream);
}

template <int RCP, bool BF16>
hipError_t run_expand(const ExpandArgs &p, bool few, bool vec, uint32_t groups, hipStream_t stream) {
  constexpr int TF = kExpandRows<BF16> / 16;
  const bool once = p.base && 2 * p.rows.M * p.N * (BF16 ? 2 : 4) >= kStreamBytes;
  const dim3 grid(groups), threads(256);
  if (p.a) {
    if constexpr (RCP <= kOwnRank / 8) {
      if (vec)
        expand_kernel<RCP, 1, BF16, false, true, true><<<grid, threads, 0, stream>>>(p);
      else
        expand_kernel<RCP, 1, BF16, false, false, true><<<grid, threads, 0, stream>>>(p);
    }
  } else if (!vec) {
    if (few)
      expand_kernel<RCP, 1, BF16, false, false, false><<<grid, threads, 0, stream>>>(p);
    else
      expand_kernel<RCP, TF, BF16, false, false, false><<<grid, threads, 0, stream>>>(p);
  } else if (few) {
    expand_kernel<RCP, 1, BF16, false, true, false><<<grid, threads, 0, stream>>>(p);
  } else if (once) {
    expand_kernel<RCP, TF, BF16, true, true, false><<<grid, threads, 0, stream>>>(p);
  } else {
    expand_kernel<RCP, TF, BF16, false, true, false><<<grid, threads, 0, stream>>>(p);
  }
  return hipGetLastError();
}
template <bool BF16>
hipError_t run_expand(const ExpandArgs &p, bool few, bool vec, uint32_t groups, hipStream_t stream) {
  if (p.R <= 8) return run_expand<1, BF16>(p, few, vec, groups, stream);
  if (p.R <= 16) return run_expand<2, BF16>(p, few, vec, groups, stream);
  if (p.R <= 32) return run_expand<4, BF16>(p, few, vec, groups, stream);
  if (p.R <= 64) return run_expand<8, BF16>(p, few, vec, groups, stream);
  return run_expand<16, BF16>(p, few, vec, groups, stream);
}
hipError_t run_expand(const AdapterArgs &a, const void *f, int64_t N, float *part, int32_t splits, float *h, uint8_t *pieces,
                      const void *base, int64_t ldb, void *c, int64_t ldc, int dtype) {
  ExpandArgs p{};
  const int64_t es = dtype == 1 ? 2 : 4;
  const bool few = !part || few_rows(a.M, a.adapters);
  p.rows = rows_of(a);
  p.pos = a.pos;
  p.f = static_cast<const uint8_t *>(f);
  p.N = N;
  p.R = a.rank;
  p.part = part;
  p.splits = splits;
  if (!part) {
    p.x = static_cast<const uint8_t *>(a.x);
    p.ldx = a.ldx * 2;
    p.a = static_cast<const uint8_t *>(a.a);
    p.K = a.K;
  }
  p.scales = a.scales;
  p.h = h;
  p.pieces = pieces;
  p.base = static_cast<const uint8_t *>(base);
  p.ldb = ldb * es;
  p.c = static_cast<uint8_t *>(c);
  p.ldc = ldc * es;
  // rows of base and c aligned to 16 bytes, which N fills; else pieces at any element, and each row's last by itself (whole
  // calls of 8192 rows, rank 16, K 4096: 14336 columns 110 us, 14335 164, and 667 with all of them element by element)
  const bool vec = (reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(c) | static_cast<uintptr_t>(p.ldc) |
           static_cast<uintptr_t>(base ? p.ldb : 0) | static_cast<uintptr_t>(N * es)) % 16 == 0;
  const int32_t tile_rows = few ? 16 : dtype == 1 ? kExpandRows<true> : kExpandRows<false>;
  p.tiles_m = static_cast<int32_t>(tiles_for(a, tile_rows));
  // as many steps of 256 columns a workgroup as leave kExpandGroups workgroups
  const int64_t steps = (N + 255) / 256, tiles = (a.M + tile_rows - 1) / tile_rows;
  const int64_t used = few && a.offsets ? (a.M < a.adapters ? a.M : a.adapters) : 0;  // at most so many tiles in use
  int64_t each = steps * (tiles > used ? tiles : used) / (few ? kFewGroups : kExpandGroups);
  if (each < 1 || !part) each = 1;
  if (each > steps) each = steps;
  // the splits are summed first where each workgroup's own sums would read more than a quarter of what it moves of c
  if (!few && splits > 1 && splits * p.R * 4 * 4 > each * 256 * 2 * es) {
    const int64_t size = a.M * p.R;
    split_sum_kernel<<<dim3(static_cast<uint32_t>((size + 1023) / 1024)), dim3(256), 0, a.stream>>>(part, size, splits);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.splits = 1;
  }
  p.columns = static_cast<int32_t>((steps + (steps + each - 1) / each - 1) / ((steps + each - 1) / each) * 256);
  p.tiles_n = static_cast<int32_t>((N + p.columns - 1) / p.columns);
  // rows without an adapter have to be written unless c is base
  const int64_t copies = a.offsets && base != c ? (a.M + 63) / 64 : 0;
  const uint32_t groups = static_cast<uint32_t>(p.tiles_n * (p.tiles_m + copies));
  return dtype == 1 ? run_expand<true>(p, few, vec, groups, a.stream) : run_expand<false>(p, few, vec, groups, a.stream);
}

// Rows of a workgroup of the factors' gradients: the workgroups are to come near a multiple of those that run at once, two a
// compute unit or, of ranks above 64, one (for 56 column tiles and 8192 rows: 504 workgroups of 928 rows and not 896 of 512,
// which leave a quarter of the second round idle; each further adapter is counted as a partial tile).  Workgroups of few rows
// write and read more partial sums than rows of y: four times the rank makes them equal, and from twice the rank on more
// workgroups gain more (2047 rows of 4096 and rank 64: 24.6 us with at least 256 rows, 20.4 with 128).
int32_t outer_chunk(int64_t M, int64_t N, int32_t rank, int32_t adapters) {
  const int64_t tiles_n = (N + 255) / 256, slots = rank <= 64 ? 512 : 256;
  int64_t rounds = 1, n, chunk;
  do {
    n = rounds++ * slots / tiles_n - (adapters - 1);
    if (n < 1) n = 1;
    chunk = (M + n - 1) / n;
  } while (chunk > kMaxChunk && rounds <= 64);
  auto steps = [](int64_t rows) { return (rows + kOuterStep - 1) / kOuterStep * kOuterStep; };
  const int64_t least = 2 * rank > 64 ? steps(2 * rank) : 64;
  chunk = steps(chunk);
  return static_cast<int32_t>(chunk < least ? least : chunk > kMaxChunk ? kMaxChunk : chunk);
}
template <int RF>
hipError_t run_outer(const OuterArgs &p, uint32_t groups, hipStream_t stream) {
  if (p.f)
    outer_kernel<RF, true><<<dim3(groups), dim3(kOuterThreads), 0, stream>>>(p);
  else
    outer_kernel<RF, false><<<dim3(groups), dim3(kOuterThreads), 0, stream>>>(p);
  return hipGetLastError();
}
hipError_t run_outer(const AdapterArgs &a, OuterArgs p) {
  p.rows = rows_of(a);
  p.ldy *= 2;
  p.R = a.rank;
  p.chunk = outer_chunk(a.M, p.N, a.rank, a.adapters);
  p.tiles_n = static_cast<int32_t>((p.N + 255) / 256);
  const uint32_t groups = static_cast<uint32_t>(p.tiles_n * tiles_for(a, p.chunk));
  if (a.rank <= 16) return run_outer<1>(p, groups, a.stream);
  if (a.rank <= 32) return run_outer<2>(p, groups, a.stream);
  if (a.rank <= 64) return run_outer<4>(p, groups, a.stream);
  return run_outer<8>(p, groups, a.stream);
}

// The workspace's parts, each a multiple of 256 bytes.
struct Layout {
  size_t at = 0;
  size_t take(int64_t bytes) {
    const size_t here = at;
    at += (static_cast<size_t>(bytes) + 255) / 256 * 256;
    return here;
  }
};
struct ForwardLayout {
  size_t part, size;
  ForwardLayout(int64_t M, int64_t N, int64_t K, int32_t R, int32_t adapters) {
    Layout l;
    part = size = 0;
    if (own_h(M, N, K, R, adapters)) return;
    // (as large for gathered rows as for others)
    const int64_t own = splits_for(M, adapters, K, false), gathered = splits_for(M, adapters, K, true);
    part = l.take((own > gathered ? own : gathered) * M * R * 4);
    size = l.at;
  }
};
struct BackwardLayout {
  size_t at, h_pieces, part, g_pieces, da_part, db_part, size;
  BackwardLayout(const AdapterArgs &a) {
    Layout l;
    const int64_t factor = static_cast<int64_t>(a.adapters) * a.rank;
    at = l.take(factor * a.K * 2);
    h_pieces = l.take(a.M * a.rank * 6);
    part = l.take((a.N + 255) / 256 * a.M * a.rank * 4);
    g_pieces = l.take(a.M * a.rank * 6);
    da_part = l.take(tiles_for(a, outer_chunk(a.M, a.K, a.rank, a.adapters)) * a.K * a.rank * 4);
    db_part = l.take(tiles_for(a, outer_chunk(a.M, a.N, a.rank, a.adapters)) * a.N * a.rank * 4);
    size = l.at;
  }
};

}  // namespace

size_t adapter_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t rank, int32_t adapters) {
  return ForwardLayout(M, N, K, rank, adapters).size;
}
size_t adapter_backward_workspace_bytes(const AdapterArgs &a) { return BackwardLayout(a).size; }

// (2^32 threads or more do not launch)
bool adapter_launches(const AdapterArgs &a, bool backward) {
  constexpr int64_t kMost = int64_t(1) << 23;
  const int64_t widest = ((a.N > a.K ? a.N : a.K) + 255) / 256;
  const bool few = few_rows(a.M, a.adapters);
  const int64_t tiles = tiles_for(a, 16) + (a.M + 63) / 64;
  const int64_t splits = backward ? 1 : splits_for(a.M, a.adapters, a.K, a.gather);
  const int64_t sums = backward ? a.adapters * ((a.N + a.K) * a.rank / kOuterSumSize + 2) : 0;
  const int64_t prep = backward ? a.adapters * ((a.rank + 63) / 64) * ((a.K + 63) / 64) + tiles : 0;
  return tiles * widest < kMost && tiles * splits < kMost && sums < kMost && prep < kMost &&
         (!backward || widest * tiles_for(a, 64) < kMost);
}

hipError_t launch_adapter(const AdapterArgs &a) {
  if (own_h(a.M, a.N, a.K, a.rank, a.adapters))
    return run_expand(a, a.b, a.N, nullptr, 0, a.h, nullptr, a.base, a.ldb, a.c, a.ldc, a.c_dtype);
  const ForwardLayout l(a.M, a.N, a.K, a.rank, a.adapters);
  uint8_t *const w = static_cast<uint8_t *>(a.workspace);
  float *const part = reinterpret_cast<float *>(w + l.part);
  int32_t splits;
  const hipError_t e = run_shrink(a, part, splits);
  if (e != hipSuccess) return e;
  return run_expand(a, a.b, a.N, part, splits, a.h, nullptr, a.base, a.ldb, a.c, a.ldc, a.c_dtype);
}

hipError_t launch_adapter_backward(const AdapterArgs &a) {
  const BackwardLayout l(a);
  uint8_t *const w = static_cast<uint8_t *>(a.workspace);
  float *const part = reinterpret_cast<float *>(w + l.part), *const da_part = reinterpret_cast<float *>(w + l.da_part),
              *const db_part = reinterpret_cast<float *>(w + l.db_part);
  const Rows rows = rows_of(a);
  hipError_t e;
  if (a.M > 0) {
    // A^T [K][R], and the pieces of s h
    auto tiles = [](int64_t n) { return static_cast<int32_t>((n + 63) / 64); };
    const TransposeArgs ta{static_cast<const uint16_t *>(a.a), reinterpret_cast<uint16_t *>(w + l.at), a.rank, a.K,
                           tiles(a.rank), tiles(a.K)};
    const PiecesArgs h{rows, a.h, a.rank, a.scales, w + l.h_pieces};
    const int64_t na = static_cast<int64_t>(a.adapters) * ta.tiles_r * ta.tiles_c;
    adapter_prep_kernel<<<dim3(static_cast<uint32_t>(na + tiles_for(a, kPiecesRows))), dim3(256), 0, a.stream>>>(ta, na, h);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    // dB's parts and g's from one pass over dc; dx from g, and its pieces; dA's parts
    OuterArgs o{};
    o.y = static_cast<const uint8_t *>(a.dc);
    o.ldy = a.lddc;
    o.N = a.N;
    o.pieces = w + l.h_pieces;
    o.n_major = true;
    o.part = db_part;
    o.out = a.db;
    o.f = static_cast<const uint8_t *>(a.b);
    o.g_part = part;
    if ((e = run_outer(a, o)) != hipSuccess) return e;
    const int32_t tiles_n = static_cast<int32_t>((a.N + 255) / 256);
    e = run_expand(a, w + l.at, a.K, part, tiles_n, nullptr, w + l.g_pieces, a.base, a.ldb, a.c, a.ldc, a.c_dtype);
    if (e != hipSuccess) return e;
    o = {};
    o.y = static_cast<const uint8_t *>(a.x);
    o.ldy = a.ldx;
    o.N = a.K;
    o.pieces = w + l.g_pieces;
    o.part = da_part;
    o.out = a.da;
    if ((e = run_outer(a, o)) != hipSuccess) return e;
  }
  const int32_t ca = outer_chunk(a.M, a.K, a.rank, a.adapters), cb = outer_chunk(a.M, a.N, a.rank, a.adapters);
  OuterSumArgs sa{rows, ca, tiles_for(a, ca), a.K * a.rank, 0, da_part, a.da};
  OuterSumArgs sb{rows, cb, tiles_for(a, cb), a.N * a.rank, 0, db_part, a.db};
  sa.blocks = static_cast<int32_t>((sa.size + kOuterSumSize - 1) / kOuterSumSize);
  sb.blocks = static_cast<int32_t>((sb.size + kOuterSumSize - 1) / kOuterSumSize);
  const int64_t na = static_cast<int64_t>(a.adapters) * sa.blocks, nb = static_cast<int64_t>(a.adapters) * sb.blocks;
  outer_sum_kernel<<<dim3(static_cast<uint32_t>(na + nb)), dim3(256), 0, a.stream>>>(sa, sb, na);
  return hipGetLastError();
}

}  // namespace nvfp4
