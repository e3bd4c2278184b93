// gemm_int8.hip -- products of 8-bit integers on the gfx950 matrix cores, with a scale for each token and
// each channel, plain or by expert:
//   C[i][j] = (sa_i sb_j) sum_k a_ik b_jk,
// the sum exact in 32-bit integers (v_mfma_i32_32x32x32_i8), so neither tiling nor the split of K changes a
// bit.
//
// Tiles.  A workgroup of four waves owns a BM x BN tile, each wave a quarter of it.  K advances 128 bytes
// a step through a ring of LDS stages filled by direct global->LDS loads; a stage holds A [BM][128 B] and
// B [BN][128 B], 16-byte chunk c of row r at position c ^ swz(r) (conflict-free ds_read_b128).  Within
// a step, lane half h and sub-step s take the chunk 2 s + h of both operands.  The last step of a K
// that is no multiple of 128 reads zeros for A beyond K (and any valid bytes for B).
//
// By expert.  The row offsets live on the device, so the launch has as many workgroups as any offsets
// could need (a partial tile more for every expert), and each finds its tile by a scan over the experts'
// tile counts; those beyond the last tile leave.  A's rows may be read through the plan's slots.
#include "gemm_common.hpp"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

using namespace gemm;

typedef int intx16 __attribute__((ext_vector_type(16)));
typedef int intx4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;  // bytes of K a step

struct I8Args {
  const uint8_t *a;
  const float *a_scales;
  int64_t a_rows;
  const uint8_t *b;
  const float *b_scales;
  int64_t M, N;
  uint32_t K;
  uint8_t *c;
  int64_t ldc;
  int32_t tiles_n;
  int32_t tiles;  // plain form: all tiles
  int32_t groups;
  const int32_t *offsets;  // NULL: one group of M rows
  const int32_t *rows;     // NULL: row r of C is row r of A
  int32_t row_div;
  int32_t vec_store;
};

// What A reads beyond K in the last step.
__device__ const uint4 kZeros = {0u, 0u, 0u, 0u};

__device__ __forceinline__ uint32_t swz(uint32_t r) { return (r + ((r >> 3) & 3u)) & 7u; }

// The rows of C of a tile row: rows [m0, m_end) of group g.
struct TileRows {
  int32_t group;
  int64_t m0, m_end;
};

// Finds tile row `tm` among the groups' ceil(rows / BM) tile rows; false beyond the last.  Every lane of
// the wave takes part and has the result.
template <int BM>
__device__ __forceinline__ bool find_rows(const int32_t *offsets, int groups, int32_t tm, TileRows &out) {
  const int lane = threadIdx.x & 63;
  int32_t before = 0;
  for (int g0 = 0; g0 < groups; g0 += 64) {
    const int g = g0 + lane;
    const int32_t lo = g < groups ? offsets[g] : 0, hi = g < groups ? offsets[g + 1] : 0;
    const int32_t n = hi > lo ? (hi - lo + BM - 1) / BM : 0;
    int32_t s = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int32_t o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    const uint64_t past = __ballot(before + s > tm);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int32_t first = before + __shfl(s - n, at);
      out.group = g0 + at;
      out.m0 = __shfl(lo, at) + static_cast<int64_t>(tm - first) * BM;
      out.m_end = __shfl(hi, at);
      return true;
    }
    before += __shfl(s, 63);
  }
  return false;
}
// Tile rows of all groups.
template <int BM>
__device__ __forceinline__ int32_t count_rows(const int32_t *offsets, int groups) {
  const int lane = threadIdx.x & 63;
  int32_t n = 0;
  for (int g = lane; g < groups; g += 64) {
    const int32_t lo = offsets[g], hi = offsets[g + 1];
    n += hi > lo ? (hi - lo + BM - 1) / BM : 0;
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) n += __shfl_xor(n, d);
  return n;
}

// Row of A behind row r of C.
__device__ __forceinline__ int64_t a_row(const I8Args &p, int64_t r) {
  if (!p.rows) return r;
  const int64_t s = p.rows[r] / p.row_div;
  return s >= 0 && s < p.a_rows ? s : 0;
}

template <int FM, int FN, int STAGES, bool OUT_BF16>
__global__ __launch_bounds__(kThreads, 1) void gemm_int8_kernel(I8Args p) {
  constexpr int TM = 64 * FM, TN = 64 * FN;  // the workgroup's tile; a wave has 32 FM x 32 FN
  constexpr int kB = TM * kStep, kStage = (TM + TN) * kStep;
  constexpr int NA = TM / 32, NB = TN / 32;  // direct loads a wave and step (8 rows each)
  __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * kStage];

  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t h = lane >> 5, l32 = lane & 31u;
  const uint32_t wm = (wave >> 1) * 32 * FM, wn = (wave & 1) * 32 * FN;

  // ---- this workgroup's tile
  TileRows t;
  int32_t tn;
  if (p.offsets) {
    const int32_t tiles_m = count_rows<TM>(p.offsets, p.groups);
    const int32_t total = tiles_m * p.tiles_n;
    // each XCD (workgroup i runs on XCD i mod 8) gets a contiguous range of tiles
    const int32_t per = (total + 7) >> 3, tile = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (static_cast<int32_t>(blockIdx.x >> 3) >= per || tile >= total) return;
    int32_t tm;
    band_tile(tile, p.tiles_n, tiles_m, tm, tn);
    if (!find_rows<TM>(p.offsets, p.groups, tm, t)) return;
    t.group = __builtin_amdgcn_readfirstlane(t.group);
    t.m_end = t.m_end < p.M ? t.m_end : p.M;
    if (t.m0 < 0 || t.m0 >= t.m_end) return;
  } else {
    const int32_t tile = xcd_tile(blockIdx.x, p.tiles);
    int32_t tm;
    band_tile(tile, p.tiles_n, p.tiles / p.tiles_n, tm, tn);
    t.group = 0;
    t.m0 = static_cast<int64_t>(tm) * TM;
    t.m_end = p.M;
  }
  const int64_t n0 = static_cast<int64_t>(tn) * TN;
  const uint8_t *const b = p.b + static_cast<int64_t>(t.group) * p.N * p.K;

  // ---- direct-load sources: wave w fetches rows [TM / 4 w, TM / 4 (w + 1)) of A and the like of B, 8
  // rows a load.  Rows beyond the operand read the last valid one: their products are never stored.
  const uint8_t *srcA[NA], *srcB[NB];
  uint32_t chunkA[NA], chunkB[NB];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const uint32_t R = TM / 4 * wave + 8 * i + (lane >> 3);
    chunkA[i] = ((lane & 7u) ^ swz(R)) * 16;
    srcA[i] = p.a + a_row(p, min(t.m0 + R, t.m_end - 1)) * p.K;
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const uint32_t R = TN / 4 * wave + 8 * i + (lane >> 3);
    chunkB[i] = ((lane & 7u) ^ swz(R)) * 16;
    srcB[i] = b + min(n0 + R, p.N - 1) * p.K;
  }
  const int32_t steps = static_cast<int32_t>((p.K + kStep - 1) / kStep);
  auto load = [&](uint8_t *st, int32_t kt) {
    const uint32_t k0 = static_cast<uint32_t>(kt) * kStep;
    if (k0 + kStep <= p.K) {
#pragma unroll
      for (int i = 0; i < NA; ++i) lds_load16(srcA[i] + (k0 + chunkA[i]), st + (TM / 4 * wave + 8 * i) * kStep);
#pragma unroll
      for (int i = 0; i < NB; ++i) lds_load16(srcB[i] + (k0 + chunkB[i]), st + kB + (TN / 4 * wave + 8 * i) * kStep);
    } else {
#pragma unroll
      for (int i = 0; i < NA; ++i)
        lds_load16(k0 + chunkA[i] < p.K ? srcA[i] + (k0 + chunkA[i]) : reinterpret_cast<const uint8_t *>(&kZeros),
                   st + (TM / 4 * wave + 8 * i) * kStep);
#pragma unroll
      for (int i = 0; i < NB; ++i)
        lds_load16(srcB[i] + (k0 + chunkB[i] < p.K ? k0 + chunkB[i] : 0), st + kB + (TN / 4 * wave + 8 * i) * kStep);
    }
  };

  intx16 acc[FN][FM];  // [B fragment][A fragment]
#pragma unroll
  for (int j = 0; j < FN; ++j)
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][i][r] = 0;

  constexpr int kAhead = STAGES - 1;
  for (int s = 0; s < kAhead && s < steps; ++s) load(smem + s * kStage, s);
  const uint32_t rdA = (wm + l32) * kStep, rdB = kB + (wn + l32) * kStep, sw = swz(l32);
  int cur = 0;
  for (int32_t kt = 0; kt < steps; ++kt) {
    // this wave's loads of step kt have landed; after the barrier everyone's have, and the stage of
    // step kt - 1 is free
    if (kt + kAhead <= steps)
      wait_vmcnt<(kAhead - 1) * (NA + NB)>();
    else
      wait_vmcnt<0>();
    wait_lgkmcnt0();
    lds_barrier();
    const int nxt = cur == 0 ? STAGES - 1 : cur - 1;
    if (kt + kAhead < steps) load(smem + nxt * kStage, kt + kAhead);
    const uint8_t *st = smem + cur * kStage;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t pos = 16 * ((2 * s + h) ^ sw);
      intx4 af[FM], bf[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) af[i] = *reinterpret_cast<const intx4 *>(st + rdA + 4096 * i + pos);
#pragma unroll
      for (int j = 0; j < FN; ++j) bf[j] = *reinterpret_cast<const intx4 *>(st + rdB + 4096 * j + pos);
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bf[j], af[i], acc[j][i], 0, 0, 0);
    }
    cur = cur + 1 == STAGES ? 0 : cur + 1;
  }

  // ---- epilogue: lane (h, l32) holds row l32 of tile (i, j), columns 8 (r >> 2) + 4 h + (r & 3)
  const float *sb = p.b_scales + static_cast<int64_t>(t.group) * p.N;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t row = t.m0 + wm + 32 * i + l32;
    if (row >= t.m_end) continue;
    const float sa = p.a_scales[a_row(p, row)];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t col = n0 + wn + 32 * j + 8 * q + 4 * h;
        if (col >= p.N) continue;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = static_cast<float>(acc[j][i][4 * q + e]) * (sa * sb[min(col + e, p.N - 1)]);
        uint8_t *out = p.c + (row * p.ldc + col) * (OUT_BF16 ? 2 : 4);
        if (p.vec_store && col + 4 <= p.N) {
          if constexpr (OUT_BF16) {
            const bf16x2v lo = __builtin_convertvector((float2v){v[0], v[1]}, bf16x2v);
            const bf16x2v hi = __builtin_convertvector((float2v){v[2], v[3]}, bf16x2v);
            *reinterpret_cast<uint2 *>(out) =
                make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
          } else {
            *reinterpret_cast<float4 *>(out) = make_float4(v[0], v[1], v[2], v[3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < p.N) {
              if constexpr (OUT_BF16)
                reinterpret_cast<uint16_t *>(out)[e] = static_cast<uint16_t>(bf16_rne(v[e]));
              else
                reinterpret_cast<float *>(out)[e] = v[e];
            }
        }
      }
  }
}

template <int FM, int FN, int STAGES>
hipError_t run_tiles(const Int8GemmArgs &a, I8Args p) {
  constexpr int TM = 64 * FM, TN = 64 * FN;
  p.tiles_n = static_cast<int32_t>((a.N + TN - 1) / TN);
  // by expert: every group may have one partial tile row
  const int64_t most = (a.M + TM - 1) / TM + (a.offsets ? a.num_groups : 0);
  const int64_t tiles = most * p.tiles_n;
  if (tiles > (int64_t(1) << 23)) return hipErrorInvalidValue;
  p.tiles = static_cast<int32_t>(tiles);
  const uint32_t grid = static_cast<uint32_t>(a.offsets ? (tiles + 7) / 8 * 8 : tiles);
  if (a.c_dtype == 1)
    gemm_int8_kernel<FM, FN, STAGES, true><<<dim3(grid), dim3(kThreads), 0, a.stream>>>(p);
  else
    gemm_int8_kernel<FM, FN, STAGES, false><<<dim3(grid), dim3(kThreads), 0, a.stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_gemm(const Int8GemmArgs &a) {
  I8Args p{};
  p.a = reinterpret_cast<const uint8_t *>(a.a);
  p.a_scales = a.a_scales;
  p.a_rows = a.a_rows;
  p.b = reinterpret_cast<const uint8_t *>(a.b);
  p.b_scales = a.b_scales;
  p.M = a.M;
  p.N = a.N;
  p.K = static_cast<uint32_t>(a.K);
  p.c = static_cast<uint8_t *>(a.c);
  p.ldc = a.ldc;
  p.groups = a.num_groups;
  p.offsets = a.offsets;
  p.rows = a.rows;
  p.row_div = a.row_div;
  const int64_t es = a.c_dtype == 1 ? 2 : 4;
  p.vec_store = (reinterpret_cast<uintptr_t>(a.c) % (4 * es)) == 0 && a.ldc % 4 == 0;
  const int64_t rows_each = a.M / a.num_groups;
  if (rows_each >= 256) return run_tiles<4, 4, 2>(a, p);
  return run_tiles<1, 1, 4>(a, p);
}

}  // namespace nvfp4
