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
#include "vec_io.hpp"

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
  int32_t groups;
  const int32_t *offsets;  // NULL: one group of M rows
  const int32_t *rows;     // NULL: row r of C is row r of A
  int32_t row_div;
  int32_t splits, split_steps;  // few rows, plain form: K split over workgroups
  int32_t *partial;             // [splits][M][partial_ld]
  int64_t partial_ld;
};

// What A reads beyond K in the last step.
__device__ const uint4 kZeros = {0u, 0u, 0u, 0u};

// 128-byte rows: a ds_read_b128 serves sixteen lanes a pass, lanes 0-3, 12-15 and 20-27 together and so on;
// with this swizzle the fragment rows of each such set cover all 64 banks once.
__device__ __forceinline__ uint32_t swz(uint32_t r) { return (r >> 1) & 7u; }

// The rows of C of a tile row: rows [m0, m_end) of group g.
struct TileRows {
  int32_t group;
  int64_t m0, m_end;
};

// Tile rows of a group of n rows, for tiles of BM rows: all of them, or only those of more than half a tile's rows,
// or only those of less (a group has at most one).
enum TileKind { kAllTiles, kFullTiles, kHalfTiles };
template <int BM, TileKind KIND>
__device__ __forceinline__ int32_t tile_rows(int64_t n) {
  if (n <= 0) return 0;
  const int32_t rest = static_cast<int32_t>(n % BM), whole = static_cast<int32_t>(n / BM);
  if constexpr (KIND == kAllTiles) return whole + (rest > 0);
  if constexpr (KIND == kFullTiles) return whole + (rest > BM / 2);
  return rest > 0 && rest <= BM / 2;
}

// Finds tile row `tm` among the groups' tile rows; false beyond the last.  Every lane of the wave takes part
// and has the result.
template <int BM, TileKind KIND>
__device__ __forceinline__ bool find_rows(const int32_t *offsets, int groups, int32_t tm, TileRows &out) {
  const int lane = threadIdx.x & 63;
  int32_t before = 0;
  for (int g0 = 0; g0 < groups; g0 += 64) {
    const int g = g0 + lane;
    const int32_t lo = g < groups ? offsets[g] : 0, hi = g < groups ? offsets[g + 1] : 0;
    const int32_t n = tile_rows<BM, KIND>(static_cast<int64_t>(hi) - lo);
    int32_t s = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int32_t o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    const uint64_t past = __ballot(before + s > tm);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int32_t first = before + __shfl(s - n, at), m_lo = __shfl(lo, at), m_hi = __shfl(hi, at);
      out.group = g0 + at;
      out.m0 = m_lo + static_cast<int64_t>(KIND == kHalfTiles ? (m_hi - m_lo) / BM : tm - first) * BM;
      out.m_end = m_hi;
      return true;
    }
    before += __shfl(s, 63);
  }
  return false;
}
// Tile rows of all groups.
template <int BM, TileKind KIND>
__device__ __forceinline__ int32_t count_rows(const I8Args &p) {
  if (!p.offsets) return tile_rows<BM, KIND>(p.M);
  const int lane = threadIdx.x & 63;
  int32_t n = 0;
  for (int g = lane; g < p.groups; g += 64)
    n += tile_rows<BM, KIND>(static_cast<int64_t>(p.offsets[g + 1]) - p.offsets[g]);
#pragma unroll
  for (int d = 32; d > 0; d /= 2) n += __shfl_xor(n, d);
  return __builtin_amdgcn_readfirstlane(n);
}

// Row of A behind row r of C.
__device__ __forceinline__ int64_t a_row(const I8Args &p, int64_t r) {
  if (!p.rows) return r;
  const int64_t s = p.rows[r] / p.row_div;
  return s >= 0 && s < p.a_rows ? s : 0;
}

// The number of workgroup `id` among `total` items (false beyond them), dealt so that each XCD (workgroup i runs on
// XCD i mod 8) gets a contiguous range of them.
__device__ __forceinline__ bool deal(int32_t id, int32_t total, int32_t &item) {
  const int32_t per = (total + 7) >> 3;
  item = (id & 7) * per + (id >> 3);
  return (id >> 3) < per && item < total;
}
// Tile number `tile` of `rows` tile rows, walked in bands of tile rows (band_tile); false where there is none.
template <int BM, TileKind KIND>
__device__ __forceinline__ bool find_tile(const I8Args &p, int32_t rows, int32_t tile, TileRows &t, int32_t &tn) {
  int32_t tm;
  band_tile(tile, p.tiles_n, rows, tm, tn);
  if (p.offsets) {
    if (!find_rows<BM, KIND>(p.offsets, p.groups, tm, t)) return false;
    t.group = __builtin_amdgcn_readfirstlane(t.group);
    t.m0 = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(t.m0));
    t.m_end = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(t.m_end));
    t.m_end = t.m_end < p.M ? t.m_end : p.M;
    return t.m0 >= 0 && t.m0 < t.m_end;
  }
  t.group = 0;
  t.m0 = KIND == kHalfTiles ? p.M / BM * BM : static_cast<int64_t>(tm) * BM;
  t.m_end = p.M;
  return true;
}

// 16 bytes at an address aligned to an element only (rows of C may start anywhere).
typedef uint32_t any_u32x4 __attribute__((ext_vector_type(4), aligned(2)));
struct __attribute__((packed, aligned(4))) Floats4 {
  float v[4];
};
struct __attribute__((packed, aligned(2))) Bytes8 {
  uint32_t v[2];
};

// Four consecutive values of a row of C, cut by N.
template <bool OUT_BF16>
__device__ __forceinline__ void store4(const I8Args &p, int64_t row, int64_t col, const float (&v)[4]) {
  uint8_t *out = p.c + (row * p.ldc + col) * (OUT_BF16 ? 2 : 4);
  if (col + 4 <= p.N) {
    if constexpr (OUT_BF16) {
      const bf16x2v lo = __builtin_convertvector((float2v){v[0], v[1]}, bf16x2v);
      const bf16x2v hi = __builtin_convertvector((float2v){v[2], v[3]}, bf16x2v);
      *reinterpret_cast<Bytes8 *>(out) = Bytes8{{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)}};
    } else {
      *reinterpret_cast<Floats4 *>(out) = Floats4{{v[0], v[1], v[2], v[3]}};
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

// C of a wave's FM x FN fragments (32 x 32 each) at rows t.m0 + wm, columns n0 on, 32 rows and at most 256
// bytes of a row at a time through the wave's own LDS (32 rows of kRowBytes): lane (h, l32) holds row l32 of
// fragment (i, j), columns 8 q + 4 h + e; staged rows leave in 16-byte pieces of whole row segments, piece
// c of row r staged at c ^ (r mod pieces).  The columns' scales take the region's last 512 bytes.  No other
// wave may still read the region.
constexpr uint32_t kRegion = 8192 + 512;
template <int FM, int FN, bool OUT_BF16>
__device__ __forceinline__ void store_tile(const I8Args &p, const intx16 (&acc)[FN][FM], uint8_t *region, const TileRows &t,
                                           int64_t n0, uint32_t wm, uint32_t lane) {
  constexpr int ES = OUT_BF16 ? 2 : 4, V = 16 / ES;          // element size, elements of a piece
  constexpr int JP = FN * 32 * ES > 256 ? 256 / (32 * ES) : FN;  // fragments a pass
  constexpr uint32_t kRowBytes = JP * 32 * ES, NP = kRowBytes / 16;
  // (an opaque copy: the per-lane addresses are formed here and not held through the products)
  asm volatile("" : "+v"(lane));
  const uint32_t h = lane >> 5, l32 = lane & 31u;
  const float *sb = p.b_scales + static_cast<int64_t>(t.group) * p.N;
  float s[FN][4][4], sa[FM];
  float *const staged = reinterpret_cast<float *>(region + 8192);
#pragma unroll
  for (uint32_t c = 0; c < 32 * FN; c += 64)
    if (c + lane < 32 * FN) staged[c + lane] = sb[min(n0 + c + lane, p.N - 1)];
#pragma unroll
  for (int i = 0; i < FM; ++i) sa[i] = p.a_scales[a_row(p, min(t.m0 + wm + 32 * i + l32, t.m_end - 1))];
#pragma unroll
  for (int j = 0; j < FN; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 v = *reinterpret_cast<const float4 *>(staged + 32 * j + 8 * q + 4 * h);
      s[j][q][0] = v.x;
      s[j][q][1] = v.y;
      s[j][q][2] = v.z;
      s[j][q][3] = v.w;
    }
  const int64_t rows_left = t.m_end - (t.m0 + wm), cols_left = p.N - n0;
  uint8_t *const out = p.c + ((t.m0 + wm) * p.ldc + n0) * ES;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (32 * i >= rows_left) break;  // (the same in every lane)
#pragma unroll
    for (int j0 = 0; j0 < FN; j0 += JP) {
#pragma unroll
      for (int jj = 0; jj < JP; ++jj)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = j0 + jj;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(acc[j][i][4 * q + e]) * (sa[i] * s[j][q][e]);
          if constexpr (OUT_BF16) {
            const bf16x2v lo = __builtin_convertvector((float2v){v[0], v[1]}, bf16x2v);
            const bf16x2v hi = __builtin_convertvector((float2v){v[2], v[3]}, bf16x2v);
            *reinterpret_cast<uint2 *>(region + l32 * kRowBytes + (((4 * jj + q) ^ (l32 & (NP - 1))) * 16 + 8 * h)) =
                make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
          } else {
            *reinterpret_cast<float4 *>(region + l32 * kRowBytes + ((8 * jj + 2 * q + h) ^ (l32 & (NP - 1))) * 16) =
                make_float4(v[0], v[1], v[2], v[3]);
          }
        }
      // the wave reads back its own rows (LDS accesses of one wave complete in order)
#pragma unroll
      for (uint32_t u = 0; u < 32 * NP / 64; ++u) {
        const uint32_t row = u * (64 / NP) + lane / NP, c = lane % NP;
        const uint4 v = *reinterpret_cast<const uint4 *>(region + row * kRowBytes + ((c ^ (row & (NP - 1))) * 16));
        const int64_t col = j0 * 32 + c * V;
        if (32 * i + row >= rows_left || col >= cols_left) continue;
        uint8_t *at = out + ((32 * i + row) * p.ldc + col) * ES;
        if (col + V <= cols_left) {
          __builtin_nontemporal_store((any_u32x4){v.x, v.y, v.z, v.w}, reinterpret_cast<any_u32x4 *>(at));
        } else {
          // (a loop, to keep this rare path's code short)
          uint64_t lo = v.x | static_cast<uint64_t>(v.y) << 32, hi = v.z | static_cast<uint64_t>(v.w) << 32;
#pragma clang loop unroll(disable)
          for (int64_t e = col; e < cols_left; ++e) {
            if constexpr (OUT_BF16)
              *reinterpret_cast<uint16_t *>(at) = static_cast<uint16_t>(lo);
            else
              *reinterpret_cast<uint32_t *>(at) = static_cast<uint32_t>(lo);
            at += ES;
            lo = lo >> (8 * ES) | hi << (64 - 8 * ES);
            hi >>= 8 * ES;
          }
        }
      }
    }
  }
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

  TileRows t;
  int32_t tn;
  const int32_t rows = count_rows<TM, kAllTiles>(p);
  int32_t tile;
  if (!deal(blockIdx.x, rows * p.tiles_n, tile) || !find_tile<TM, kAllTiles>(p, rows, tile, t, tn)) return;
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
    // all of the step's fragment reads go out before its first MFMA, which then waits for its own alone
    intx4 af[4][FM], bf[4][FN];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t pos = 16 * ((2 * s + h) ^ sw);
#pragma unroll
      for (int i = 0; i < FM; ++i) af[s][i] = *reinterpret_cast<const intx4 *>(st + rdA + 4096 * i + pos);
#pragma unroll
      for (int j = 0; j < FN; ++j) bf[s][j] = *reinterpret_cast<const intx4 *>(st + rdB + 4096 * j + pos);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bf[s][j], af[s][i], acc[j][i], 0, 0, 0);
    cur = cur + 1 == STAGES ? 0 : cur + 1;
  }

  // every wave is done with the stages
  wait_lgkmcnt0();
  lds_barrier();
  store_tile<FM, FN, OUT_BF16>(p, acc, smem + wave * kRegion, t, n0 + wn, wm, lane);
}

// Buffer descriptor over the bytes from p on (raw 32-bit data format, no limit below 4 GiB).
// The same in every lane: the read of lane 0's pointer only tells the compiler so.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t *p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint64_t u = static_cast<uint64_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32))) << 32 |
                     static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a)));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<uint8_t *>(u), 0, -1, 0x00020000);
}
// As lds_load16, from byte `off` (a lane's) + `step` (the wave's) of a buffer.
__device__ __forceinline__ void lds_buffer16(__amdgpu_buffer_rsrc_t rs, uint32_t off, uint32_t step, uint8_t *lds_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)lds_base, 16, off, step, 0, 0);
}

// ---- many rows: 256 x 256 tiles ---------------------------------------------------------------------
// Four waves of 128 x 128 (16 MFMA tiles, 256 accumulators a lane), one a SIMD.  K advances 128 bytes a
// step through two 64 KB stages: whole 128-byte lines, since the L2 serves one request a clock and
// channel whatever its size (with 64-byte rows its request rate was the bound).  A step has four
// sub-steps of 16 MFMAs; the fragments of the next sub-step are read under the MFMAs of this one, and
// the step's one barrier follows sub-step 2: there every fragment of the stage is in registers, so
// behind it the stage takes the loads of the step after next, and the next stage, whose loads this
// wave has waited for, is read.
constexpr int kBigLds = 3 * 384 * kStep;  // three stages of half tiles, or two of full ones

//
// HALF: 128 x 256 tiles, each wave all 128 rows by 64 columns (eight MFMAs a sub-step): half the work where a
// group's (or the matrix's) last tile row has at most 128 rows.  Such a tile has half the time a step to cover
// its loads: three stages of 48 KB, loaded two to three steps ahead.  (Lines fetched into the L2 some steps ahead, or
// weights by non-temporal loads, were no faster.)
template <bool OUT_BF16, bool HALF>
__device__ __forceinline__ void big_tile(const I8Args &p, uint8_t *smem, const TileRows &t, int32_t tn) {
  constexpr int FN = HALF ? 2 : 4;                       // B fragments a wave
  constexpr int NA = HALF ? 4 : 8, NL = NA + 8;          // direct loads a wave and step: of A, all
  constexpr int S = HALF ? 3 : 2;                        // stages
  constexpr uint32_t kB = 32 * NA * kStep, kStage = kB + 256 * kStep;
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t h = lane >> 5, l32 = lane & 31u;
  const uint32_t wm = HALF ? 0 : (wave >> 1) * 128, wn = HALF ? 64 * wave : (wave & 1) * 128;
  const int64_t n0 = static_cast<int64_t>(tn) * 256;
  // direct loads: wave w fetches rows [8 NA w, 8 NA (w + 1)) of A and [64 w, 64 w + 64) of B, 8 rows a load; rows beyond the
  // operand read its last one (their products are never stored).  Buffer loads: a lane's offset within
  // the operand stays in one register and the step's advance is a scalar, so a load takes no vector
  // arithmetic.  (Every address is inside the operand: the range check is not relied on.)
  const __amdgpu_buffer_rsrc_t rsA = buffer_of(p.rows ? p.a : p.a + t.m0 * p.K);
  const __amdgpu_buffer_rsrc_t rsB = buffer_of(p.b + (static_cast<int64_t>(t.group) * p.N + n0) * p.K);
  uint32_t off[NL];  // A, then B
  const auto row_of = [&](int q) { return (q < NA ? 8 * NA * wave + 8 * q : 64 * wave + 8 * (q - NA)) + (lane >> 3); };
  const auto chunk_of = [&](int q) { return ((lane & 7u) ^ swz(row_of(q))) * 16; };
#pragma unroll
  for (int q = 0; q < NL; ++q) {
    const uint32_t R = row_of(q);
    const int64_t r = min(t.m0 + R, t.m_end - 1);
    off[q] = (q < NA ? static_cast<uint32_t>(p.rows ? a_row(p, r) : r - t.m0)
                     : static_cast<uint32_t>(min(n0 + R, p.N - 1) - n0)) * p.K + chunk_of(q);
  }
  const int32_t steps = static_cast<int32_t>((p.K + kStep - 1) / kStep);
  const uint32_t rest = p.K - (steps - 1) * kStep;  // bytes of K in the last step
  // Each group starts elsewhere in K (integer sums have no order): tiles that began together would all read the
  // same columns of their weights, rows a power of two apart, from the same memory channels (42 experts of
  // 128 x 1536 x 4096: 73 -> 57 us).  Not where K ends within a step.
  const uint32_t turn = steps > 0 && rest == kStep ? static_cast<uint32_t>(t.group) * 7u % static_cast<uint32_t>(steps) : 0u;
  auto load = [&](uint8_t *st, int32_t kt, int q) {
    const int32_t at = kt + static_cast<int32_t>(turn);
    lds_buffer16(q < NA ? rsA : rsB, off[q], (at < steps ? at : at - steps) * kStep,
                 st + (q < NA ? (8 * NA * wave + 8 * q) * kStep : kB + (64 * wave + 8 * (q - NA)) * kStep));
  };
  // before the loads of a last step that K does not fill: chunks beyond K read its last one (their A
  // fragments are cleared)
  auto end_of_k = [&](int32_t kt) {
    if (kt == steps - 1 && rest < kStep) {
#pragma unroll
      for (int q = 0; q < NL; ++q) {
        const uint32_t chunk = chunk_of(q);
        off[q] -= chunk > rest - 16 ? chunk - (rest - 16) : 0;
      }
    }
  };

  intx16 acc[FN][4];  // [B fragment][A fragment]
#pragma unroll
  for (int j = 0; j < FN; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][i][r] = 0;

  const uint32_t rdA = (wm + l32) * kStep, rdB = kB + (wn + l32) * kStep, sw = swz(l32);
  intx4 a0[4], b0[FN], a1[4], b1[FN];  // fragments of the even and the odd sub-steps
  auto read = [&](const uint8_t *st, int s, intx4 (&af)[4], intx4 (&bf)[FN]) {
    const uint32_t pos = 16 * ((2 * s + h) ^ sw);
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      af[f] = *reinterpret_cast<const intx4 *>(st + rdA + 32 * kStep * f + pos);
      if (f < FN) bf[f] = *reinterpret_cast<const intx4 *>(st + rdB + 32 * kStep * f + pos);
    }
  };
  auto multiply = [&](const intx4 (&af)[4], const intx4 (&bf)[FN]) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bf[j], af[i], acc[j][i], 0, 0, 0);
  };
  // clears the A fragments of K beyond the end
  auto clear = [&](int32_t kt, int s, intx4 (&af)[4]) {
    const bool in = static_cast<uint32_t>(kt) * kStep + 16 * (2 * s + h) < p.K;
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e) af[f][e] = in ? af[f][e] : 0;
  };
  // an MFMA, then a fragment read, for every read, and the other MFMAs, under which the reads land
  auto order = [&]() {
#pragma unroll
    for (int q = 0; q < 4 + FN; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, HALF ? 2 : 8, 0);
  };

  if (steps > 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (s < steps) {
        end_of_k(s);
#pragma unroll
        for (int q = 0; q < NL; ++q) load(smem + s * kStage, s, q);
      }
    }
    if (steps >= S)
      wait_vmcnt<(S - 1) * NL>();
    else
      wait_vmcnt<0>();
    lds_barrier();
    read(smem, 0, a0, b0);
  }
  // One step out of stage cur, whose sub-step 0 is in a0, b0; then cur takes the loads of step kt + S.
  auto step = [&](uint8_t *__restrict__ cur, const uint8_t *__restrict__ nxt, int32_t kt) {
    end_of_k(kt + S);
    read(cur, 1, a1, b1);
    multiply(a0, b0);
    order();
    read(cur, 2, a0, b0);
    multiply(a1, b1);
    order();
    read(cur, 3, a1, b1);
    multiply(a0, b0);
    order();
    wait_vmcnt<(S - 2) * NL>();
    wait_lgkmcnt0();
    lds_barrier();
    read(nxt, 0, a0, b0);
#pragma unroll
    for (int q = 0; q < NL; ++q) load(cur, kt + S, q);
    multiply(a1, b1);
#pragma unroll
    for (int q = 0; q < 4 * FN; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (q < 4 + FN) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // a direct load
      if (HALF && q < 4) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
  };
  int32_t kt = 0;
  uint32_t cur = 0;
  const auto after = [](uint32_t st) { return st == (S - 1) * kStage ? 0 : st + kStage; };
#pragma clang loop unroll(disable)
  for (; kt + S < steps; ++kt) {
    step(smem + cur, smem + after(cur), kt);
    cur = after(cur);
  }
  // the last S steps: nothing left to load
#pragma clang loop unroll(disable)
  for (; kt < steps; ++kt) {
    const uint8_t *const st = smem + cur;
    read(st, 1, a1, b1);
    clear(kt, 0, a0);
    multiply(a0, b0);
    read(st, 2, a0, b0);
    clear(kt, 1, a1);
    multiply(a1, b1);
    read(st, 3, a1, b1);
    clear(kt, 2, a0);
    multiply(a0, b0);
    if (S > 2 && kt + 2 < steps)
      wait_vmcnt<NL>();
    else
      wait_vmcnt<0>();
    wait_lgkmcnt0();
    lds_barrier();
    cur = after(cur);
    if (kt + 1 < steps) read(smem + cur, 0, a0, b0);
    clear(kt, 3, a1);
    multiply(a1, b1);
  }

  // every wave is done with the stages
  wait_lgkmcnt0();
  lds_barrier();
  store_tile<4, FN, OUT_BF16>(p, acc, smem + wave * kRegion, t, n0 + wn, wm, lane);
}

// Full tiles that stay whole: all of them, or, where what exceeds whole rounds of 256 workgroups is at most a round of
// half tiles, the whole rounds'.  Half tiles run last.  32768 x 1536 x 4096 over 64 experts (3.4 rounds): 256 us with half
// tiles in between and none split, 245 so, against 183 for one expert; 16384 rows (1.9 rounds) 184 -> 150; plain 4096 x
// 6144 x 4096 (1.5 rounds) 104 -> 92.
__host__ __device__ inline int32_t kept_tiles(int32_t full, int32_t half) {
  const int64_t halves = 2ll * full + half;
  const int64_t whole = halves / 512 * 256;
  return halves % 512 <= 256 && whole < full ? static_cast<int32_t>(whole) : full;
}

template <bool OUT_BF16>
__global__ __launch_bounds__(kThreads, 1) void gemm_int8_big_kernel(I8Args p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kBigLds];
  TileRows t;
  int32_t tn;
  const int32_t full_rows = count_rows<256, kFullTiles>(p), half_rows = count_rows<256, kHalfTiles>(p);
  const int32_t full = full_rows * p.tiles_n, half = half_rows * p.tiles_n;
  // the last round, in half tiles: where all of its work fits one round of them, the full tiles of it are split
  const int32_t kept = kept_tiles(full, half), id = blockIdx.x, full_ids = (kept + 7) / 8 * 8;
  int32_t item;
  if (id < full_ids) {
    if (deal(id, kept, item) && find_tile<256, kFullTiles>(p, full_rows, item, t, tn))
      big_tile<OUT_BF16, false>(p, smem, t, tn);
    return;
  }
  if (!deal(id - full_ids, half + 2 * (full - kept), item)) return;
  if (item < half) {
    if (!find_tile<256, kHalfTiles>(p, half_rows, item, t, tn)) return;
  } else {
    if (!find_tile<256, kFullTiles>(p, full_rows, kept + (item - half) / 2, t, tn)) return;
    if ((item - half) & 1) t.m0 += 128;
    if (t.m0 >= t.m_end) return;  // (a full tile has more than 128 rows, unless offsets pass the rows)
  }
  big_tile<OUT_BF16, true>(p, smem, t, tn);
}

// ---- few rows: weight streaming -------------------------------------------------------------------------
// With few rows the product is bound by reading the weight once.  A workgroup owns 64 weight rows and
// 16 MT rows of its expert: both pass through a deep LDS ring of whole 128-byte lines (direct loads, so
// that the bytes in flight cost no registers), wave w multiplying weight rows [16 w, 16 w + 16) by all rows
// (v_mfma_i32_16x16x64_i8; lane l: row l mod 16, bytes 16 (l / 16) of every 64).  Where that leaves compute
// units without work (the plain form), the steps of K are split over grid.y, each split's integer sums go to the
// workspace, and a second kernel adds and scales them.  (By expert the grid's y is the expert and z its tile of rows.)
template <int MT>
struct Few {
  static constexpr int kRows = 16 * MT;
  static constexpr int kA = MT < 2 ? 1 : MT / 2;  // direct loads of A a wave and step (MT 1: two waves load the same)
  static constexpr int kLoads = kA + 2;
  static constexpr int kB = kRows * kStep, kStage = (kRows + 64) * kStep;
  static constexpr int kStages = MT <= 2 ? 6 : MT == 4 ? 5 : 6;  // MT <= 4: two workgroups share a compute unit's LDS
};

// Rows [m0, m0 + kRows) of C, up to m_end, of one group.
template <int MT, bool OUT_BF16, bool ONCE>
__device__ __forceinline__ void few_tile(const I8Args &p, uint8_t *smem, int32_t group, int64_t m0, int64_t m_end) {
  using F = Few<MT>;
  // (an opaque copy: what depends on the lane is not held in registers over further tiles)
  uint32_t tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const uint32_t lane = tid & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t r16 = lane & 15u, g = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 64;
  // this split's steps
  const int32_t all = static_cast<int32_t>((p.K + kStep - 1) / kStep);
  const int32_t kt0 = p.splits > 1 ? static_cast<int32_t>(blockIdx.y) * p.split_steps : 0;
  const int32_t steps = p.splits > 1 ? min(p.split_steps, all - kt0) : all;

  const uint8_t *srcA[F::kA], *srcB[2];
  uint32_t chunkA[F::kA], chunkB[2], dstA[F::kA];
#pragma unroll
  for (int i = 0; i < F::kA; ++i) {
    const uint32_t R0 = (8 * (F::kA * wave + i)) % F::kRows, R = R0 + (lane >> 3);
    dstA[i] = R0 * kStep;
    chunkA[i] = ((lane & 7u) ^ swz(R)) * 16;
    srcA[i] = p.a + a_row(p, min(m0 + R, m_end - 1)) * p.K;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t R = 16 * wave + 8 * i + (lane >> 3);
    chunkB[i] = ((lane & 7u) ^ swz(R)) * 16;
    srcB[i] = p.b + (static_cast<int64_t>(group) * p.N + min(n0 + R, p.N - 1)) * p.K;
  }
  auto load = [&](uint8_t *st, int32_t kt) {
    const uint32_t k0 = static_cast<uint32_t>(kt0 + kt) * kStep;
    const bool whole = k0 + kStep <= p.K;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t *from = srcB[i] + (whole || k0 + chunkB[i] < p.K ? k0 + chunkB[i] : 0);
      uint8_t *to = st + F::kB + (16 * wave + 8 * i) * kStep;
      if constexpr (ONCE)
        __builtin_amdgcn_global_load_lds((global_void *)from, (lds_void *)to, 16, 0, 2);  // (2: non-temporal)
      else
        lds_load16(from, to);
    }
#pragma unroll
    for (int i = 0; i < F::kA; ++i)
      lds_load16(whole || k0 + chunkA[i] < p.K ? srcA[i] + (k0 + chunkA[i]) : reinterpret_cast<const uint8_t *>(&kZeros),
                 st + dstA[i]);
  };
  intx4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = (intx4){0, 0, 0, 0};
  constexpr int kAhead = F::kStages - 1;
  for (int s = 0; s < kAhead && s < steps; ++s) load(smem + s * F::kStage, s);
  const uint32_t rdA = r16 * kStep, rdB = F::kB + (16 * wave + r16) * kStep, sw = swz(r16);
  int cur = 0;
  for (int32_t kt = 0; kt < steps; ++kt) {
    // this wave's loads of step kt have landed; after the barrier everyone's have, and the stage of
    // step kt - 1 is free
    if (kt + kAhead <= steps)
      wait_vmcnt<(kAhead - 1) * F::kLoads>();
    else
      wait_vmcnt<0>();
    wait_lgkmcnt0();
    lds_barrier();
    const int nxt = cur == 0 ? F::kStages - 1 : cur - 1;
    if (kt + kAhead < steps) load(smem + nxt * F::kStage, kt + kAhead);
    const uint8_t *st = smem + cur * F::kStage;
    intx4 w[2], a[2][MT];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t pos = 16 * ((4 * s + g) ^ sw);
      w[s] = *reinterpret_cast<const intx4 *>(st + rdB + pos);
#pragma unroll
      for (int i = 0; i < MT; ++i) a[s][i] = *reinterpret_cast<const intx4 *>(st + rdA + 16 * kStep * i + pos);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[s], a[s][i], acc[i], 0, 0, 0);
    cur = cur + 1 == F::kStages ? 0 : cur + 1;
  }
  // lane (r16, g) of tile i holds row 16 i + r16, columns 4 g + e
  const int64_t col = n0 + 16 * wave + 4 * g;
  if (col >= p.N) return;
  const float *sb = p.b_scales + static_cast<int64_t>(group) * p.N;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = m0 + 16 * i + r16;
    if (row >= m_end) continue;
    if (p.splits > 1) {
      // (the workspace's rows are padded to 64 columns)
      *reinterpret_cast<intx4 *>(p.partial + (static_cast<int64_t>(blockIdx.y) * p.M + row) * p.partial_ld + col) = acc[i];
      continue;
    }
    const float sa = p.a_scales[a_row(p, row)];
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(acc[i][e]) * (sa * sb[min(col + e, p.N - 1)]);
    store4<OUT_BF16>(p, row, col, v);
  }
}

template <int MT, bool OUT_BF16, bool ONCE>
__global__ __launch_bounds__(kThreads) void gemm_int8_few_kernel(I8Args p) {
  using F = Few<MT>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[F::kStages * F::kStage];
  const int32_t group = p.offsets ? blockIdx.y : 0;
  int64_t m0 = static_cast<int64_t>(blockIdx.z) * F::kRows, m_end = p.M;
  if (p.offsets) {
    const int64_t lo = p.offsets[group], hi = p.offsets[group + 1];
    m0 += lo;
    m_end = min(hi, p.M);
    if (lo < 0 || m0 >= m_end) return;
  }
  few_tile<MT, OUT_BF16, ONCE>(p, smem, group, m0, m_end);
  // An expert's rows beyond the grid's (a token may name an expert more than once, so there can be more rows than tokens):
  // this workgroup's further tiles of rows.  (The code of a tile twice: as one loop it took 1% more time where there is
  // one tile.)
  const int64_t further = static_cast<int64_t>(gridDim.z) * F::kRows;
  for (m0 += further; m0 < m_end; m0 += further) {  // (the same in every wave)
    // every wave is done with the stages
    wait_vmcnt<0>();
    wait_lgkmcnt0();
    lds_barrier();
    few_tile<MT, OUT_BF16, ONCE>(p, smem, group, m0, m_end);
  }
}

// C from the splits' sums: four columns a lane, a row of the grid a row.
template <bool OUT_BF16>
__global__ __launch_bounds__(kThreads) void int8_sum_kernel(I8Args p) {
  const int64_t row = blockIdx.y, col = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 4;
  if (col >= p.N) return;
  intx4 t = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s)
    t += *reinterpret_cast<const intx4 *>(p.partial + (s * p.M + row) * p.partial_ld + col);
  const float sa = p.a_scales[row];
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(t[e]) * (sa * p.b_scales[min(col + e, p.N - 1)]);
  store4<OUT_BF16>(p, row, col, v);
}

constexpr int64_t kMaxTiles = int64_t(1) << 23;  // workgroups of a launch

template <int TM, int TN>
hipError_t run_tiles(const Int8GemmArgs &a, I8Args p, void (*bf16_kernel)(I8Args), void (*f32_kernel)(I8Args)) {
  p.tiles_n = static_cast<int32_t>((a.N + TN - 1) / TN);
  // by expert: every group may have one partial tile row
  const int64_t rows = (a.M + TM - 1) / TM + (a.offsets ? a.num_groups : 0);
  // (256-row tiles: both kinds are dealt in eights, and up to 128 full ones are split)
  const int64_t tiles = (rows * p.tiles_n + 7) / 8 * 8 + (TM == 256 ? 8 + 128 : 0);
  if (tiles > kMaxTiles) return hipErrorInvalidValue;
  (a.c_dtype == 1 ? bf16_kernel : f32_kernel)<<<dim3(static_cast<uint32_t>(tiles)), dim3(kThreads), 0, a.stream>>>(p);
  return hipGetLastError();
}

// The tile for these sizes: 256 (256 x 256), 128 (128 x 128 in two stages, two workgroups a compute unit),
// 129 (128 x 128 in four stages, one workgroup a compute unit) or 64 (64 x 64).  The estimates are lines
// through measured times in us (fixed costs, and a time for every step of 128 bytes of K and every 256 tiles,
// e.g. 8192 x 4096 x 4096: 123 / 152 / 191 / 236; 1024 x 4096 x 14336: 160 / 103 / 81 / 117; 512 x 4096 x
// 4096: 48 / 27 / 24 / 18), within about a fifth of the measured times over such sizes.
int pick_tile(const Int8GemmArgs &a) {
  const double steps = static_cast<double>((a.K + kStep - 1) / kStep);
  const auto tiles = [&](int64_t t) {
    const int64_t rows = (a.M + t - 1) / t + (a.offsets ? a.num_groups / 2 : 0);
    return rows * ((a.N + t - 1) / t);
  };
  const auto rounds = [](int64_t t) { return static_cast<double>((t + 255) / 256); };
  const double t64 = rounds(tiles(64)) * (0.21 * steps + 0.5) + 3.5;
  const bool one = tiles(128) <= 256;
  const double t128 = one ? 0.65 * steps + 4 : rounds(tiles(128)) * (0.5 * steps + 2) + 3;
  // (a last round of half tiles takes 0.62 of one: kept_tiles)
  const int64_t last = tiles(256) % 256;
  const double r256 = static_cast<double>(tiles(256) / 256) + (last == 0 ? 0.0 : last <= 128 ? 0.62 : 1.0);
  const double t256 = r256 * (1.2 * steps + 6) + 6;
  // (a launch's tiles are bounded; larger tiles are fewer)
  const bool large = tiles(64) + (a.num_groups + 1) * ((a.N + 63) / 64) > kMaxTiles;
  if (large || (t256 < t128 && t256 < t64)) return 256;
  return t128 < t64 ? (one ? 129 : 128) : 64;
}

// ONCE: the weights are too large for the cache, so they are read past it.  All experts' bytes count, since which
// experts a call reads is known on the device alone and over some calls they all are (8 tokens, 8 of 64 experts of 1536 x 4096,
// 403 MB, about 40 of them read: 46 -> 40 us; 59 MB of weights with non-temporal loads 12.2 -> 13.1).
template <int MT, bool ONCE>
hipError_t run_few(const Int8GemmArgs &a, const I8Args &p, int64_t most) {
  const uint32_t tiles_n = static_cast<uint32_t>((a.N + 63) / 64), rows = static_cast<uint32_t>((most + 16 * MT - 1) / (16 * MT));
  // (rows last: further tiles of rows, which most experts do not have, start after all first ones)
  const dim3 grid(tiles_n, a.offsets ? a.num_groups : p.splits, rows);
  if (a.c_dtype == 1)
    gemm_int8_few_kernel<MT, true, ONCE><<<grid, dim3(kThreads), 0, a.stream>>>(p);
  else
    gemm_int8_few_kernel<MT, false, ONCE><<<grid, dim3(kThreads), 0, a.stream>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const dim3 sums(static_cast<uint32_t>((p.partial_ld / 4 + kThreads - 1) / kThreads), static_cast<uint32_t>(a.M));
  if (a.c_dtype == 1)
    int8_sum_kernel<true><<<sums, dim3(kThreads), 0, a.stream>>>(p);
  else
    int8_sum_kernel<false><<<sums, dim3(kThreads), 0, a.stream>>>(p);
  return hipGetLastError();
}

// Splits of K of the few-row kernel: towards one workgroup a compute unit, at least eight steps each, and only
// where the steps saved (0.28 us each) are worth the second kernel (3 us).
int few_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t steps = (K + kStep - 1) / kStep, tiles = (N + 63) / 64;
  if (M > 128 || steps < 24 || tiles > 128) return 1;
  const int64_t s = 256 / tiles, most = steps / 8;
  return static_cast<int>(s < most ? s : most);
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
  // rows an expert has at most where a token's experts differ: the kernel's tile and its grid.  (It takes any number of
  // rows; those of a token that names an expert more than once come one tile after the other.)
  const int64_t most = a.rows && a.a_rows < a.M ? a.a_rows : a.M;
  const int splits = !a.offsets && a.workspace ? few_splits(a.M, a.N, a.K) : 1;
  // (from 65 to 128 rows the few-row kernel pays only where it splits K: 100 x 4096 x 14336 24.5 us against 36
  // in 64 x 64 tiles, but 100 x 1000 x 1008 9.2 against 5.8)
  // By expert also where an expert has at most 24 rows on average, whatever it could have (64 experts of 1536 x 4096, 8 a
  // token: 65 tokens 90 -> 72 us, 128 tokens 93 -> 75, with falling loads 105 -> 83; 256 tokens, 32 rows each, 91 -> 82
  // with equal loads but 90 -> 101 with falling ones).
  if (most <= 64 || splits > 1 || (a.offsets && a.M <= 24ll * a.num_groups)) {
    const int steps = static_cast<int>((a.K + kStep - 1) / kStep);
    p.split_steps = (steps + splits - 1) / splits;
    p.splits = steps > 0 ? (steps + p.split_steps - 1) / p.split_steps : 1;
    p.partial = a.workspace;
    p.partial_ld = (a.N + 63) / 64 * 64;
    const auto few = [&](auto once) {
      constexpr bool kOnce = decltype(once)::value;
      if (most <= 16) return run_few<1, kOnce>(a, p, most);
      if (most <= 32) return run_few<2, kOnce>(a, p, most);
      if (most <= 64 || a.offsets) return run_few<4, kOnce>(a, p, most);
      return run_few<8, kOnce>(a, p, most);
    };
    return a.num_groups * a.N * a.K >= kStreamBytes ? few(std::true_type{}) : few(std::false_type{});
  }
  const int tile = pick_tile(a);
  if (tile == 256) return run_tiles<256, 256>(a, p, gemm_int8_big_kernel<true>, gemm_int8_big_kernel<false>);
  if (tile == 129) return run_tiles<128, 128>(a, p, gemm_int8_kernel<2, 2, 4, true>, gemm_int8_kernel<2, 2, 4, false>);
  if (tile == 128) return run_tiles<128, 128>(a, p, gemm_int8_kernel<2, 2, 2, true>, gemm_int8_kernel<2, 2, 2, false>);
  return run_tiles<64, 64>(a, p, gemm_int8_kernel<1, 1, 4, true>, gemm_int8_kernel<1, 1, 4, false>);
}

size_t int8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const int splits = few_splits(M, N, K);
  return splits > 1 ? static_cast<size_t>(splits) * M * ((N + 63) / 64 * 64) * sizeof(int32_t) : 0;
}

}  // namespace nvfp4
