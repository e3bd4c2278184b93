// int8_quantize.hip -- rows of fp32 / bf16 to 8-bit integers, one fp32 scale a row: s = RN(amax * RN(1 / 127)),
// q = rint(RN(x * RN(1 / s))).  HBM-bound: a row is read once and stays in registers between its
// maximum and its encode (rows too long for that are read again, from the cache).  Rounding to the
// nearest integer, ties to even, is the addition of 1.5 * 2^23, whose sum holds q in its low byte
// (|x / s| < 128, so the addition is exact up to that rounding).  8192 x 4096 bf16 from HBM: 20 us, 5.0 TB/s (a 1
// GiB copy: 5.1), 8192 x 14336: 71 us, 4.9 TB/s; 65536 x 512: 21 us, 4.8 TB/s.
#include "nvfp4_internal.h"
#include "vec_io.hpp"

namespace nvfp4 {
namespace {

constexpr float kTiny = 1.17549435e-38f;  // 2^-126

__device__ __forceinline__ float absmax8(const float (&f)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}

__device__ __forceinline__ uint2 encode8(const float (&f)[8], float inv) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(f[i] * inv + 12582912.0f);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000C0Cu);
    w[h] = lo | hi;
  }
  return make_uint2(w[0], w[1]);
}

// T threads a row (64: four rows a workgroup), NV pieces of 8 elements a thread in registers (NV == 0: any row
// length, read twice).
template <bool BF16, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void int8_quantize_kernel(const void *x, int64_t rows, int64_t cols, int64_t ldx,
                                                            int8_t *q, float *scales) {
  constexpr int kRows = T < 256 ? 256 / T : 1;
  __shared__ float part[16];
  const uint32_t tid = threadIdx.x % T;
  const int pieces = static_cast<int>(cols / 8);
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < rows; r0 += gridDim.x * static_cast<int64_t>(kRows)) {
    const int64_t r = r0 + threadIdx.x / T;
    const bool live = r < rows;
    const int64_t row = live ? r : rows - 1;
    const uint8_t *xr = static_cast<const uint8_t *>(x) + row * ldx * (BF16 ? 2 : 4);
    Raw8<BF16> raw[NV > 0 ? NV : 1];
    float m = 0.0f;
    if constexpr (NV > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + T * i;
        if (c < pieces) raw[i] = load8<BF16>(xr, 8ll * c);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (static_cast<int>(tid + T * i) < pieces) {
          float f[8];
          unpack8<BF16>(raw[i], f);
          m = fmaxf(m, absmax8(f));
        }
      }
    } else {
      for (int c = tid; c < pieces; c += T) {
        float f[8];
        unpack8<BF16>(load8<BF16>(xr, 8ll * c), f);
        m = fmaxf(m, absmax8(f));
      }
    }
    m = wave_max(m);
    if constexpr (T >= 256) {
      if ((threadIdx.x & 63u) == 0) part[threadIdx.x >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < T / 64; ++w) m = fmaxf(m, part[w]);
      __syncthreads();
    }
    if (!live) continue;  // (only with T == 64, where nothing waits for this wave)
    const float s = m * (1.0f / 127.0f);
    const bool zero = !(s >= kTiny);
    const float inv = zero ? 0.0f : 1.0f / s;
    if (tid == 0) scales[r] = zero ? 0.0f : s;
    int8_t *qr = q + r * cols;
    if constexpr (NV > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + T * i;
        if (c < pieces) {
          float f[8];
          unpack8<BF16>(raw[i], f);
          *reinterpret_cast<uint2 *>(qr + 8ll * c) = encode8(f, inv);
        }
      }
    } else {
      for (int c = tid; c < pieces; c += T) {
        float f[8];
        unpack8<BF16>(load8<BF16>(xr, 8ll * c), f);
        *reinterpret_cast<uint2 *>(qr + 8ll * c) = encode8(f, inv);
      }
    }
  }
}

template <bool BF16>
hipError_t run(const Int8QuantArgs &a) {
  const int64_t pieces = a.cols / 8;
  auto go = [&](auto *kernel, int threads_per_row) {
    const int64_t per_block = threads_per_row < 256 ? 256 / threads_per_row : 1;
    const int64_t blocks = (a.rows + per_block - 1) / per_block;
    // (a grid of 2^32 threads or more does not launch: a workgroup walks several rows then)
    kernel<<<dim3(static_cast<uint32_t>(blocks < (1 << 20) ? blocks : 1 << 20)),
             dim3(threads_per_row < 256 ? 256 : threads_per_row), 0, a.stream>>>(a.x, a.rows, a.cols, a.ldx, a.q, a.scales);
    return hipGetLastError();
  };
  // a few long rows: as many threads a row as there are, since only the latency of a row counts (37 x 14336: 3.5 us,
  // with 256 threads a row 6.0)
  if (a.rows <= 256 && pieces > 256) {
    if (pieces <= 1024) return go(int8_quantize_kernel<BF16, 1024, 1>, 1024);
    if (pieces <= 2048) return go(int8_quantize_kernel<BF16, 1024, 2>, 1024);
    if (pieces <= 4096) return go(int8_quantize_kernel<BF16, 1024, 4>, 1024);
  }
  // rows of up to 1024 elements: a wave each, so that short rows still fill their lanes
  if (pieces <= 64) return go(int8_quantize_kernel<BF16, 64, 1>, 64);
  if (pieces <= 128) return go(int8_quantize_kernel<BF16, 64, 2>, 64);
  if (pieces <= 256) return go(int8_quantize_kernel<BF16, 256, 1>, 256);
  if (pieces <= 512) return go(int8_quantize_kernel<BF16, 256, 2>, 256);
  if (pieces <= 1024) return go(int8_quantize_kernel<BF16, 256, 4>, 256);
  if (pieces <= 2048) return go(int8_quantize_kernel<BF16, 256, 8>, 256);
  return go(int8_quantize_kernel<BF16, 256, 0>, 256);
}

}  // namespace

hipError_t launch_int8_quantize(const Int8QuantArgs &a) { return a.dtype == 1 ? run<true>(a) : run<false>(a); }

}  // namespace nvfp4
