// vec_io.hpp -- 16-byte pieces of fp32 or bf16 rows as fp32 values, and sums over a wave, shared by the
// kernels that stream rows (gather / combine, 8-bit quantize, block norms).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace nvfp4 {

typedef __bf16 vec_bf16x2 __attribute__((ext_vector_type(2)));
typedef float vec_f32x2 __attribute__((ext_vector_type(2)));

// Two fp32 values to packed bf16, nearest-even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((vec_f32x2){lo, hi}, vec_bf16x2));
}

// From this many bytes on (the Infinity Cache's 256 MiB) data cannot stay in it: what a call reads or multiplies of
// such data goes through non-temporal loads, which keep it from pushing out what the call writes.  Below, those
// loads cost time where the data is still cached.
constexpr int64_t kStreamBytes = int64_t(256) << 20;

typedef uint32_t vec_u32x4 __attribute__((ext_vector_type(4)));
template <bool ONCE>
__device__ __forceinline__ uint4 load16(const uint8_t *p) {
  if constexpr (ONCE) {
    const vec_u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const vec_u32x4 *>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
  } else {
    return *reinterpret_cast<const uint4 *>(p);
  }
}

// Eight consecutive elements from element index i (a multiple of 8) on.
template <bool BF16>
struct Raw8 {
  uint4 v[BF16 ? 1 : 2];
};
template <bool BF16, bool ONCE = false>
__device__ __forceinline__ Raw8<BF16> load8(const void *base, int64_t i) {
  Raw8<BF16> r;
  const uint8_t *p = static_cast<const uint8_t *>(base) + i * (BF16 ? 2 : 4);
  r.v[0] = load16<ONCE>(p);
  if constexpr (!BF16) r.v[1] = load16<ONCE>(p + 16);
  return r;
}
template <bool BF16>
__device__ __forceinline__ void unpack8(const Raw8<BF16> &r, float (&f)[8]) {
  if constexpr (BF16) {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = __uint_as_float(w[q] << 16);
      f[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
  } else {
    const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = __uint_as_float(w[q]);
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void *base, int64_t i, const float (&f)[8]) {
  uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(base) + i * (BF16 ? 2 : 4));
  if constexpr (BF16) {
    p[0] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  } else {
    p[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    p[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  const int b = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false));
}

// Sum / maximum over the wave's 64 lanes, in every lane, in one fixed order: within rows of 16 lanes by
// DPP, then across the four rows.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_move<0xB1>(v);   // 1 apart
  v += dpp_move<0x4E>(v);   // 2 apart
  v += dpp_move<0x141>(v);  // the other quad of eight
  v += dpp_move<0x140>(v);  // the other half of sixteen
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_move<0xB1>(v));
  v = fmaxf(v, dpp_move<0x4E>(v));
  v = fmaxf(v, dpp_move<0x141>(v));
  v = fmaxf(v, dpp_move<0x140>(v));
  v = fmaxf(v, __shfl_xor(v, 16));
  v = fmaxf(v, __shfl_xor(v, 32));
  return v;
}

}  // namespace nvfp4
