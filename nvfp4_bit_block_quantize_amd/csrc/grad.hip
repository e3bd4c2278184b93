// grad.hip -- the norm of many gradient tensors together, and their clipping to a largest norm.
//   norm = sqrt(sum g^2) or max |g|;   out = g * min(1, max_norm / (norm + eps))
// Both are one pass over the bytes (HBM-bound).  Tensors are cut into chunks of kChunk elements; a launch carries the
// addresses of up to kNormTensors (kClipTensors) tensors in its arguments, so that nothing has to be copied to the device
// first and a captured graph holds all it needs; each workgroup walks the launch's chunks and finds a chunk's tensor
// by bisection of the chunks' running counts.  Squares and their sums are 64-bit numbers: the square of any fp32 value
// is exact there and neither overflows nor vanishes, and the conversion and multiply-add still cost less than the
// loads.  A workgroup leaves one partial result, and one workgroup adds these in order: the same bits on every call.
// Eight bf16 tensors, 352 M elements: norm 107 to 110 us (704 MB, 6.5 TB/s: what of the last call's output the cache holds
// costs no reads), clipping into other tensors 256 to 264 us (1.41 GB, 5.4 TB/s; a 1 GiB copy runs at 5.1 to 5.2, an
// elementwise pass at 6.2).  160 fp32 tensors,
// 19 M elements: 15 + 2 + 25 us on the GPU; the walk over the list in Python and C takes 95.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "nvfp4_internal.h"
#include "vec_io.hpp"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kChunk = 16384;  // elements
// Launch arguments stay below 4096 bytes.
constexpr int kNormTensors = 240, kClipTensors = 160;
constexpr int64_t kMaxGroups = 2048;  // workgroups of a launch: eight a compute unit

struct NormBatch {
  const uint8_t *g[kNormTensors];
  uint32_t first[kNormTensors];  // number of the tensor's first chunk in this launch
  uint32_t last[kNormTensors];   // elements of its last chunk, and kBf16Bit
  uint32_t tensors, chunks;
};
struct ClipBatch {
  const uint8_t *g[kClipTensors];
  uint8_t *out[kClipTensors];
  uint32_t first[kClipTensors], last[kClipTensors];
  uint32_t tensors, chunks;
  const float *norm;
  float max_norm, eps;
};
constexpr int32_t kBf16 = 1;  // GradArgs::dtypes
constexpr uint32_t kBf16Bit = 1u << 31;
static_assert(sizeof(NormBatch) <= 4000 && sizeof(ClipBatch) <= 4000, "launch arguments");

// A chunk: its tensor, first element and number of elements.
struct Chunk {
  uint32_t tensor;
  int64_t at;
  uint32_t n;
  bool bf16;
};
template <class BATCH>
__device__ __forceinline__ Chunk find_chunk(const BATCH &p, uint32_t c) {
  uint32_t lo = 0, hi = p.tensors;  // first[lo] <= c < first[hi]
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (p.first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  const uint32_t next = lo + 1 < p.tensors ? p.first[lo + 1] : p.chunks;
  const uint32_t last = p.last[lo];
  return {lo, static_cast<int64_t>(c - p.first[lo]) * kChunk, c + 1 == next ? last & ~kBf16Bit : static_cast<uint32_t>(kChunk),
          (last & kBf16Bit) != 0};
}

// One value of a sum of squares, or of a maximum of magnitudes: as integers, so that NaN is above infinity.
template <bool MAX>
struct Fold {
  double sum = 0.0;
  uint32_t top = 0;
  __device__ __forceinline__ void add(float v) {
    if constexpr (MAX) {
      top = max(top, __float_as_uint(v) & 0x7FFFFFFFu);
    } else {
      const double d = static_cast<double>(v);
      sum = fma(d, d, sum);
    }
  }
};

__device__ __forceinline__ double wave_add(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = max(v, __shfl_xor(v, d));
  return v;
}

// `n` elements from `g` on, all threads of the workgroup.
template <bool MAX, bool BF16, bool ONCE>
__device__ __forceinline__ void fold_chunk(const uint8_t *g, uint32_t n, Fold<MAX> &f) {
  constexpr uint32_t V = BF16 ? 8 : 4, ES = 16 / V, U = 4;
  const uint32_t whole = n / V;
  for (uint32_t i0 = threadIdx.x; i0 < whole; i0 += U * kThreads) {
    any_u32x4 v[U];
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      const uint32_t i = i0 + u * kThreads;
      v[u] = (any_u32x4){0, 0, 0, 0};
      if (i < whole) {
        const any_u32x4 *at = reinterpret_cast<const any_u32x4 *>(g + static_cast<int64_t>(i) * 16);
        v[u] = ONCE ? __builtin_nontemporal_load(at) : *at;
      }
    }
#pragma unroll
    for (uint32_t u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (BF16) {
          f.add(__uint_as_float(v[u][q] << 16));
          f.add(__uint_as_float(v[u][q] & 0xFFFF0000u));
        } else {
          f.add(__uint_as_float(v[u][q]));
        }
      }
  }
  const uint32_t i = whole * V + threadIdx.x;
  if (threadIdx.x < V && i < n) {
    if constexpr (BF16)
      f.add(__uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(g)[i]) << 16));
    else
      f.add(reinterpret_cast<const float *>(g)[i]);
  }
  static_assert(ES == (BF16 ? 2 : 4), "");
}

template <bool MAX, bool ONCE>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(NormBatch p, double *partial) {
  __shared__ double part[kThreads / 64];
  Fold<MAX> f;
  for (uint32_t c = blockIdx.x; c < p.chunks; c += gridDim.x) {
    const Chunk k = find_chunk(p, c);
    const uint8_t *g = p.g[k.tensor] + k.at * (k.bf16 ? 2 : 4);
    if (k.bf16)
      fold_chunk<MAX, true, ONCE>(g, k.n, f);
    else
      fold_chunk<MAX, false, ONCE>(g, k.n, f);
  }
  const double v = MAX ? __longlong_as_double(wave_top(f.top)) : wave_add(f.sum);
  if ((threadIdx.x & 63u) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    double r = part[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w)
      r = MAX ? __longlong_as_double(max(__double_as_longlong(r), __double_as_longlong(part[w]))) : r + part[w];
    partial[blockIdx.x] = r;
  }
}

// The launches' partial results in one workgroup.  (Maxima are integers in a double's place.)
template <bool MAX>
__global__ __launch_bounds__(1024) void grad_norm_sum_kernel(const double *partial, int64_t n, float *norm) {
  __shared__ double part[16];
  double sum = 0.0;
  long long top = 0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) {
    if constexpr (MAX)
      top = max(top, __double_as_longlong(partial[i]));
    else
      sum += partial[i];
  }
  const double v = MAX ? __longlong_as_double(wave_top(static_cast<uint32_t>(top))) : wave_add(sum);
  if ((threadIdx.x & 63u) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    double r = part[0];
    for (int w = 1; w < 16; ++w)
      r = MAX ? __longlong_as_double(max(__double_as_longlong(r), __double_as_longlong(part[w]))) : r + part[w];
    *norm = MAX ? __uint_as_float(static_cast<uint32_t>(__double_as_longlong(r))) : static_cast<float>(sqrt(r));
  }
}

template <bool BF16, bool ONCE>
__device__ __forceinline__ void clip_chunk(const uint8_t *g, uint8_t *out, uint32_t n, float factor) {
  constexpr uint32_t V = BF16 ? 8 : 4, U = 4;
  const uint32_t whole = n / V;
  for (uint32_t i0 = threadIdx.x; i0 < whole; i0 += U * kThreads) {
    any_u32x4 v[U];
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      const uint32_t i = i0 + u * kThreads;
      v[u] = (any_u32x4){0, 0, 0, 0};
      if (i < whole) v[u] = *reinterpret_cast<const any_u32x4 *>(g + static_cast<int64_t>(i) * 16);
    }
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      const uint32_t i = i0 + u * kThreads;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (BF16)
          v[u][q] = pack_bf16(__uint_as_float(v[u][q] << 16) * factor, __uint_as_float(v[u][q] & 0xFFFF0000u) * factor);
        else
          v[u][q] = __float_as_uint(__uint_as_float(v[u][q]) * factor);
      }
      if (i < whole) {
        any_u32x4 *at = reinterpret_cast<any_u32x4 *>(out + static_cast<int64_t>(i) * 16);
        if constexpr (ONCE)
          __builtin_nontemporal_store(v[u], at);
        else
          *at = v[u];
      }
    }
  }
  const uint32_t i = whole * V + threadIdx.x;
  if (threadIdx.x < V && i < n) {
    if constexpr (BF16) {
      const float f = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(g)[i]) << 16) * factor;
      reinterpret_cast<uint16_t *>(out)[i] = static_cast<uint16_t>(pack_bf16(f, 0.0f));
    } else {
      reinterpret_cast<float *>(out)[i] = reinterpret_cast<const float *>(g)[i] * factor;
    }
  }
}

// Chunks are walked from the last: what the norm's pass read last may still be in the cache.
template <bool ONCE>
__global__ __launch_bounds__(kThreads) void grad_clip_kernel(ClipBatch p) {
  const float norm = *p.norm;
  // a norm that is no number leaves the gradients as they are
  float factor = isfinite(norm) ? p.max_norm / (norm + p.eps) : 1.0f;
  factor = factor < 1.0f ? factor : 1.0f;
  for (uint32_t i = blockIdx.x; i < p.chunks; i += gridDim.x) {
    const Chunk k = find_chunk(p, p.chunks - 1 - i);
    if (factor == 1.0f && p.g[k.tensor] == p.out[k.tensor]) continue;
    const int64_t at = k.at * (k.bf16 ? 2 : 4);
    if (k.bf16)
      clip_chunk<true, ONCE>(p.g[k.tensor] + at, p.out[k.tensor] + at, k.n, factor);
    else
      clip_chunk<false, ONCE>(p.g[k.tensor] + at, p.out[k.tensor] + at, k.n, factor);
  }
}

int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }
uint32_t last_of(int64_t n, int dtype) {
  return static_cast<uint32_t>(n - (chunks_of(n) - 1) * kChunk) | (dtype == kBf16 ? kBf16Bit : 0);
}
// Workgroups of a launch of `chunks` chunks: as many rounds as the largest number of workgroups needs, all of one length.
uint32_t groups_of(int64_t chunks) {
  const int64_t rounds = (chunks + kMaxGroups - 1) / kMaxGroups;
  return static_cast<uint32_t>((chunks + rounds - 1) / rounds);
}

// Calls launch(i0, i1, chunks) for runs of at most `most` tensors that are not empty and 2^31 chunks.
template <class F>
hipError_t in_batches(const GradArgs &a, int most, F &&launch) {
  int64_t i0 = 0, chunks = 0;
  int tensors = 0;
  for (int64_t i = 0; i < a.tensors; ++i) {
    const int64_t c = chunks_of(a.counts[i]);
    if (c == 0) continue;
    if (tensors == most || chunks + c >= (int64_t(1) << 31)) {
      const hipError_t e = launch(i0, i, chunks);
      if (e != hipSuccess) return e;
      i0 = i;
      chunks = 0;
      tensors = 0;
    }
    chunks += c;
    ++tensors;
  }
  return tensors ? launch(i0, a.tensors, chunks) : hipSuccess;
}

}  // namespace

size_t grad_workspace_bytes(int64_t tensors, int64_t elements) {
  // one partial result a workgroup: at most kMaxGroups a launch, and no more than there are chunks
  const int64_t chunks = elements / kChunk + tensors, launches = (tensors + kNormTensors - 1) / kNormTensors;
  const int64_t most = (launches + (chunks >> 31)) * kMaxGroups;
  return static_cast<size_t>(chunks < most ? chunks : most) * sizeof(double);
}

hipError_t launch_grad_norm(const GradArgs &a) {
  int64_t parts = 0, bytes = 0;
  for (int64_t i = 0; i < a.tensors; ++i) bytes += a.counts[i] * (a.dtypes[i] == kBf16 ? 2 : 4);
  const bool once = bytes >= kStreamBytes;
  const hipError_t e = in_batches(a, kNormTensors, [&](int64_t i0, int64_t i1, int64_t chunks) {
    NormBatch p;
    p.tensors = 0;
    p.chunks = 0;
    for (int64_t i = i0; i < i1; ++i) {
      if (a.counts[i] == 0) continue;
      p.g[p.tensors] = static_cast<const uint8_t *>(a.grads[i]);
      p.first[p.tensors] = p.chunks;
      p.last[p.tensors++] = last_of(a.counts[i], a.dtypes[i]);
      p.chunks += static_cast<uint32_t>(chunks_of(a.counts[i]));
    }
    const uint32_t groups = groups_of(chunks);
    auto *kernel = a.max ? (once ? grad_norm_kernel<true, true> : grad_norm_kernel<true, false>)
                         : (once ? grad_norm_kernel<false, true> : grad_norm_kernel<false, false>);
    kernel<<<dim3(groups), dim3(kThreads), 0, a.stream>>>(p, a.workspace + parts);
    parts += groups;
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  auto *kernel = a.max ? grad_norm_sum_kernel<true> : grad_norm_sum_kernel<false>;
  kernel<<<dim3(1), dim3(1024), 0, a.stream>>>(a.workspace, parts, a.norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradArgs &a) {
  int64_t bytes = 0;
  for (int64_t i = 0; i < a.tensors; ++i) bytes += a.counts[i] * (a.dtypes[i] == kBf16 ? 2 : 4);
  const bool once = bytes >= kStreamBytes;
  return in_batches(a, kClipTensors, [&](int64_t i0, int64_t i1, int64_t chunks) {
    ClipBatch p;
    p.tensors = 0;
    p.chunks = 0;
    for (int64_t i = i0; i < i1; ++i) {
      if (a.counts[i] == 0) continue;
      p.g[p.tensors] = static_cast<const uint8_t *>(a.grads[i]);
      p.out[p.tensors] = static_cast<uint8_t *>(a.outs[i]);
      p.first[p.tensors] = p.chunks;
      p.last[p.tensors++] = last_of(a.counts[i], a.dtypes[i]);
      p.chunks += static_cast<uint32_t>(chunks_of(a.counts[i]));
    }
    p.norm = a.norm;
    p.max_norm = a.max_norm;
    p.eps = a.eps;
    auto *kernel = once ? grad_clip_kernel<true> : grad_clip_kernel<false>;
    kernel<<<dim3(groups_of(chunks)), dim3(kThreads), 0, a.stream>>>(p);
    return hipGetLastError();
  });
}

}  // namespace nvfp4
