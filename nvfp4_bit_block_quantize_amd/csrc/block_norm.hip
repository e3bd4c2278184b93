// block_norm.hip -- the norms between two blocks, with gate and residual scale, and their gradients.
//
//   p = y r_y w_post,  x' = x + alpha g p,  n = x' r_x w_pre,  r_v = 1 / sqrt(mean(v^2) + eps)
//
// HBM-bound: a row of x and y is read once and stays in registers through both sums; x', n and the
// gradients are written once.  A row belongs to a wave (up to 1024 columns), to 256 or to 512 threads.
//
// Gradients, with yh = y r_y, xh = x' r_x, d = dL/dx' through both uses of x':
//   d  = dx' + r_x (w_pre dn - xh mean(w_pre dn xh)),          dx = d
//   dy = r_y (w_post q - yh mean(w_post q yh)),   q = alpha g d  (w_post NULL: dy = q)
//   dw_pre = sum dn xh,  dw_post = sum q yh,  dgate = sum alpha d p
// With a gate by channel both dw_post = g S and dgate = w_post S for S = sum alpha d yh, so two column
// sums serve three gradients.  A workgroup walks rows with its column sums in registers and leaves
// one partial row a sum; a second kernel adds the partial rows in order (no atomics: the bits do not
// depend on the schedule).
#include "nvfp4_internal.h"
#include "vec_io.hpp"

namespace nvfp4 {
namespace {

struct NormArgs {
  const void *x, *y;
  int64_t tokens;
  int d, pieces;
  const float *w_post;
  const float *gate_c;  // by channel
  const void *gate_t;   // by token, y's dtype
  const float *w_pre;
  float alpha, eps, shift;
  void *x_out, *n;
  float *rstd_post, *rstd_pre;
  const void *dx_out, *dn;
  void *dx, *dy, *dgate_t;
  float *parts;  // [2][parts][d]
};

// Sum over the T threads of a row (T == 64: a wave; else the workgroup, through `part`, which must not
// be in use by an earlier sum).
template <int T>
__device__ __forceinline__ float row_total(float v, float *part) {
  v = wave_sum(v);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63u) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < T / 64; w += 4) v += (part[w] + part[w + 1]) + (part[w + 2] + part[w + 3]);
  }
  return v;
}

__device__ __forceinline__ void load_factors(const float *w, int c, float shift, float (&f)[8]) {
  unpack8<false>(load8<false>(w, 8ll * c), f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] += shift;
}

// Factors of a lane's columns, loaded at once where they fit in registers (EARLY: their latency then
// hides behind the row's own loads) or when they are used.
template <int T, int NV, bool EARLY>
struct Factors {
  float v[EARLY ? NV : 1][8];
  const float *p;
  float shift;
  __device__ __forceinline__ Factors(const float *w, float s, int pieces) : p(w), shift(s) {
    if constexpr (EARLY) {
      const int tid = threadIdx.x % T;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (p && tid + T * i < pieces) load_factors(p, tid + T * i, shift, v[i]);
    }
  }
  __device__ __forceinline__ void get(int i, int c, float (&f)[8]) const {
    if constexpr (EARLY) {
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = v[i][q];
    } else {
      load_factors(p, c, shift, f);
    }
  }
};

template <bool XB, bool YB, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void block_norm_kernel(NormArgs p) {
  constexpr bool kEarly = NV <= 2 && T <= 256;
  constexpr int kRows = T < 256 ? 256 / T : 1;
  __shared__ float part[2][16];
  const int tid = threadIdx.x % T;
  const Factors<T, NV, kEarly> w_post(p.w_post, p.shift, p.pieces), gate(p.gate_c, 0.0f, p.pieces),
      w_pre(p.w_pre, p.shift, p.pieces);
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < p.tokens; r0 += gridDim.x * static_cast<int64_t>(kRows)) {
    const int64_t r = r0 + threadIdx.x / T;
    const bool live = r < p.tokens;
    const int64_t base = (live ? r : p.tokens - 1) * p.d;
    Raw8<XB> xr[NV];
    Raw8<YB> yr[NV], gr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + T * i;
      if (c < p.pieces) {
        xr[i] = load8<XB>(p.x, base + 8ll * c);
        if (p.y) yr[i] = load8<YB>(p.y, base + 8ll * c);
        if (p.gate_t) gr[i] = load8<YB>(p.gate_t, base + 8ll * c);
      }
    }
    float r_post = 1.0f;
    if (p.w_post) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (tid + T * i < p.pieces) {
          float y[8];
          unpack8<YB>(yr[i], y);
#pragma unroll
          for (int q = 0; q < 8; ++q) ss = fmaf(y[q], y[q], ss);
        }
      }
      ss = row_total<T>(ss, part[0]);
      r_post = 1.0f / sqrtf(ss / static_cast<float>(p.d) + p.eps);
      if (p.rstd_post && live && tid == 0) p.rstd_post[r] = r_post;
    }
    float x1[NV][8], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + T * i;
      if (c < p.pieces) {
        unpack8<XB>(xr[i], x1[i]);
        if (p.y) {
          float y[8], f[8];
          unpack8<YB>(yr[i], y);
          if (p.w_post) {
            w_post.get(i, c, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] = (y[q] * r_post) * f[q];
          }
          if (p.gate_t) {
            unpack8<YB>(gr[i], f);
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] *= f[q];
          } else if (p.gate_c) {
            gate.get(i, c, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] *= f[q];
          }
#pragma unroll
          for (int q = 0; q < 8; ++q) x1[i][q] = fmaf(p.alpha, y[q], x1[i][q]);
          if (live) store8<XB>(p.x_out, base + 8ll * c, x1[i]);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) ss = fmaf(x1[i][q], x1[i][q], ss);
      }
    }
    if (p.w_pre) {
      ss = row_total<T>(ss, part[1]);
      const float r_pre = 1.0f / sqrtf(ss / static_cast<float>(p.d) + p.eps);
      if (p.rstd_pre && live && tid == 0) p.rstd_pre[r] = r_pre;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + T * i;
        if (c < p.pieces && live) {
          float f[8], n[8];
          w_pre.get(i, c, f);
#pragma unroll
          for (int q = 0; q < 8; ++q) n[q] = (x1[i][q] * r_pre) * f[q];
          store8<YB>(p.n, base + 8ll * c, n);
        }
      }
    }
    if constexpr (T > 64) __syncthreads();  // the next row's sums reuse `part`
  }
}

template <bool XB, bool YB, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void block_norm_backward_kernel(NormArgs p) {
  constexpr int kRows = T < 256 ? 256 / T : 1;
  constexpr bool kEarly = NV <= 2 && T <= 256;
  __shared__ float part[2][16];
  const int tid = threadIdx.x % T;
  const Factors<T, NV, kEarly> w_post(p.w_post, p.shift, p.pieces), gate(p.gate_c, 0.0f, p.pieces),
      w_pre(p.w_pre, p.shift, p.pieces);
  float s_pre[NV][8], s_post[NV][8];  // column sums of this workgroup's (wave's) rows
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) s_pre[i][q] = s_post[i][q] = 0.0f;

  const float inv_d = 1.0f / static_cast<float>(p.d);
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < p.tokens; r0 += gridDim.x * static_cast<int64_t>(kRows)) {
    const int64_t r = r0 + threadIdx.x / T;
    if (T == 64 && r >= p.tokens) break;  // (a wave of its own: nothing waits for it)
    const int64_t base = r * p.d;
    Raw8<XB> xr[NV], dr[NV];
    Raw8<YB> yr[NV], nr[NV], gr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + T * i;
      if (c < p.pieces) {
        const int64_t at = base + 8ll * c;
        if (p.w_pre) {
          xr[i] = load8<XB>(p.x, at);
          nr[i] = load8<YB>(p.dn, at);
        }
        if (p.dx_out) dr[i] = load8<XB>(p.dx_out, at);
        if (p.y) yr[i] = load8<YB>(p.y, at);
        if (p.gate_t) gr[i] = load8<YB>(p.gate_t, at);
      }
    }
    const float r_post = p.w_post ? p.rstd_post[r] : 1.0f, r_pre = p.w_pre ? p.rstd_pre[r] : 0.0f;

    // the lane's factors of y: alpha g w_post, then the second norm's sum
    float xh[NV][8], c1 = 0.0f;
    if (p.w_pre) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + T * i;
        if (c < p.pieces) {
          float f[8], dn[8];
          unpack8<XB>(xr[i], xh[i]);
          if (p.y) {
            float y[8];
            unpack8<YB>(yr[i], y);
            if (p.w_post) {
              w_post.get(i, c, f);
#pragma unroll
              for (int q = 0; q < 8; ++q) y[q] = (y[q] * r_post) * f[q];
            }
            if (p.gate_t) {
              unpack8<YB>(gr[i], f);
#pragma unroll
              for (int q = 0; q < 8; ++q) y[q] *= f[q];
            } else if (p.gate_c) {
              gate.get(i, c, f);
#pragma unroll
              for (int q = 0; q < 8; ++q) y[q] *= f[q];
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) xh[i][q] = fmaf(p.alpha, y[q], xh[i][q]);
          }
          unpack8<YB>(nr[i], dn);
          w_pre.get(i, c, f);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            xh[i][q] *= r_pre;
            s_pre[i][q] = fmaf(dn[q], xh[i][q], s_pre[i][q]);
            c1 = fmaf(dn[q] * f[q], xh[i][q], c1);
          }
        }
      }
      c1 = row_total<T>(c1, part[0]) * inv_d;
    }
    float d[NV][8], c2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + T * i;
      if (c < p.pieces) {
        float f[8];
        if (p.dx_out) {
          unpack8<XB>(dr[i], d[i]);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) d[i][q] = 0.0f;
        }
        if (p.w_pre) {
          float dn[8];
          unpack8<YB>(nr[i], dn);
          w_pre.get(i, c, f);
#pragma unroll
          for (int q = 0; q < 8; ++q) d[i][q] = fmaf(r_pre, dn[q] * f[q] - xh[i][q] * c1, d[i][q]);
        }
        store8<XB>(p.dx, base + 8ll * c, d[i]);
        if (p.y) {
          // d becomes q = alpha g d, and with the first norm w_post q
          float yh[8], g[8], w[8];
          unpack8<YB>(yr[i], yh);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            yh[q] *= r_post;
            d[i][q] *= p.alpha;
            w[q] = 1.0f;
          }
          if (p.w_post) w_post.get(i, c, w);
          if (p.gate_t) {
            float dg[8];
            unpack8<YB>(gr[i], g);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              dg[q] = d[i][q] * (yh[q] * w[q]);
              d[i][q] *= g[q];
              s_post[i][q] = fmaf(d[i][q], yh[q], s_post[i][q]);
            }
            store8<YB>(p.dgate_t, base + 8ll * c, dg);
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) s_post[i][q] = fmaf(d[i][q], yh[q], s_post[i][q]);
            if (p.gate_c) {
              gate.get(i, c, g);
#pragma unroll
              for (int q = 0; q < 8; ++q) d[i][q] *= g[q];
            }
          }
          if (p.w_post) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              d[i][q] *= w[q];
              c2 = fmaf(d[i][q], yh[q], c2);
            }
          }
        }
      }
    }
    if (p.y) {
      if (p.w_post) c2 = row_total<T>(c2, part[1]) * inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + T * i;
        if (c < p.pieces) {
          if (p.w_post) {
            float yh[8];
            unpack8<YB>(yr[i], yh);
#pragma unroll
            for (int q = 0; q < 8; ++q) d[i][q] = r_post * (d[i][q] - (yh[q] * r_post) * c2);
          }
          store8<YB>(p.dy, base + 8ll * c, d[i]);
        }
      }
    }
    if constexpr (T > 64) __syncthreads();
  }
  const int64_t parts = static_cast<int64_t>(gridDim.x) * kRows;
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / T;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + T * i;
    if (c < p.pieces) {
      if (p.w_pre) store8<false>(p.parts, mine * p.d + 8ll * c, s_pre[i]);
      if (p.y) store8<false>(p.parts, (parts + mine) * p.d + 8ll * c, s_post[i]);
    }
  }
}

// Column sums of the partial rows: 16 lanes of four columns by 16 groups of rows, whose sums are added
// in the order of the groups.  grid.y = 0: dw_pre, 1: dw_post and dgate.
struct NormSumArgs {
  const float *parts;
  int64_t count;
  int d;
  float *dw_pre, *dw_post, *dgate_c;
  const float *w_post, *gate_c;
  float shift;
};
__global__ __launch_bounds__(256) void block_norm_sum_kernel(NormSumArgs p) {
  __shared__ float4 part[16][16];
  const int c = (blockIdx.x * 16 + (threadIdx.x & 15)) * 4, g = threadIdx.x >> 4;
  const bool second = blockIdx.y == 1;
  if (second ? (!p.dw_post && !p.dgate_c) : !p.dw_pre) return;
  const float *src = p.parts + (second ? p.count * p.d : 0);
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < p.d) {
#pragma unroll 4
    for (int64_t r = g; r < p.count; r += 16) {
      const float4 v = *reinterpret_cast<const float4 *>(src + r * p.d + c);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  part[g][threadIdx.x & 15] = s;
  __syncthreads();
  if (g != 0 || c >= p.d) return;
  for (int i = 1; i < 16; ++i) {
    const float4 v = part[i][threadIdx.x & 15];
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (!second) {
      p.dw_pre[c + q] = v[q];
    } else {
      if (p.dw_post) p.dw_post[c + q] = p.gate_c ? p.gate_c[c + q] * v[q] : v[q];
      if (p.dgate_c) p.dgate_c[c + q] = p.w_post ? (p.w_post[c + q] + p.shift) * v[q] : v[q];
    }
  }
}

NormArgs norm_args(const BlockNormArgs &a) {
  NormArgs p{};
  p.x = a.x;
  p.y = a.y;
  p.tokens = a.tokens;
  p.d = static_cast<int>(a.d);
  p.pieces = p.d / 8;
  p.w_post = a.w_post;
  p.gate_c = a.token_gate ? nullptr : static_cast<const float *>(a.gate);
  p.gate_t = a.token_gate ? a.gate : nullptr;
  p.w_pre = a.w_pre;
  p.alpha = a.alpha;
  p.eps = a.eps;
  p.shift = a.one_plus ? 1.0f : 0.0f;
  p.x_out = a.x_out;
  p.n = a.n;
  p.rstd_post = a.rstd_post;
  p.rstd_pre = a.rstd_pre;
  p.dx_out = a.dx_out;
  p.dn = a.dn;
  p.dx = a.dx;
  p.dy = a.dy;
  p.dgate_t = a.token_gate ? a.dgate : nullptr;
  p.parts = a.workspace;
  return p;
}

constexpr int64_t kForwardBlocks = int64_t(1) << 20;
constexpr int64_t kBackwardBlocks = 256;

// Rows a workgroup works on at once: four of up to 1024 columns.
int64_t rows_at_once(int64_t d) { return d <= 1024 ? 4 : 1; }
int64_t backward_blocks(int64_t tokens, int64_t d) {
  const int64_t n = (tokens + rows_at_once(d) - 1) / rows_at_once(d);
  return n < kBackwardBlocks ? n : kBackwardBlocks;
}

template <bool BWD, bool XB, bool YB, int T, int NV>
hipError_t go(const NormArgs &p, int64_t blocks, hipStream_t stream) {
  if constexpr (BWD)
    block_norm_backward_kernel<XB, YB, T, NV>
        <<<dim3(static_cast<uint32_t>(blocks)), dim3(T < 256 ? 256 : T), 0, stream>>>(p);
  else
    block_norm_kernel<XB, YB, T, NV><<<dim3(static_cast<uint32_t>(blocks)), dim3(T < 256 ? 256 : T), 0, stream>>>(p);
  return hipGetLastError();
}

template <bool BWD, bool XB, bool YB>
hipError_t run(const NormArgs &p, int64_t blocks, hipStream_t stream) {
  if (p.pieces <= 64) return go<BWD, XB, YB, 64, 1>(p, blocks, stream);
  if (p.pieces <= 128) return go<BWD, XB, YB, 64, 2>(p, blocks, stream);
  if (p.pieces <= 256) return go<BWD, XB, YB, 256, 1>(p, blocks, stream);
  if (p.pieces <= 512) return go<BWD, XB, YB, 256, 2>(p, blocks, stream);
  if (p.pieces <= 1024) return go<BWD, XB, YB, 256, 4>(p, blocks, stream);
  return go<BWD, XB, YB, 512, 4>(p, blocks, stream);
}

template <bool BWD>
hipError_t run_types(const BlockNormArgs &a, const NormArgs &p, int64_t blocks) {
  if (a.x_dtype == 1)
    return a.y_dtype == 1 ? run<BWD, true, true>(p, blocks, a.stream) : run<BWD, true, false>(p, blocks, a.stream);
  return a.y_dtype == 1 ? run<BWD, false, true>(p, blocks, a.stream) : run<BWD, false, false>(p, blocks, a.stream);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs &a) {
  const int64_t n = (a.tokens + rows_at_once(a.d) - 1) / rows_at_once(a.d);
  return run_types<false>(a, norm_args(a), n < kForwardBlocks ? n : kForwardBlocks);
}

size_t block_norm_workspace_bytes(int64_t tokens, int64_t d) {
  return static_cast<size_t>(2 * backward_blocks(tokens, d) * rows_at_once(d) * d) * sizeof(float);
}

hipError_t launch_block_norm_backward(const BlockNormArgs &a) {
  const NormArgs p = norm_args(a);
  const int64_t blocks = backward_blocks(a.tokens, a.d);
  if (blocks > 0) {
    const hipError_t e = run_types<true>(a, p, blocks);
    if (e != hipSuccess) return e;
  }
  NormSumArgs s{};
  s.parts = a.workspace;
  s.count = blocks * rows_at_once(a.d);  // (no rows: the sums are zero)
  s.d = p.d;
  s.dw_pre = a.dw_pre;
  s.dw_post = a.dw_post;
  s.dgate_c = a.token_gate ? nullptr : static_cast<float *>(a.dgate);
  s.w_post = a.w_post;
  s.gate_c = p.gate_c;
  s.shift = p.shift;
  if (!s.dw_pre && !s.dw_post && !s.dgate_c) return hipSuccess;
  block_norm_sum_kernel<<<dim3((p.d + 63) / 64, 2), dim3(256), 0, a.stream>>>(s);
  return hipGetLastError();
}

}  // namespace nvfp4
