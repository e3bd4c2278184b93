// block_norm.hip -- the norms between two blocks, with gate and residual scale, and their gradients.
//
//   p = y r_y w_post,  x' = x + alpha g p,  n = x' r_x w_pre,  r_v = 1 / sqrt(mean(v^2) + eps)
//
// HBM-bound: a row of x and y is read once and stays in registers through both sums; x', n and the
// gradients are written once.  A row belongs to a workgroup of 64 to 512 threads with one
// 8-column piece each (two above 4096 columns, four above 8192).
//
// Gradients, with yh = y r_y, xh = x' r_x, d = dL/dx' through both uses of x':
//   d  = dx' + r_x (w_pre dn - xh mean(w_pre dn xh)),          dx = d
//   dy = r_y (w_post q - yh mean(w_post q yh)),   q = alpha g d  (w_post NULL: dy = q)
//   dw_pre = sum dn xh,  dw_post = sum q yh,  dgate = sum alpha d p
// With a gate by channel both dw_post = g S and dgate = w_post S for S = sum alpha d yh, so two column
// sums serve three gradients.  A workgroup walks rows with its column sums in registers (LDS above
// 4096 columns) and leaves one partial row a sum; a second kernel adds the partial rows in order (no atomics: the bits do not
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

// Sums over the workgroup's T threads (one row), in one fixed order.  `part` must not be in use by earlier sums.
template <int T, int N>
__device__ __forceinline__ void row_totals(float (&v)[N], float (*part)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63u) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) part[threadIdx.x >> 6][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < T / 64; w += 2) v[i] += part[w][i] + part[w + 1][i];
    }
  }
}

// Factors of a lane's columns: in registers for the whole call (EARLY pieces a lane at most) or loaded at each use.
template <int T, int NV, int EARLY>
struct Factors {
  static constexpr bool kEarly = NV <= EARLY;
  float v[kEarly ? NV : 1][8];
  const float *p;
  float shift;
  __device__ __forceinline__ void load(int c, float (&f)[8]) const {
    unpack8<false>(load8<false>(p, 8ll * c), f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += shift;
  }
  __device__ __forceinline__ Factors(const float *w, float s, int pieces) : p(w), shift(s) {
    if constexpr (kEarly)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (p && static_cast<int>(threadIdx.x) + T * i < pieces) load(threadIdx.x + T * i, v[i]);
  }
  __device__ __forceinline__ void get(int i, float (&f)[8]) const {
    if constexpr (kEarly) {
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = v[i][q];
    } else {
      load(threadIdx.x + T * i, f);
    }
  }
};

// y (a piece of the block's output) to its share of x' - x without alpha: gate (y r_post w_post); yh: y r_post.
template <bool YB, class F>
__device__ __forceinline__ void block_output(const NormArgs &p, const F &w_post, const F &gate, const Raw8<YB> &gr, int i,
                                             float r_post, float (&y)[8]) {
  float f[8];
  if (p.w_post) {
    w_post.get(i, f);
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] = (y[q] * r_post) * f[q];
  }
  if (p.gate_t) {
    unpack8<YB>(gr, f);
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] *= f[q];
  } else if (p.gate_c) {
    gate.get(i, f);
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] *= f[q];
  }
}

// A workgroup a row at a time, NV pieces of 8 columns a thread; with one piece a thread the next row's loads go
// out before this row's sums.
template <bool XB, bool YB, int T, int NV, bool ONCE>
__global__ __launch_bounds__(T) void block_norm_kernel(NormArgs p) {
  __shared__ float part[2][16][1];
  const int tid = threadIdx.x;
  const Factors<T, NV, 1> w_post(p.w_post, p.shift, p.pieces), gate(p.gate_c, 0.0f, p.pieces),
      w_pre(p.w_pre, p.shift, p.pieces);
  auto fetch = [&](int64_t row, Raw8<XB> (&a)[NV], Raw8<YB> (&b)[NV], Raw8<YB> (&g)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + T * i;
      if (c < p.pieces) {
        if (p.y) b[i] = load8<YB, ONCE>(p.y, row * p.d + 8ll * c);
        a[i] = load8<XB, ONCE>(p.x, row * p.d + 8ll * c);
        if (p.gate_t) g[i] = load8<YB, ONCE>(p.gate_t, row * p.d + 8ll * c);
      }
    }
  };
  Raw8<XB> xr[NV];
  Raw8<YB> yr[NV], gr[NV];
  fetch(blockIdx.x, xr, yr, gr);
  for (int64_t r = blockIdx.x; r < p.tokens; r += gridDim.x) {
    const int64_t base = r * p.d;
    const bool more = NV == 1 && r + gridDim.x < p.tokens;
    Raw8<XB> nx[NV];
    Raw8<YB> ny[NV], ng[NV];
    if (more) fetch(r + gridDim.x, nx, ny, ng);
    float r_post = 1.0f;
    if (p.w_post) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (tid + T * i < p.pieces) {
          float y[8];
          unpack8<YB>(yr[i], y);
#pragma unroll
          for (int q = 0; q < 8; ++q) ss[0] = fmaf(y[q], y[q], ss[0]);
        }
      }
      row_totals<T>(ss, part[0]);
      r_post = 1.0f / sqrtf(ss[0] / static_cast<float>(p.d) + p.eps);
      if (p.rstd_post && tid == 0) p.rstd_post[r] = r_post;
    }
    float x1[NV][8], ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + T * i;
      if (c < p.pieces) {
        unpack8<XB>(xr[i], x1[i]);
        if (p.y) {
          float y[8];
          unpack8<YB>(yr[i], y);
          block_output<YB>(p, w_post, gate, gr[i], i, r_post, y);
#pragma unroll
          for (int q = 0; q < 8; ++q) x1[i][q] = fmaf(p.alpha, y[q], x1[i][q]);
          store8<XB>(p.x_out, base + 8ll * c, x1[i]);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) ss[0] = fmaf(x1[i][q], x1[i][q], ss[0]);
      }
    }
    if (p.w_pre) {
      row_totals<T>(ss, part[1]);
      const float r_pre = 1.0f / sqrtf(ss[0] / static_cast<float>(p.d) + p.eps);
      if (p.rstd_pre && tid == 0) p.rstd_pre[r] = r_pre;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + T * i;
        if (c < p.pieces) {
          float f[8], n[8];
          w_pre.get(i, f);
#pragma unroll
          for (int q = 0; q < 8; ++q) n[q] = (x1[i][q] * r_pre) * f[q];
          store8<YB>(p.n, base + 8ll * c, n);
        }
      }
    }
    if constexpr (T > 64) __syncthreads();  // the next row's sums reuse `part`
    if (more) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        xr[i] = nx[i];
        yr[i] = ny[i];
        gr[i] = ng[i];
      }
    } else if (r + gridDim.x < p.tokens) {
      fetch(r + gridDim.x, xr, yr, gr);
    }
  }
}

// A row's inputs of the backward pass.
template <bool XB, bool YB, int NV>
struct BackwardRow {
  Raw8<XB> x[NV], dx[NV];
  Raw8<YB> y[NV], dn[NV], gate[NV];
  float r_post, r_pre;
};
template <bool ONCE, int T, bool XB, bool YB, int NV>
__device__ __forceinline__ void load_row(const NormArgs &p, int64_t r, BackwardRow<XB, YB, NV> &v) {
  v.r_post = p.w_post ? p.rstd_post[r] : 1.0f;
  v.r_pre = p.w_pre ? p.rstd_pre[r] : 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + T * i;
    if (c < p.pieces) {
      const int64_t at = r * p.d + 8ll * c;
      if (p.w_pre) {
        v.x[i] = load8<XB, ONCE>(p.x, at);
        v.dn[i] = load8<YB, ONCE>(p.dn, at);
      }
      if (p.y) v.y[i] = load8<YB, ONCE>(p.y, at);
      if (p.dx_out) v.dx[i] = load8<XB, ONCE>(p.dx_out, at);
      if (p.gate_t) v.gate[i] = load8<YB, ONCE>(p.gate_t, at);
    }
  }
}

// Sums over a workgroup's rows of a lane's columns, two kinds: in registers with one piece a lane, else each lane's own
// 16-byte pieces in LDS, whose traffic is an eighth of what a row's time has room for.
template <int T, int NV>
struct ColumnSums {
  static constexpr bool kLds = NV > 1;
  static constexpr int kBytes = kLds ? 2 * NV * T * 32 : 16;
  float v[2][8];
  float4 *lds;
  __device__ __forceinline__ float4 &piece(int kind, int i, int half) const {
    return lds[((kind * NV + i) * 2 + half) * T + threadIdx.x];
  }
  __device__ __forceinline__ explicit ColumnSums(uint8_t *area) : lds(reinterpret_cast<float4 *>(area)) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[k][q] = 0.0f;
      if constexpr (kLds)
#pragma unroll
        for (int i = 0; i < 2 * NV; ++i) piece(k, i / 2, i & 1) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
  }
  __device__ __forceinline__ void get(int kind, int i, float (&s)[8]) const {
    if constexpr (kLds) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 w = piece(kind, i, h);
        s[4 * h] = w.x;
        s[4 * h + 1] = w.y;
        s[4 * h + 2] = w.z;
        s[4 * h + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] = v[kind][q];
    }
  }
  __device__ __forceinline__ void add(int kind, int i, const float (&a)[8], const float (&b)[8]) {
    float s[8];
    get(kind, i, s);
#pragma unroll
    for (int q = 0; q < 8; ++q) s[q] = fmaf(a[q], b[q], s[q]);
    if constexpr (kLds) {
#pragma unroll
      for (int h = 0; h < 2; ++h) piece(kind, i, h) = make_float4(s[4 * h], s[4 * h + 1], s[4 * h + 2], s[4 * h + 3]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[kind][q] = s[q];
    }
  }
};

// One barrier a row: with a = alpha g w_post yh, the second sum mean(a d) follows from three sums that need no
// other, mean(a d) = mean(a (dx' + r_x w_pre dn)) - r_x mean(w_pre dn xh) mean(a xh).  The loads
// of the next row (bf16 up to 4096 columns: of the next two, for as many bytes in flight) go out before this row's
// sums, up to 8192 columns; more would not fit in registers.  Measured with the column sums: 8192 x 4096 bf16 72 us,
// 5.6 TB/s (84 us before the loads were non-temporal, 97 us with one row ahead, 190 us with none and 16 columns a
// thread); 4096 x 8192 93 us, 4.3 TB/s (factors loaded at each use 105); 2048 x 16384 118 us, 3.4 TB/s (187 us with
// the column sums in registers, which spilled); fp32 4096 x 8192 174 us, 4.6 TB/s (factors in registers spill: 264).
template <bool XB, bool YB, int T, int NV, bool ONCE>
__global__ __launch_bounds__(T) void block_norm_backward_kernel(NormArgs p) {
  constexpr int kAhead = NV > 2 ? 0 : XB && YB && NV == 1 ? 2 : 1;
  __shared__ float part[2][16][3];
  __shared__ __attribute__((aligned(16))) uint8_t column_area[ColumnSums<T, NV>::kBytes];
  const int tid = threadIdx.x;
  const Factors<T, NV, XB && YB ? 2 : 1> w_post(p.w_post, p.shift, p.pieces), gate(p.gate_c, 0.0f, p.pieces),
      w_pre(p.w_pre, p.shift, p.pieces);
  ColumnSums<T, NV> columns(column_area);  // 0: of dn xh, 1: of q yh
  const float inv_d = 1.0f / static_cast<float>(p.d);
  BackwardRow<XB, YB, NV> row, next, after;
  int64_t r = blockIdx.x;  // (there are no more workgroups than rows)
  load_row<ONCE, T>(p, r, row);
  if constexpr (kAhead == 2)
    if (r + gridDim.x < p.tokens) load_row<ONCE, T>(p, r + gridDim.x, next);
  for (int turn = 0; r < p.tokens; r += gridDim.x, turn ^= 1) {
    const int64_t base = r * p.d;
    const bool more = r + gridDim.x < p.tokens;
    if constexpr (kAhead == 1)
      if (more) load_row<ONCE, T>(p, r + gridDim.x, next);
    if constexpr (kAhead == 2)
      if (r + 2ll * gridDim.x < p.tokens) load_row<ONCE, T>(p, r + 2ll * gridDim.x, after);
    const float r_post = row.r_post, r_pre = row.r_pre;
    float xh[NV][8], d[NV][8];  // x' r_pre; dx' + r_pre w_pre dn
    float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + T * i;
      if (c < p.pieces) {
        float f[8], a[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) d[i][q] = a[q] = 0.0f;
        if (p.dx_out) unpack8<XB>(row.dx[i], d[i]);
        if (p.y) {
          unpack8<YB>(row.y[i], a);
          block_output<YB>(p, w_post, gate, row.gate[i], i, r_post, a);
#pragma unroll
          for (int q = 0; q < 8; ++q) a[q] *= p.alpha;
        }
        if (p.w_pre) {
          float dn[8];
          unpack8<XB>(row.x[i], xh[i]);
          unpack8<YB>(row.dn[i], dn);
          w_pre.get(i, f);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            xh[i][q] = (xh[i][q] + a[q]) * r_pre;
            const float u = dn[q] * f[q];
            sums[0] = fmaf(u, xh[i][q], sums[0]);
            d[i][q] = fmaf(r_pre, u, d[i][q]);
            sums[2] = fmaf(a[q], xh[i][q], sums[2]);
          }
          columns.add(0, i, dn, xh[i]);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) sums[1] = fmaf(a[q], d[i][q], sums[1]);
      }
    }
    row_totals<T>(sums, part[turn]);  // (the other half of `part` may still be read)
    const float c1 = sums[0] * inv_d * r_pre, c2 = (sums[1] - c1 * sums[2]) * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + T * i;
      if (c < p.pieces) {
        if (p.w_pre) {
#pragma unroll
          for (int q = 0; q < 8; ++q) d[i][q] = fmaf(-c1, xh[i][q], d[i][q]);
        }
        store8<XB>(p.dx, base + 8ll * c, d[i]);
        if (p.y) {
          // d becomes q = alpha g d, then the gradient of y
          float yh[8], f[8];
          unpack8<YB>(row.y[i], yh);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            yh[q] *= r_post;
            d[i][q] *= p.alpha;
          }
          if (p.gate_t) {
            float dg[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) dg[q] = d[i][q] * yh[q];
            if (p.w_post) {
              w_post.get(i, f);
#pragma unroll
              for (int q = 0; q < 8; ++q) dg[q] *= f[q];
            }
            store8<YB>(p.dgate_t, base + 8ll * c, dg);
            unpack8<YB>(row.gate[i], f);
#pragma unroll
            for (int q = 0; q < 8; ++q) d[i][q] *= f[q];
          }
          columns.add(1, i, d[i], yh);
          if (p.gate_c) {
            gate.get(i, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) d[i][q] *= f[q];
          }
          if (p.w_post) {
            w_post.get(i, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) d[i][q] = r_post * fmaf(-c2, yh[q], d[i][q] * f[q]);
          }
          store8<YB>(p.dy, base + 8ll * c, d[i]);
        }
      }
    }
    if constexpr (kAhead > 0) {
      row = next;
      if constexpr (kAhead == 2) next = after;
    } else {
      if (more) load_row<ONCE, T>(p, r + gridDim.x, row);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + T * i;
    if (c < p.pieces) {
      float v[8];
      if (p.w_pre) {
        columns.get(0, i, v);
        store8<false>(p.parts, blockIdx.x * static_cast<int64_t>(p.d) + 8ll * c, v);
      }
      if (p.y) {
        columns.get(1, i, v);
        store8<false>(p.parts, (static_cast<int64_t>(gridDim.x) + blockIdx.x) * p.d + 8ll * c, v);
      }
    }
  }
}

// Column sums of the partial rows: 16 lanes of four columns by 64 groups of rows, whose sums are added
// in the order of the groups.  grid.y = 0: dw_pre, 1: dw_post and dgate.
struct NormSumArgs {
  const float *parts;
  int64_t count;
  int d;
  float *dw_pre, *dw_post, *dgate_c;
  const float *w_post, *gate_c;
  float shift;
};
__global__ __launch_bounds__(1024) void block_norm_sum_kernel(NormSumArgs p) {
  __shared__ float4 part[64][16];
  const int c = (blockIdx.x * 16 + (threadIdx.x & 15)) * 4, g = threadIdx.x >> 4;
  const bool second = blockIdx.y == 1;
  if (second ? (!p.dw_post && !p.dgate_c) : !p.dw_pre) return;
  const float *src = p.parts + (second ? p.count * p.d : 0);
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < p.d) {
#pragma unroll 8
    for (int64_t r = g; r < p.count; r += 64) {
      const float4 v = *reinterpret_cast<const float4 *>(src + r * p.d + c);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  part[g][threadIdx.x & 15] = s;
  __syncthreads();
  // the groups' sums in a tree
  for (int n = 32; n > 0; n /= 2) {
    if (g < n) {
      const float4 v = part[g + n][threadIdx.x & 15];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
      part[g][threadIdx.x & 15] = s;
    }
    __syncthreads();
  }
  if (g != 0 || c >= p.d) return;
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

// Workgroups of the backward pass: what the compute units hold at once (8 waves each), since each leaves a
// partial row that is written and read again (8192 x 4096: 96 us with 256, 98 with 512 before rows were
// fetched two ahead).
int64_t backward_blocks(int64_t tokens, int64_t d) {
  const int64_t n = d <= 512 ? 2048 : d <= 1024 ? 1024 : d <= 2048 ? 512 : 256;
  return tokens < n ? tokens : n;
}

template <bool BWD, bool XB, bool YB, bool ONCE, int T, int NV>
hipError_t go(const NormArgs &p, int64_t blocks, hipStream_t stream) {
  if constexpr (BWD)
    block_norm_backward_kernel<XB, YB, T, NV, ONCE><<<dim3(static_cast<uint32_t>(blocks)), dim3(T), 0, stream>>>(p);
  else
    block_norm_kernel<XB, YB, T, NV, ONCE><<<dim3(static_cast<uint32_t>(blocks)), dim3(T), 0, stream>>>(p);
  return hipGetLastError();
}

template <bool BWD, bool XB, bool YB, bool ONCE>
hipError_t run(const NormArgs &p, int64_t blocks, hipStream_t stream) {
  if (p.pieces <= 64) return go<BWD, XB, YB, ONCE, 64, 1>(p, blocks, stream);
  if (p.pieces <= 128) return go<BWD, XB, YB, ONCE, 128, 1>(p, blocks, stream);
  if (p.pieces <= 256) return go<BWD, XB, YB, ONCE, 256, 1>(p, blocks, stream);
  if (p.pieces <= 512) return go<BWD, XB, YB, ONCE, 512, 1>(p, blocks, stream);
  if (p.pieces <= 1024) return go<BWD, XB, YB, ONCE, 512, 2>(p, blocks, stream);
  return go<BWD, XB, YB, ONCE, 512, 4>(p, blocks, stream);
}

// Non-temporal loads where the forward pass's four matrices are too large for the cache: forward and backward of
// 8192 x 4096 bf16 132 -> 121 us, 16384 x 4096 258 -> 223, 65536 x 512 148 -> 138; with
// half the rows, 4096 x 4096, 63 -> 69.  Not for fp32, whose lanes read 32 bytes in two such loads (each half of a
// line then comes from the L2 twice: 258 -> 267).
template <bool BWD>
hipError_t run_types(const BlockNormArgs &a, const NormArgs &p, int64_t blocks) {
  const bool once = a.tokens * a.d * 8 >= kStreamBytes;
  if (a.x_dtype == 1 && a.y_dtype == 1)
    return once ? run<BWD, true, true, true>(p, blocks, a.stream) : run<BWD, true, true, false>(p, blocks, a.stream);
  if (a.x_dtype == 1) return run<BWD, true, false, false>(p, blocks, a.stream);
  return a.y_dtype == 1 ? run<BWD, false, true, false>(p, blocks, a.stream)
                        : run<BWD, false, false, false>(p, blocks, a.stream);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs &a) {
  // bf16 rows above 2048 columns: three workgroups a compute unit, which then fetch their next row ahead (8192 x
  // 4096: 50 us, 5.3 TB/s; a workgroup a row 59 us).  fp32 rows keep enough in flight by themselves (102 us
  // against 112), and shorter rows run more workgroups at once.
  const int64_t most = a.x_dtype == 1 && a.y_dtype == 1 && a.d > 2048 ? 768 : kForwardBlocks;
  return run_types<false>(a, norm_args(a), a.tokens < most ? a.tokens : most);
}

size_t block_norm_workspace_bytes(int64_t tokens, int64_t d) {
  return static_cast<size_t>(2 * backward_blocks(tokens, d) * d) * sizeof(float);
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
  s.count = blocks;  // (no rows: the sums are zero)
  s.d = p.d;
  s.dw_pre = a.dw_pre;
  s.dw_post = a.dw_post;
  s.dgate_c = a.token_gate ? nullptr : static_cast<float *>(a.dgate);
  s.w_post = a.w_post;
  s.gate_c = p.gate_c;
  s.shift = p.shift;
  if (!s.dw_pre && !s.dw_post && !s.dgate_c) return hipSuccess;
  block_norm_sum_kernel<<<dim3((p.d + 63) / 64, 2), dim3(1024), 0, a.stream>>>(s);
  return hipGetLastError();
}

}  // namespace nvfp4
