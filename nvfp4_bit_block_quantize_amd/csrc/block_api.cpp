// block_api.cpp -- C ABI front end of the operators around the quantized products (routing, plans, rows
// between tokens and experts, 8-bit integer products, block norms): argument validation on the host,
// then the kernel launchers.  As in nvfp4_api.cpp, validation never touches the GPU.
#pragma GCC visibility push(default)
#include "../../include/nvfp4.h"
#pragma GCC visibility pop

#include <hip/hip_runtime.h>

#include <cmath>

#include "nvfp4_internal.h"

namespace {

constexpr int64_t kMaxIndex32 = int64_t(1) << 32;
constexpr int64_t kMaxSlots = int64_t(1) << 31;
constexpr int64_t kMaxExperts = 512;
constexpr int32_t kMaxTopK = 32, kMaxGroups = 16;
constexpr int64_t kMaxNormColumns = 16384;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int dtype_size(int dt) { return dt == NVFP4_F32 ? 4 : (dt == NVFP4_BF16 ? 2 : 0); }
int status_of(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }
hipStream_t stream_of(void *s) { return static_cast<hipStream_t>(s); }

// a * b for non-negative factors, or -1 where it would pass 2^62.
int64_t product(int64_t a, int64_t b) {
  int64_t r;
  return __builtin_mul_overflow(a, b, &r) || r > (int64_t(1) << 62) ? -1 : r;
}

int check_slots(int64_t tokens, int64_t experts, int32_t top_k) {
  if (tokens < 0 || experts < 1 || experts > kMaxExperts || top_k < 1 || top_k > kMaxTopK) return NVFP4_ERR_SHAPE;
  const int64_t slots = product(tokens, top_k);
  return slots < 0 || slots >= kMaxSlots ? NVFP4_ERR_SHAPE : NVFP4_OK;
}

// Rows of d elements of size es: leading dimension and alignment of a 16-byte piece walk.
int check_rows(const void *p, int64_t d, int64_t ld, int es) {
  if (ld < d) return NVFP4_ERR_SHAPE;
  if (!p) return NVFP4_ERR_NULL;
  return !aligned(p, 16) || (ld * es) % 16 != 0 ? NVFP4_ERR_ALIGN : NVFP4_OK;
}

int check_moe_rows(int dtype, int64_t tokens, int64_t d, int32_t top_k) {
  const int es = dtype_size(dtype);
  if (es == 0) return NVFP4_ERR_UNSUPPORTED;
  const int st = check_slots(tokens, 1, top_k);
  if (st != NVFP4_OK) return st;
  if (d < 0 || d >= (int64_t(1) << 30)) return NVFP4_ERR_SHAPE;
  return (d * es) % 16 != 0 ? NVFP4_ERR_ALIGN : NVFP4_OK;
}

int check_route_common(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t ld, int32_t top_k) {
  const int es = dtype_size(dtype);
  if (es == 0) return NVFP4_ERR_UNSUPPORTED;
  const int st = check_slots(tokens, experts, top_k);
  if (st != NVFP4_OK) return st;
  if (top_k > experts || ld < experts || product(tokens, ld) < 0) return NVFP4_ERR_SHAPE;
  if (tokens > 0 && !logits) return NVFP4_ERR_NULL;
  return aligned(logits, es) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

int check_plan(int64_t tokens, int64_t experts, const int32_t *offsets, const int32_t *rows, const int32_t *pos,
               const void *workspace) {
  if (!offsets || (tokens > 0 && (!rows || !pos))) return NVFP4_ERR_NULL;
  if (nvfp4::moe_workspace_bytes(tokens, experts) > 0 && !workspace) return NVFP4_ERR_NULL;
  return aligned(offsets, 4) && aligned(rows, 4) && aligned(pos, 4) && aligned(workspace, 16) ? NVFP4_OK
                                                                                               : NVFP4_ERR_ALIGN;
}

int check_norm(const void *x, int x_dtype, const void *y, int y_dtype, int64_t tokens, int64_t d, const float *w_post,
               const void *gate, const float *w_pre, uint32_t flags) {
  if (dtype_size(x_dtype) == 0 || dtype_size(y_dtype) == 0 || (flags & ~(NVFP4_NORM_ONE_PLUS | NVFP4_NORM_TOKEN_GATE)))
    return NVFP4_ERR_UNSUPPORTED;
  if (tokens < 0 || d < 8 || d > kMaxNormColumns || d % 8 != 0 || product(tokens, d * 4) < 0) return NVFP4_ERR_SHAPE;
  // (without rows, matrices have no address)
  if (tokens > 0 && !y && (w_post || gate || !w_pre)) return NVFP4_ERR_UNSUPPORTED;
  if (tokens > 0 && !x) return NVFP4_ERR_NULL;
  return aligned(x, 16) && aligned(y, 16) && aligned(w_post, 16) && aligned(gate, 16) && aligned(w_pre, 16)
             ? NVFP4_OK
             : NVFP4_ERR_ALIGN;
}

}  // namespace

extern "C" {

size_t nvfp4_moe_workspace_size(int64_t tokens, int64_t experts, int32_t top_k) {
  (void)top_k;
  return tokens < 0 || experts < 1 || experts > kMaxExperts
             ? 0
             : (nvfp4::moe_workspace_bytes(tokens, experts) + 15) / 16 * 16;
}

int nvfp4_moe_route(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t ld, const float *bias,
                    int32_t num_groups, int32_t group_top_k, int32_t top_k, uint32_t flags, float scale, int32_t *ids,
                    float *weights, int32_t *offsets, int32_t *rows, int32_t *pos, void *workspace, void *hip_stream) {
  if (flags & ~(NVFP4_ROUTE_SIGMOID | NVFP4_ROUTE_RENORM | NVFP4_ROUTE_GROUP_SUM2)) return NVFP4_ERR_UNSUPPORTED;
  int st = check_route_common(logits, dtype, tokens, experts, ld, top_k);
  if (st != NVFP4_OK) return st;
  if (num_groups < 1 || num_groups > kMaxGroups || experts % num_groups != 0 || group_top_k < 1 ||
      group_top_k > num_groups || group_top_k * (experts / num_groups) < top_k)
    return NVFP4_ERR_SHAPE;
  if (tokens > 0 && (!ids || !weights)) return NVFP4_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(bias, 4)) return NVFP4_ERR_ALIGN;
  if (offsets || rows || pos) {
    st = check_plan(tokens, experts, offsets, rows, pos, workspace);
    if (st != NVFP4_OK) return st;
  }
  nvfp4::MoeRouteArgs a{};
  a.logits = logits;
  a.dtype = dtype == NVFP4_BF16 ? 1 : 0;
  a.tokens = tokens;
  a.experts = experts;
  a.ld = ld;
  a.bias = bias;
  a.num_groups = num_groups;
  a.group_top_k = group_top_k;
  a.top_k = top_k;
  a.sigmoid = flags & NVFP4_ROUTE_SIGMOID;
  a.renorm = flags & NVFP4_ROUTE_RENORM;
  a.sum2 = flags & NVFP4_ROUTE_GROUP_SUM2;
  a.scale = scale;
  a.ids = ids;
  a.weights = weights;
  a.offsets = offsets;
  a.rows = rows;
  a.pos = pos;
  a.workspace = static_cast<int32_t *>(workspace);
  a.stream = stream_of(hip_stream);
  return status_of(nvfp4::launch_moe_route(a));
}

int nvfp4_moe_route_backward(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t ld,
                             const int32_t *ids, const float *dweights, int32_t top_k, uint32_t flags, float scale,
                             void *dlogits, int64_t ldd, void *hip_stream) {
  if (flags & ~(NVFP4_ROUTE_SIGMOID | NVFP4_ROUTE_RENORM | NVFP4_ROUTE_GROUP_SUM2)) return NVFP4_ERR_UNSUPPORTED;
  const int st = check_route_common(logits, dtype, tokens, experts, ld, top_k);
  if (st != NVFP4_OK) return st;
  if (ldd < experts || product(tokens, ldd) < 0) return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  if (!ids || !dweights || !dlogits) return NVFP4_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(dweights, 4) || !aligned(dlogits, dtype_size(dtype))) return NVFP4_ERR_ALIGN;
  nvfp4::MoeRouteBackwardArgs a{};
  a.logits = logits;
  a.dtype = dtype == NVFP4_BF16 ? 1 : 0;
  a.tokens = tokens;
  a.experts = experts;
  a.ld = ld;
  a.ids = ids;
  a.dweights = dweights;
  a.top_k = top_k;
  a.sigmoid = flags & NVFP4_ROUTE_SIGMOID;
  a.renorm = flags & NVFP4_ROUTE_RENORM;
  a.scale = scale;
  a.dlogits = dlogits;
  a.ldd = ldd;
  a.stream = stream_of(hip_stream);
  return status_of(nvfp4::launch_moe_route_backward(a));
}

int nvfp4_moe_plan(const int32_t *ids, int64_t tokens, int32_t top_k, int64_t experts, int32_t *offsets, int32_t *rows,
                   int32_t *pos, void *workspace, void *hip_stream) {
  int st = check_slots(tokens, experts, top_k);
  if (st != NVFP4_OK) return st;
  if (tokens > 0 && !ids) return NVFP4_ERR_NULL;
  if (!aligned(ids, 4)) return NVFP4_ERR_ALIGN;
  st = check_plan(tokens, experts, offsets, rows, pos, workspace);
  if (st != NVFP4_OK) return st;
  return status_of(nvfp4::launch_moe_plan(ids, tokens * top_k, experts, offsets, rows, pos,
                                          static_cast<int32_t *>(workspace), stream_of(hip_stream)));
}

int nvfp4_moe_gather(const void *x, int dtype, int64_t tokens, int64_t d, int64_t ldx, const int32_t *rows,
                     int32_t top_k, void *y, int64_t ldy, void *hip_stream) {
  int st = check_moe_rows(dtype, tokens, d, top_k);
  if (st != NVFP4_OK) return st;
  if (ldx < d || ldy < d) return NVFP4_ERR_SHAPE;
  if (tokens == 0 || d == 0) return NVFP4_OK;
  const int es = dtype_size(dtype);
  if ((st = check_rows(x, d, ldx, es)) != NVFP4_OK || (st = check_rows(y, d, ldy, es)) != NVFP4_OK) return st;
  if (!rows) return NVFP4_ERR_NULL;
  if (!aligned(rows, 4)) return NVFP4_ERR_ALIGN;
  nvfp4::MoeRowsArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.dtype = dtype == NVFP4_BF16 ? 1 : 0;
  a.tokens = tokens;
  a.d = d;
  a.rows = rows;
  a.top_k = top_k;
  a.out = y;
  a.ldo = ldy;
  a.stream = stream_of(hip_stream);
  return status_of(nvfp4::launch_moe_gather(a));
}

int nvfp4_moe_combine(const void *y, int dtype, int64_t tokens, int64_t d, int64_t ldy, const int32_t *pos,
                      const float *weights, int32_t top_k, void *out, int64_t ldo, void *hip_stream) {
  int st = check_moe_rows(dtype, tokens, d, top_k);
  if (st != NVFP4_OK) return st;
  if (ldy < d || ldo < d) return NVFP4_ERR_SHAPE;
  if (tokens == 0 || d == 0) return NVFP4_OK;
  const int es = dtype_size(dtype);
  if ((st = check_rows(y, d, ldy, es)) != NVFP4_OK || (st = check_rows(out, d, ldo, es)) != NVFP4_OK) return st;
  if (!pos) return NVFP4_ERR_NULL;
  if (!aligned(pos, 4) || !aligned(weights, 4)) return NVFP4_ERR_ALIGN;
  nvfp4::MoeRowsArgs a{};
  a.x = y;
  a.ldx = ldy;
  a.dtype = dtype == NVFP4_BF16 ? 1 : 0;
  a.tokens = tokens;
  a.d = d;
  a.pos = pos;
  a.weights = weights;
  a.top_k = top_k;
  a.out = out;
  a.ldo = ldo;
  a.stream = stream_of(hip_stream);
  return status_of(nvfp4::launch_moe_combine(a));
}

int nvfp4_moe_combine_backward(const void *dout, int64_t ldo, const void *y, int64_t ldy, int dtype, int64_t tokens,
                               int64_t d, const int32_t *pos, const int32_t *rows, const float *weights, int32_t top_k,
                               void *dy, int64_t lddy, float *dweights, void *hip_stream) {
  int st = check_moe_rows(dtype, tokens, d, top_k);
  if (st != NVFP4_OK) return st;
  if (ldo < d || ldy < d || lddy < d || d == 0) return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  const int es = dtype_size(dtype);
  if ((st = check_rows(dout, d, ldo, es)) != NVFP4_OK || (st = check_rows(y, d, ldy, es)) != NVFP4_OK ||
      (st = check_rows(dy, d, lddy, es)) != NVFP4_OK)
    return st;
  if (!pos || !rows || !weights || !dweights) return NVFP4_ERR_NULL;
  if (!aligned(pos, 4) || !aligned(rows, 4) || !aligned(weights, 4) || !aligned(dweights, 4)) return NVFP4_ERR_ALIGN;
  nvfp4::MoeRowsArgs a{};
  a.x = y;
  a.ldx = ldy;
  a.dout = dout;
  a.ld_dout = ldo;
  a.dtype = dtype == NVFP4_BF16 ? 1 : 0;
  a.tokens = tokens;
  a.d = d;
  a.pos = pos;
  a.rows = rows;
  a.weights = weights;
  a.top_k = top_k;
  a.out = dy;
  a.ldo = lddy;
  a.dweights = dweights;
  a.stream = stream_of(hip_stream);
  return status_of(nvfp4::launch_moe_combine_backward(a));
}

int nvfp4_int8_quantize(const void *x, int dtype, int64_t rows, int64_t cols, int64_t ldx, int8_t *q, float *scales,
                        void *hip_stream) {
  const int es = dtype_size(dtype);
  if (es == 0) return NVFP4_ERR_UNSUPPORTED;
  if (rows < 0 || cols < 0 || cols % 16 != 0 || cols >= (int64_t(1) << 31) || ldx < cols || product(rows, ldx) < 0)
    return NVFP4_ERR_SHAPE;
  if (rows == 0) return NVFP4_OK;
  if (!scales || (cols > 0 && (!x || !q))) return NVFP4_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 4) || (ldx * es) % 16 != 0) return NVFP4_ERR_ALIGN;
  nvfp4::Int8QuantArgs a{x, dtype == NVFP4_BF16 ? 1 : 0, rows, cols, ldx, q, scales, stream_of(hip_stream)};
  return status_of(nvfp4::launch_int8_quantize(a));
}

size_t nvfp4_int8_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  return M < 1 || N < 1 || K < 1 || N >= kMaxSlots ? 0 : (nvfp4::int8_gemm_workspace_bytes(M, N, K) + 15) / 16 * 16;
}

int nvfp4_int8_gemm(const int8_t *a, const float *a_scales, int64_t a_rows, const int8_t *b, const float *b_scales,
                    int64_t M, int64_t N, int64_t K, void *c, int c_dtype, int64_t ldc, int32_t num_groups,
                    const int32_t *offsets, const int32_t *rows, int32_t row_div, void *workspace, void *hip_stream) {
  const int es = dtype_size(c_dtype);
  if (es == 0) return NVFP4_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || K < 0 || a_rows < 0 || K % 16 != 0 || K >= (int64_t(1) << 17) || M >= kMaxSlots ||
      a_rows >= kMaxSlots || N >= kMaxSlots || N * K >= kMaxIndex32 || ldc < N || ldc < 1 || product(M, ldc) < 0)
    return NVFP4_ERR_SHAPE;
  if (num_groups < 1 || num_groups > kMaxExperts || (num_groups > 1 && !offsets)) return NVFP4_ERR_SHAPE;
  if (rows ? (!offsets || row_div < 1 || a_rows * K >= kMaxIndex32) : a_rows != M) return NVFP4_ERR_SHAPE;
  if (M == 0 || N == 0) return NVFP4_OK;
  if (a_rows == 0) return NVFP4_ERR_SHAPE;
  if (!a_scales || !b_scales || !c || (K > 0 && (!a || !b))) return NVFP4_ERR_NULL;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scales, 4) || !aligned(b_scales, 4) || !aligned(c, es) ||
      !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  nvfp4::Int8GemmArgs g{};
  g.a = a;
  g.a_scales = a_scales;
  g.a_rows = a_rows;
  g.b = b;
  g.b_scales = b_scales;
  g.M = M;
  g.N = N;
  g.K = K;
  g.c = c;
  g.c_dtype = c_dtype == NVFP4_BF16 ? 1 : 0;
  g.ldc = ldc;
  g.num_groups = num_groups;
  g.offsets = offsets;
  g.rows = rows;
  g.row_div = row_div;
  g.workspace = static_cast<int32_t *>(workspace);
  g.stream = stream_of(hip_stream);
  return status_of(nvfp4::launch_int8_gemm(g));
}

int nvfp4_block_norm(const void *x, int x_dtype, const void *y, int y_dtype, int64_t tokens, int64_t d,
                     const float *w_post, const void *gate, const float *w_pre, float alpha, float eps,
                     uint32_t flags, void *x_out, void *n, float *rstd_post, float *rstd_pre, void *hip_stream) {
  const int st = check_norm(x, x_dtype, y, y_dtype, tokens, d, w_post, gate, w_pre, flags);
  if (st != NVFP4_OK) return st;
  if (!std::isnormal(eps) || eps < 0.0f) return NVFP4_ERR_UNSUPPORTED;
  if (tokens == 0) return NVFP4_OK;
  if (!y != !x_out || !w_pre != !n) return NVFP4_ERR_NULL;
  if (!aligned(x_out, 16) || !aligned(n, 16) || !aligned(rstd_post, 4) || !aligned(rstd_pre, 4)) return NVFP4_ERR_ALIGN;
  nvfp4::BlockNormArgs a{};
  a.x = x;
  a.y = y;
  a.x_dtype = x_dtype == NVFP4_BF16 ? 1 : 0;
  a.y_dtype = y_dtype == NVFP4_BF16 ? 1 : 0;
  a.tokens = tokens;
  a.d = d;
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.alpha = alpha;
  a.eps = eps;
  a.one_plus = flags & NVFP4_NORM_ONE_PLUS;
  a.token_gate = flags & NVFP4_NORM_TOKEN_GATE;
  a.x_out = x_out;
  a.n = n;
  a.rstd_post = rstd_post;
  a.rstd_pre = rstd_pre;
  a.stream = stream_of(hip_stream);
  return status_of(nvfp4::launch_block_norm(a));
}

size_t nvfp4_block_norm_workspace_size(int64_t tokens, int64_t d) {
  if (tokens < 0 || d < 8 || d > kMaxNormColumns) return 0;
  return (nvfp4::block_norm_workspace_bytes(tokens, d) + 15) / 16 * 16;
}

int nvfp4_block_norm_backward(const void *dx_out, const void *dn, const void *x, int x_dtype, const void *y,
                              int y_dtype, int64_t tokens, int64_t d, const float *w_post, const void *gate,
                              const float *w_pre, float alpha, uint32_t flags, const float *rstd_post,
                              const float *rstd_pre, void *dx, void *dy, float *dw_post, void *dgate, float *dw_pre,
                              void *workspace, void *hip_stream) {
  const int st = check_norm(x, x_dtype, y, y_dtype, tokens, d, w_post, gate, w_pre, flags);
  if (st != NVFP4_OK) return st;
  if (!w_post != !dw_post || !w_pre != !dw_pre || !gate != !dgate) return NVFP4_ERR_NULL;
  if (tokens > 0 && (!dx || !y != !dy || !w_pre != !dn || (w_post && !rstd_post) || (w_pre && !rstd_pre) || !workspace))
    return NVFP4_ERR_NULL;
  const void *const all[] = {dx_out, dn, dx, dy, dw_post, dgate, dw_pre, workspace};
  for (const void *p : all)
    if (!aligned(p, 16)) return NVFP4_ERR_ALIGN;
  if (!aligned(rstd_post, 4) || !aligned(rstd_pre, 4)) return NVFP4_ERR_ALIGN;
  nvfp4::BlockNormArgs a{};
  a.x = x;
  a.y = y;
  a.x_dtype = x_dtype == NVFP4_BF16 ? 1 : 0;
  a.y_dtype = y_dtype == NVFP4_BF16 ? 1 : 0;
  a.tokens = tokens;
  a.d = d;
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.alpha = alpha;
  a.one_plus = flags & NVFP4_NORM_ONE_PLUS;
  a.token_gate = flags & NVFP4_NORM_TOKEN_GATE;
  a.rstd_post = const_cast<float *>(rstd_post);
  a.rstd_pre = const_cast<float *>(rstd_pre);
  a.dx_out = dx_out;
  a.dn = dn;
  a.dx = dx;
  a.dy = dy;
  a.dgate = dgate;
  a.dw_post = dw_post;
  a.dw_pre = dw_pre;
  a.workspace = static_cast<float *>(workspace);
  a.stream = stream_of(hip_stream);
  return status_of(nvfp4::launch_block_norm_backward(a));
}

}  // extern "C"
