// tune_api.cpp -- C ABI front end of the operators of fine-tuning beside the quantized products (adapters,
// balance loss, gradient norm and clipping): argument validation on the host, then the kernel launchers.  As in
// nvfp4_api.cpp, validation never touches the GPU.
#pragma GCC visibility push(default)
#include "../../include/nvfp4.h"
#pragma GCC visibility pop

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "nvfp4_internal.h"

namespace {

constexpr int64_t kMaxSlots = int64_t(1) << 31;
constexpr int64_t kMaxExperts = 512, kMaxSequences = 65535;
constexpr int32_t kMaxTopK = 32;
constexpr int32_t kMaxRank = 128;
constexpr int64_t kMaxWidth = int64_t(1) << 24;
constexpr int64_t kMaxElements = int64_t(1) << 40, kMaxTensors = int64_t(1) << 20;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int dtype_size(int dt) { return dt == NVFP4_F32 ? 4 : (dt == NVFP4_BF16 ? 2 : 0); }
int status_of(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

// a * b for non-negative factors, or -1 where it would pass 2^62.
int64_t product(int64_t a, int64_t b) {
  int64_t r;
  return __builtin_mul_overflow(a, b, &r) || r > (int64_t(1) << 62) ? -1 : r;
}

int check_balance(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t ld, const int32_t *ids,
                  int32_t top_k, int64_t sequences, uint32_t flags, float coef) {
  const int es = dtype_size(dtype);
  if (es == 0 || (flags & ~(NVFP4_ROUTE_SIGMOID | NVFP4_ROUTE_RENORM | NVFP4_ROUTE_GROUP_SUM2)) || !std::isfinite(coef))
    return NVFP4_ERR_UNSUPPORTED;
  if (tokens < 0 || experts < 1 || experts > kMaxExperts || top_k < 1 || top_k > kMaxTopK || top_k > experts ||
      ld < experts || product(tokens, ld) < 0 || sequences < 1 || sequences > kMaxSequences || tokens % sequences != 0)
    return NVFP4_ERR_SHAPE;
  const int64_t slots = product(tokens, top_k);
  if (slots < 0 || slots >= kMaxSlots) return NVFP4_ERR_SHAPE;
  if (tokens > 0 && (!logits || !ids)) return NVFP4_ERR_NULL;
  return aligned(logits, es) && aligned(ids, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

int check_grads(const void *const *grads, const int64_t *counts, const int32_t *dtypes, int64_t tensors) {
  if (tensors < 0 || tensors > kMaxTensors) return NVFP4_ERR_SHAPE;
  if (tensors > 0 && (!grads || !counts || !dtypes)) return NVFP4_ERR_NULL;
  int64_t all = 0;
  for (int64_t i = 0; i < tensors; ++i) {
    const int es = dtype_size(dtypes[i]);
    if (es == 0) return NVFP4_ERR_UNSUPPORTED;
    if (counts[i] < 0 || counts[i] > kMaxElements || (all += counts[i]) > kMaxElements) return NVFP4_ERR_SHAPE;
    if (counts[i] > 0 && !grads[i]) return NVFP4_ERR_NULL;
    if (!aligned(grads[i], es)) return NVFP4_ERR_ALIGN;
  }
  return NVFP4_OK;
}

// Whether any two of the ranges of bytes that a clip reads or writes overlap, an in-place tensor being one range.
struct Range {
  uintptr_t lo, hi;
};
bool before(const Range &a, const Range &b) { return a.lo < b.lo; }
int check_overlap(const void *const *grads, void *const *outs, const int64_t *counts, const int32_t *dtypes,
                  int64_t tensors) {
  try {
    // (both lists are often in the order of their addresses already)
    std::vector<Range> all, other;
    all.reserve(2 * tensors);
    other.reserve(tensors);
    for (int64_t i = 0; i < tensors; ++i) {
      if (counts[i] == 0) continue;
      const uintptr_t bytes = static_cast<uintptr_t>(counts[i]) * dtype_size(dtypes[i]);
      const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]), o = reinterpret_cast<uintptr_t>(outs[i]);
      all.push_back({g, g + bytes});
      if (o != g) other.push_back({o, o + bytes});
    }
    if (!std::is_sorted(all.begin(), all.end(), before)) std::sort(all.begin(), all.end(), before);
    if (!std::is_sorted(other.begin(), other.end(), before)) std::sort(other.begin(), other.end(), before);
    const size_t first = all.size();
    all.insert(all.end(), other.begin(), other.end());
    std::inplace_merge(all.begin(), all.begin() + first, all.end(), before);
    for (size_t i = 1; i < all.size(); ++i)
      if (all[i].lo < all[i - 1].hi) return NVFP4_ERR_UNSUPPORTED;
  } catch (const std::bad_alloc &) {
    return NVFP4_ERR_SHAPE;
  }
  return NVFP4_OK;
}

// What the forward and backward calls of an adapter share.  ldo, es: of the output and its dtype.
int check_adapter(const nvfp4::AdapterArgs &a, int x_dtype, int out_dtype, uint32_t flags) {
  if (x_dtype != NVFP4_BF16 || dtype_size(out_dtype) == 0 || (flags & ~(NVFP4_ADAPTER_GATHER | NVFP4_ADAPTER_BY_TOKEN)) ||
      (a.gather && a.by_token))
    return NVFP4_ERR_UNSUPPORTED;
  if (a.M < 0 || a.M >= kMaxSlots || a.x_rows < 0 || a.x_rows >= kMaxSlots || a.N < 1 || a.N > kMaxWidth || a.K < 8 ||
      a.K > kMaxWidth || a.K % 8 != 0 || a.rank < 8 || a.rank > kMaxRank || a.rank % 8 != 0 || a.adapters < 1 ||
      a.adapters > kMaxExperts || a.ldx < a.K || product(a.x_rows, a.ldx) < 0)
    return NVFP4_ERR_SHAPE;
  if (!a.offsets && (a.adapters != 1 || flags)) return NVFP4_ERR_SHAPE;
  if (a.gather ? a.row_div < 1 : a.x_rows != a.M) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}
// Their pointers, for M > 0.
int check_adapter_pointers(const nvfp4::AdapterArgs &a, int out_dtype, size_t workspace_bytes) {
  if ((a.x_rows > 0 && !a.x) || !a.a || !a.b || !a.scales || !a.c || (workspace_bytes > 0 && !a.workspace)) return NVFP4_ERR_NULL;
  if ((a.gather || a.by_token) && !a.rows) return NVFP4_ERR_NULL;
  if (a.by_token && !a.pos) return NVFP4_ERR_NULL;
  const int es = dtype_size(out_dtype);
  if (!aligned(a.x, 16) || a.ldx % 8 != 0 || !aligned(a.a, 16) || !aligned(a.b, 16) || !aligned(a.scales, 4) ||
      !aligned(a.offsets, 4) || !aligned(a.rows, 4) || !aligned(a.pos, 4) || !aligned(a.base, es) || !aligned(a.c, es) || !aligned(a.h, 16) ||
      !aligned(a.workspace, 16))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

nvfp4::AdapterArgs adapter_args(const void *x, int64_t x_rows, int64_t ldx, const void *a, const void *b, const float *scales,
                                int64_t M, int64_t N, int64_t K, int32_t rank, int32_t adapters, const int32_t *offsets,
                                const int32_t *rows, const int32_t *pos, int32_t row_div, uint32_t flags) {
  nvfp4::AdapterArgs p{};
  p.x = x;
  p.x_rows = x_rows;
  p.ldx = ldx;
  p.a = a;
  p.b = b;
  p.scales = scales;
  p.M = M;
  p.N = N;
  p.K = K;
  p.rank = rank;
  p.adapters = adapters;
  p.offsets = offsets;
  p.rows = rows;
  p.pos = pos;
  p.row_div = row_div;
  p.gather = flags & NVFP4_ADAPTER_GATHER;
  p.by_token = flags & NVFP4_ADAPTER_BY_TOKEN;
  return p;
}

// Whether a size is one that the workspace functions answer for.
bool adapter_sizes(int64_t M, int64_t N, int64_t K, int32_t rank, int32_t adapters) {
  return M >= 0 && M < kMaxSlots && N >= 1 && N <= kMaxWidth && K >= 8 && K <= kMaxWidth && rank >= 8 && rank <= kMaxRank &&
         adapters >= 1 && adapters <= kMaxExperts;
}

}  // namespace

extern "C" {

size_t nvfp4_adapter_workspace_size(int64_t M, int64_t N, int64_t K, int32_t rank, int32_t adapters) {
  return adapter_sizes(M, N, K, rank, adapters) ? (nvfp4::adapter_workspace_bytes(M, N, K, rank, adapters) + 15) / 16 * 16 : 0;
}

size_t nvfp4_adapter_backward_workspace_size(int64_t M, int64_t N, int64_t K, int32_t rank, int32_t adapters) {
  if (!adapter_sizes(M, N, K, rank, adapters)) return 0;
  // (with a plan as without one: more than one tile of rows may end early)
  static const int32_t some = 0;
  const nvfp4::AdapterArgs a =
      adapter_args(nullptr, M, K, nullptr, nullptr, nullptr, M, N, K, rank, adapters, &some, nullptr, nullptr, 1, 0);
  return (nvfp4::adapter_backward_workspace_bytes(a) + 15) / 16 * 16;
}

int nvfp4_adapter(const void *x, int x_dtype, int64_t x_rows, int64_t ldx, const void *a, const void *b,
                  const float *scales, int64_t M, int64_t N, int64_t K, int32_t rank, int32_t adapters,
                  const int32_t *offsets, const int32_t *rows, const int32_t *pos, int32_t row_div, uint32_t flags,
                  const void *base, int64_t ldb, void *c, int c_dtype, int64_t ldc, float *h, void *workspace,
                  void *hip_stream) {
  nvfp4::AdapterArgs p = adapter_args(x, x_rows, ldx, a, b, scales, M, N, K, rank, adapters, offsets, rows, pos, row_div, flags);
  int st = check_adapter(p, x_dtype, c_dtype, flags);
  if (st != NVFP4_OK) return st;
  if (ldc < N || product(M, ldc) < 0 || (base && (ldb < N || product(M, ldb) < 0)) || !nvfp4::adapter_launches(p, false))
    return NVFP4_ERR_SHAPE;
  if (base == c && base && ldb != ldc && M > 1) return NVFP4_ERR_SHAPE;
  if (M == 0) return NVFP4_OK;
  p.base = base;
  p.ldb = ldb;
  p.c = c;
  p.ldc = ldc;
  p.c_dtype = c_dtype == NVFP4_BF16 ? 1 : 0;
  p.h = h;
  p.workspace = workspace;
  p.stream = static_cast<hipStream_t>(hip_stream);
  if ((st = check_adapter_pointers(p, c_dtype, nvfp4::adapter_workspace_bytes(M, N, K, rank, adapters))) != NVFP4_OK) return st;
  return status_of(nvfp4::launch_adapter(p));
}

int nvfp4_adapter_backward(const void *dc, int dc_dtype, int64_t lddc, const void *x, int x_dtype, int64_t ldx,
                           const void *a, const void *b, const float *scales, int64_t M, int64_t N, int64_t K,
                           int32_t rank, int32_t adapters, const int32_t *offsets, const int32_t *rows,
                           const int32_t *pos, uint32_t flags, const float *h, const void *dx_base, int64_t ldb,
                           void *dx, int dx_dtype, int64_t lddx, float *da, float *db, void *workspace,
                           void *hip_stream) {
  nvfp4::AdapterArgs p = adapter_args(x, M, ldx, a, b, scales, M, N, K, rank, adapters, offsets, rows, pos, 1, flags);
  if (dc_dtype != NVFP4_BF16 || p.gather) return NVFP4_ERR_UNSUPPORTED;
  int st = check_adapter(p, x_dtype, dx_dtype, flags);
  if (st != NVFP4_OK) return st;
  if (N % 8 != 0 || lddc < N || product(M, lddc) < 0 || lddx < K || product(M, lddx) < 0 ||
      (dx_base && (ldb < K || product(M, ldb) < 0)) || (dx_base && dx_base == dx && ldb != lddx && M > 1) ||
      !nvfp4::adapter_launches(p, true))
    return NVFP4_ERR_SHAPE;
  p.base = dx_base;
  p.ldb = ldb;
  p.c = dx;
  p.ldc = lddx;
  p.c_dtype = dx_dtype == NVFP4_BF16 ? 1 : 0;
  p.h = const_cast<float *>(h);
  p.dc = dc;
  p.lddc = lddc;
  p.da = da;
  p.db = db;
  p.workspace = workspace;
  p.stream = static_cast<hipStream_t>(hip_stream);
  if (!da || !db) return NVFP4_ERR_NULL;
  if (!aligned(da, 16) || !aligned(db, 16)) return NVFP4_ERR_ALIGN;
  if (M > 0 && (!dc || !h)) return NVFP4_ERR_NULL;
  if (M > 0 && (st = check_adapter_pointers(p, dx_dtype, 1)) != NVFP4_OK) return st;
  if (!aligned(dc, 16) || lddc % 8 != 0) return NVFP4_ERR_ALIGN;
  return status_of(nvfp4::launch_adapter_backward(p));
}

size_t nvfp4_moe_balance_workspace_size(int64_t tokens, int64_t experts, int64_t sequences) {
  if (tokens < 0 || experts < 1 || experts > kMaxExperts || sequences < 1 || sequences > kMaxSequences) return 0;
  return (nvfp4::moe_balance_workspace_bytes(tokens, experts, sequences) + 15) / 16 * 16;
}

int nvfp4_moe_balance(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t ld, const int32_t *ids,
                      int32_t top_k, int64_t sequences, uint32_t flags, float coef, float *loss, int32_t *counts,
                      float *probs, int32_t *live, void *workspace, void *hip_stream) {
  const int st = check_balance(logits, dtype, tokens, experts, ld, ids, top_k, sequences, flags, coef);
  if (st != NVFP4_OK) return st;
  if (!loss || !counts || !probs || !live) return NVFP4_ERR_NULL;
  if (nvfp4::moe_balance_workspace_bytes(tokens, experts, sequences) > 0 && !workspace) return NVFP4_ERR_NULL;
  if (!aligned(loss, 4) || !aligned(counts, 4) || !aligned(probs, 4) || !aligned(live, 4) || !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  nvfp4::MoeBalanceArgs a{};
  a.logits = logits;
  a.dtype = dtype == NVFP4_BF16 ? 1 : 0;
  a.tokens = tokens;
  a.experts = experts;
  a.ld = ld;
  a.sequences = sequences;
  a.ids = ids;
  a.top_k = top_k;
  a.sigmoid = flags & NVFP4_ROUTE_SIGMOID;
  a.coef = coef;
  a.loss = loss;
  a.probs = probs;
  a.counts = counts;
  a.live = live;
  a.workspace = workspace;
  a.stream = static_cast<hipStream_t>(hip_stream);
  return status_of(nvfp4::launch_moe_balance(a));
}

int nvfp4_moe_balance_backward(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t ld,
                               const int32_t *ids, int32_t top_k, int64_t sequences, uint32_t flags, float coef,
                               const int32_t *counts, const int32_t *live, const float *dloss, const void *dlogits_in,
                               int64_t ld_in, void *dlogits, int64_t ldd, void *hip_stream) {
  const int st = check_balance(logits, dtype, tokens, experts, ld, ids, top_k, sequences, flags, coef);
  if (st != NVFP4_OK) return st;
  if (ldd < experts || product(tokens, ldd) < 0 || (dlogits_in && (ld_in < experts || product(tokens, ld_in) < 0)) ||
      (dlogits_in && dlogits_in == dlogits && ld_in != ldd && tokens > 1))
    return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  if (!counts || !live || !dlogits) return NVFP4_ERR_NULL;
  const int es = dtype_size(dtype);
  if (!aligned(counts, 4) || !aligned(live, 4) || !aligned(dloss, 4) || !aligned(dlogits_in, es) || !aligned(dlogits, es))
    return NVFP4_ERR_ALIGN;
  nvfp4::MoeBalanceArgs a{};
  a.logits = logits;
  a.dtype = dtype == NVFP4_BF16 ? 1 : 0;
  a.tokens = tokens;
  a.experts = experts;
  a.ld = ld;
  a.sequences = sequences;
  a.ids = ids;
  a.top_k = top_k;
  a.sigmoid = flags & NVFP4_ROUTE_SIGMOID;
  a.coef = coef;
  a.counts = const_cast<int32_t *>(counts);
  a.live = const_cast<int32_t *>(live);
  a.dloss = dloss;
  a.dlogits_in = dlogits_in;
  a.ld_in = ld_in;
  a.dlogits = dlogits;
  a.ldd = ldd;
  a.stream = static_cast<hipStream_t>(hip_stream);
  return status_of(nvfp4::launch_moe_balance_backward(a));
}

size_t nvfp4_grad_workspace_size(int64_t tensors, int64_t elements) {
  if (tensors < 0 || tensors > kMaxTensors || elements < 0 || elements > kMaxElements) return 0;
  return (nvfp4::grad_workspace_bytes(tensors, elements) + 15) / 16 * 16;
}

int nvfp4_grad_norm(const void *const *grads, const int64_t *counts, const int32_t *dtypes, int64_t tensors,
                    uint32_t flags, float *norm, void *workspace, void *hip_stream) {
  if (flags & ~NVFP4_GRAD_MAX) return NVFP4_ERR_UNSUPPORTED;
  const int st = check_grads(grads, counts, dtypes, tensors);
  if (st != NVFP4_OK) return st;
  if (!norm || (tensors > 0 && !workspace)) return NVFP4_ERR_NULL;
  if (!aligned(norm, 4) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  nvfp4::GradArgs a{};
  a.grads = grads;
  a.counts = counts;
  a.dtypes = dtypes;
  a.tensors = tensors;
  a.max = flags & NVFP4_GRAD_MAX;
  a.norm = norm;
  a.workspace = static_cast<double *>(workspace);
  a.stream = static_cast<hipStream_t>(hip_stream);
  return status_of(nvfp4::launch_grad_norm(a));
}

int nvfp4_grad_clip(const void *const *grads, void *const *outs, const int64_t *counts, const int32_t *dtypes,
                    int64_t tensors, const float *norm, float max_norm, float eps, void *hip_stream) {
  // (written so that NaN is refused)
  if (!(max_norm >= 0.0f) || !(eps >= 0.0f) || (max_norm == 0.0f && eps == 0.0f)) return NVFP4_ERR_UNSUPPORTED;
  int st = check_grads(grads, counts, dtypes, tensors);
  if (st != NVFP4_OK) return st;
  if (!norm || (tensors > 0 && !outs)) return NVFP4_ERR_NULL;
  if (!aligned(norm, 4)) return NVFP4_ERR_ALIGN;
  for (int64_t i = 0; i < tensors; ++i) {
    if (counts[i] > 0 && !outs[i]) return NVFP4_ERR_NULL;
    if (!aligned(outs[i], dtype_size(dtypes[i]))) return NVFP4_ERR_ALIGN;
  }
  if ((st = check_overlap(grads, outs, counts, dtypes, tensors)) != NVFP4_OK) return st;
  nvfp4::GradArgs a{};
  a.grads = grads;
  a.outs = outs;
  a.counts = counts;
  a.dtypes = dtypes;
  a.tensors = tensors;
  a.max_norm = max_norm;
  a.eps = eps;
  a.norm = const_cast<float *>(norm);
  a.stream = static_cast<hipStream_t>(hip_stream);
  return status_of(nvfp4::launch_grad_clip(a));
}

}  // extern "C"
