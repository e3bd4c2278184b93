// nvfp4_internal.h -- private interface between the C-ABI front end (nvfp4_api.cpp) and the kernel
// launchers (*.hip).  Not installed; not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// Upper bound on the number of amax-pass workgroups; the workspace holds one partial maximum each.
constexpr uint32_t kMaxParts = 4096;

struct QuantArgs {
  const void *x;
  int dtype;              // 0 = f32, 1 = bf16
  int64_t rows, cols, ldx;
  int64_t R, K;           // logical Y shape
  uint32_t flags;
  uint64_t seed;
  uint32_t stream_id;
  bool rht;
  uint32_t sign_word;
  float *rht_out;
  uint8_t *data;
  uint8_t *scales;
  float *ts;
  uint32_t *workspace;
  hipStream_t stream;
  int64_t groups = 1;         // equally shaped tensors quantized by one call (grid dimension y)
  int64_t x_group_bytes = 0;  // bytes between consecutive groups' inputs
};

struct DequantArgs {
  const uint8_t *data;
  const uint8_t *scales;
  const float *ts;
  int64_t R, K;
  bool block2d;
  void *y;
  int y_dtype;
  int64_t ldy;
  hipStream_t stream;
};

struct GemmArgs {
  const uint8_t *a_data, *a_scales;
  const float *a_ts;
  bool a_2d;
  const uint8_t *b_data, *b_scales;
  const float *b_ts;
  bool b_2d;
  int64_t M, N, K;
  void *c;
  int c_dtype;
  int64_t ldc;
  int32_t num_groups;
  const int64_t *group_offsets;  // host, num_groups + 1 (nullptr for a plain GEMM)
  hipStream_t stream;
  // c_dtype 2: C quantized to NVFP4 (1D, nearest-even) with tensor scale *q_ts; amax nullable
  uint8_t *q_data = nullptr, *q_scales = nullptr;
  const float *q_ts = nullptr;
  float *amax = nullptr;
};

struct W4A16Args {
  const void *a;  // bf16 [M x lda]
  int64_t lda;    // elements
  const uint8_t *b_data, *b_scales;
  const float *b_ts;
  bool b_2d;
  int64_t M, N, K;
  void *c;
  int c_dtype;
  int64_t ldc;
  hipStream_t stream;
};

struct TransposeLaunch {
  const uint8_t *in_data, *in_scales;
  const float *in_ts;
  uint8_t *out_data, *out_scales;
  float *out_ts;
  int64_t R, K;  // input logical shape
  hipStream_t stream;
};

// Chunks of the counting sort behind a plan: at most one row of counts each in the workspace.
constexpr int kPlanChunks = 256;

struct MoeRouteArgs {
  const void *logits;
  int dtype;
  int64_t tokens, experts, ld;
  const float *bias;
  int32_t num_groups, group_top_k, top_k;
  bool sigmoid, renorm, sum2;
  float scale;
  int32_t *ids;
  float *weights;
  int32_t *offsets, *rows, *pos;  // all or none
  int32_t *workspace;
  hipStream_t stream;
};

struct MoeRouteBackwardArgs {
  const void *logits;
  int dtype;
  int64_t tokens, experts, ld;
  const int32_t *ids;
  const float *dweights;
  int32_t top_k;
  bool sigmoid, renorm;
  float scale;
  void *dlogits;
  int64_t ldd;
  hipStream_t stream;
};

struct MoeRowsArgs {  // gather, combine and combine's gradient
  const void *x;       // gather: x; combine: y; gradient: y
  int64_t ldx;
  const void *dout;    // gradient only
  int64_t ld_dout;
  int dtype;
  int64_t tokens, d;
  const int32_t *pos, *rows;
  const float *weights;
  int32_t top_k;
  void *out;           // gather: y; combine: out; gradient: dy
  int64_t ldo;
  float *dweights;
  hipStream_t stream;
};

struct Int8QuantArgs {
  const void *x;
  int dtype;
  int64_t rows, cols, ldx;
  int8_t *q;
  float *scales;
  hipStream_t stream;
};

struct Int8GemmArgs {
  const int8_t *a;
  const float *a_scales;
  int64_t a_rows;
  const int8_t *b;
  const float *b_scales;
  int64_t M, N, K;
  void *c;
  int c_dtype;
  int64_t ldc;
  int32_t num_groups;
  const int32_t *offsets, *rows;  // device
  int32_t row_div;
  int32_t *workspace;  // int8_gemm_workspace_bytes() of the plain form (nullptr: none)
  hipStream_t stream;
};

struct BlockNormArgs {
  const void *x, *y;
  int x_dtype, y_dtype;
  int64_t tokens, d;
  const float *w_post;
  const void *gate;
  const float *w_pre;
  float alpha, eps;
  bool one_plus, token_gate;
  void *x_out, *n;              // forward
  float *rstd_post, *rstd_pre;  // forward: written; backward: read
  const void *dx_out, *dn;      // backward
  void *dx, *dy, *dgate;
  float *dw_post, *dw_pre;
  float *workspace;
  hipStream_t stream;
};

// Each returns hipSuccess or the launch error.
hipError_t launch_moe_route(const MoeRouteArgs &a);
hipError_t launch_moe_route_backward(const MoeRouteBackwardArgs &a);
hipError_t launch_moe_plan(const int32_t *ids, int64_t slots, int64_t experts, int32_t *offsets, int32_t *rows,
                           int32_t *pos, int32_t *counts, hipStream_t stream);
size_t moe_workspace_bytes(int64_t tokens, int64_t experts);
hipError_t launch_moe_gather(const MoeRowsArgs &a);
hipError_t launch_moe_combine(const MoeRowsArgs &a);
hipError_t launch_moe_combine_backward(const MoeRowsArgs &a);
hipError_t launch_int8_quantize(const Int8QuantArgs &a);
hipError_t launch_int8_gemm(const Int8GemmArgs &a);
size_t int8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_block_norm(const BlockNormArgs &a);
hipError_t launch_block_norm_backward(const BlockNormArgs &a);
size_t block_norm_workspace_bytes(int64_t tokens, int64_t d);
hipError_t launch_quantize(const QuantArgs &a);
hipError_t launch_dequantize(const DequantArgs &a);
hipError_t launch_gemm(const GemmArgs &a);
hipError_t launch_transpose(const TransposeLaunch &a);
hipError_t launch_gemm_w4a16(const W4A16Args &a);
hipError_t launch_scale_from_amax(const float *amax, float *ts, hipStream_t stream);

// Host copy of the Philox4x32-10 block function (for the RHT sign word).
void philox4x32_10_host(const uint32_t ctr[4], const uint32_t key[2], uint32_t out[4]);

}  // namespace nvfp4
