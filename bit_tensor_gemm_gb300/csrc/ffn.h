// ffn.h -- parameters and launchers of the feed-forward operators: 4-bit
// weights with group scales (w4_*.cu), the router (moe_route.cu) and the norms
// around a block (residual_norm.cu); their C ABI is in ffn_api.cu.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "attn.h"
#include "lbgemm.h"

namespace lbg {

// The feed-forward operators' scratch on this device; the caller holds one lock
// from acquire to release.
lbgemm_status ffn_scratch_acquire(const CallDevice& dev, size_t bytes, cudaStream_t s, void** ptr);
lbgemm_status ffn_scratch_release(const CallDevice& dev, cudaStream_t s, void* ptr);

// ---- 4-bit weights ------------------------------------------------------------------
// Rows of k codes: the weight (n, i) is code * e4m3 scale of the group * row scale.
struct W4 {
  const uint8_t* codes = nullptr;   // [rows][k / 2]
  const uint8_t* scales = nullptr;  // [rows][k / group]
  const float* row_scales = nullptr;
};

struct W4QuantParams {
  int64_t rows = 0, k = 0, group = 0;
  const void* w = nullptr;
  int64_t w_stride = 0;
  uint8_t* codes = nullptr;
  int64_t code_stride = 0;
  uint8_t* scales = nullptr;
  int64_t scale_stride = 0;
  float* row_scales = nullptr;
  int64_t row_stride = 0;
};
cudaError_t launch_w4_quantize(int dtype, const W4QuantParams& p, cudaStream_t s);

struct W4LinearParams {
  int64_t m = 0, n = 0, k = 0;
  int group = 0;
  const void* x = nullptr;
  int64_t x_stride = 0;
  W4 w;
  void* y = nullptr;
  int64_t y_stride = 0;
  int* status = nullptr;
};

// A mixture of experts: y[t] = sum over j of weights[t][j] * down(act(up(x[t]))) of
// expert ids[t][j].  Weights of all experts are stacked by rows.
struct MoeParams {
  int64_t tokens = 0;
  int hidden = 0, inter = 0, experts = 0, top_k = 0, group = 0;
  const void* x = nullptr;
  int64_t x_stride = 0;
  const int32_t* ids = nullptr;
  const float* weights = nullptr;
  W4 up, down;  // [experts][2 inter][hidden], [experts][hidden][inter]
  void* y = nullptr;
  int64_t y_stride = 0;
  int* status = nullptr;
};

// How a call runs on this device, and the scratch that it needs.
size_t w4_linear_scratch(const W4LinearParams& p, int sm_count);
cudaError_t launch_w4_linear(int dtype, const W4LinearParams& p, void* scratch, int sm_count,
                             int* launches, cudaStream_t s);
size_t moe_w4_scratch(const MoeParams& p, int sm_count);
cudaError_t launch_moe_w4(int dtype, const MoeParams& p, void* scratch, int sm_count,
                          int* launches, cudaStream_t s);

// ---- the router ------------------------------------------------------------------------
struct RouteParams {
  int64_t tokens = 0;
  int experts = 0, top_k = 0, renormalize = 0;
  const void* logits = nullptr;
  int64_t stride = 0;
  int32_t* ids = nullptr;
  float* weights = nullptr;
};
cudaError_t launch_moe_route(int dtype, const RouteParams& p, cudaStream_t s);

// ---- norms around a block ----------------------------------------------------------------
// z = y * rstd(y) * post (or y); x' = a * x + b * gate * z; n = x' * rstd(x') * next.
// Rows of `width`; gate_stride 0: one row of gates for all.
struct ResidualNormParams {
  int64_t tokens = 0;
  int width = 0;
  const void *x = nullptr, *y = nullptr, *post = nullptr, *gate = nullptr, *next = nullptr;
  int64_t x_stride = 0, y_stride = 0, gate_stride = 0;
  float a = 1.0f, b = 1.0f, eps = 0.0f;
  // forward
  void *x_out = nullptr, *n_out = nullptr;
  int64_t x_out_stride = 0, n_out_stride = 0;
  // backward: the outputs' gradients, the inputs' (weights' and one row of gates' summed)
  const void *dx_out = nullptr, *dn = nullptr;
  int64_t dx_out_stride = 0, dn_stride = 0;
  void *dx = nullptr, *dy = nullptr, *dgate = nullptr;
  int64_t dx_stride = 0, dy_stride = 0, dgate_stride = 0;
  float *dpost = nullptr, *dnext = nullptr;
  int* status = nullptr;
};
cudaError_t launch_residual_norm(int dtype, const ResidualNormParams& p, int sm_count,
                                 cudaStream_t s);
// partial: scratch of residual_norm_scratch() bytes (none where nothing is summed over rows).
size_t residual_norm_scratch(int dtype, const ResidualNormParams& p, int sm_count);
cudaError_t launch_residual_norm_backward(int dtype, const ResidualNormParams& p, int sm_count,
                                          float* partial, int* launches, cudaStream_t s);

}  // namespace lbg
