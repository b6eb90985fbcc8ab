// ffn_api.cu -- the C ABI of the feed-forward operators (include/lbgemm.h):
// argument checks, scratch and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "api_checks.h"
#include "ffn.h"
#include "lbgemm.h"

namespace {

using namespace lbg;

std::mutex g_ffn_mu;  // the feed-forward operators' scratch

// Strides in elements.  (Tensor maps hold fewer than 2^40 bytes.)
constexpr int64_t kMostStride = int64_t(1) << 38;

// Rows of `width` elements given by pointer and stride.
lbgemm_status check_rows(const char* name, const void* p, int64_t stride, int64_t rows,
                         int64_t width, int dtype) {
  if (rows == 0) return LBGEMM_OK;
  if (!p) return bad(LBGEMM_ERR_INVALID_ARG, "%s is a null pointer", name);
  if (stride > kMostStride || (rows > 1 && stride < width))
    return bad(LBGEMM_ERR_INVALID_ARG, "%s: row stride %lld does not hold %lld elements", name,
               (long long)stride, (long long)width);
  if (!aligned(p, 16) || (rows > 1 && stride * elem_size(dtype) % 16))
    return bad(LBGEMM_ERR_ALIGNMENT, "%s: pointer and row stride must be 16-byte aligned", name);
  return LBGEMM_OK;
}

constexpr int64_t kMostK = int64_t(1) << 20, kMostRows = int64_t(1) << 30;

lbgemm_status check_group(int64_t k, int64_t group) {
  if (group != 32 && group != 64 && group != 128)
    return bad(LBGEMM_ERR_INVALID_ARG, "a group has 32, 64 or 128 elements (got %lld)",
               (long long)group);
  if (k < 1 || k > kMostK || k % group)
    return bad(LBGEMM_ERR_INVALID_ARG, "%lld elements a row: not whole groups of %lld, or too many",
               (long long)k, (long long)group);
  return LBGEMM_OK;
}

lbgemm_status check_w4(const char* name, const void* codes, const void* scales,
                       const float* row_scales) {
  if (!codes || !scales || !row_scales)
    return bad(LBGEMM_ERR_INVALID_ARG, "%s: codes, scales or row scales are a null pointer", name);
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(row_scales, 16))
    return bad(LBGEMM_ERR_ALIGNMENT, "%s: codes, scales and row scales must be 16-byte aligned",
               name);
  return LBGEMM_OK;
}

// Runs `launch(scratch, &launches)` with `bytes` of scratch.
template <typename F>
lbgemm_status with_scratch(const CallDevice& dev, size_t bytes, cudaStream_t s, const char* what,
                           F launch) {
  int launches = 0;
  if (bytes == 0) {
    const cudaError_t e = launch(nullptr, &launches);
    if (e != cudaSuccess) return report_cuda_error(e, what);
  } else {
    std::lock_guard<std::mutex> lock(g_ffn_mu);
    void* scratch = nullptr;
    lbgemm_status st = ffn_scratch_acquire(dev, bytes, s, &scratch);
    if (st != LBGEMM_OK) return st;
    const cudaError_t e = launch(scratch, &launches);
    st = ffn_scratch_release(dev, s, scratch);
    if (e != cudaSuccess) return report_cuda_error(e, what);
    if (st != LBGEMM_OK) return st;
  }
  count_launches(launches);
  return LBGEMM_OK;
}

lbgemm_status check_norm(int dtype, int64_t tokens, int64_t width, const void* X, int64_t x_stride,
                         const void* Y, int64_t y_stride, const void* w_post, const void* gate,
                         int64_t gate_stride, float a, float b, const void* w_next, float eps) {
  lbgemm_status st = check_dtype(dtype, true);
  if (st != LBGEMM_OK) return st;
  if (tokens < 0 || tokens > INT32_MAX)
    return bad(LBGEMM_ERR_INVALID_ARG, "%lld tokens", (long long)tokens);
  const int64_t most = dtype == LBGEMM_F32 ? 8192 : 16384;
  if (width < 8 || width > most || width % 8)
    return bad(LBGEMM_ERR_INVALID_ARG, "width must be a multiple of 8 up to %lld (got %lld)",
               (long long)most, (long long)width);
  if (!(eps >= 0.0f) || std::isinf(eps)) return bad(LBGEMM_ERR_INVALID_ARG, "eps must be >= 0");
  if (!std::isfinite(a) || !std::isfinite(b))
    return bad(LBGEMM_ERR_INVALID_ARG, "the residual's and the block's scale must be finite");
  if (!Y && (w_post || gate) && tokens > 0)  // (an empty tensor has no address)
    return bad(LBGEMM_ERR_INVALID_ARG, "a norm or gate of a block needs its output Y");
  if (!aligned(w_post, 16) || !aligned(w_next, 16))
    return bad(LBGEMM_ERR_ALIGNMENT, "norm weights must be 16-byte aligned");
  if (gate && gate_stride == 0) {
    if (!aligned(gate, 16)) return bad(LBGEMM_ERR_ALIGNMENT, "gate must be 16-byte aligned");
  } else if (gate) {
    if (gate_stride < width)
      return bad(LBGEMM_ERR_INVALID_ARG, "gate: row stride %lld does not hold %lld elements",
                 (long long)gate_stride, (long long)width);
    st = check_rows("gate", gate, gate_stride, tokens, width, dtype);
    if (st != LBGEMM_OK) return st;
  }
  st = check_rows("X", X, x_stride, tokens, width, dtype);
  if (st == LBGEMM_OK && Y) st = check_rows("Y", Y, y_stride, tokens, width, dtype);
  return st;
}

}  // namespace

extern "C" {

lbgemm_status lbgemm_w4_quantize(int dtype, int64_t N, int64_t K, int64_t group, const void* W,
                                 int64_t w_stride, void* codes, int64_t code_stride, void* scales,
                                 int64_t scale_stride, float* row_scales, int64_t row_stride,
                                 void* stream) {
  try {
    lbgemm_status st = check_dtype(dtype, true);
    if (st == LBGEMM_OK) st = check_group(K, group);
    if (st != LBGEMM_OK) return st;
    if (N < 0 || N > kMostRows) return bad(LBGEMM_ERR_INVALID_ARG, "%lld rows", (long long)N);
    st = check_rows("W", W, w_stride, N, K, dtype);
    if (st != LBGEMM_OK || N == 0) return st;
    if (!codes || !scales || !row_scales)
      return bad(LBGEMM_ERR_INVALID_ARG, "codes, scales or row scales are a null pointer");
    if (N > 1 && (code_stride < K / 2 || code_stride > kMaxStride || scale_stride < K / group ||
                  scale_stride > kMaxStride || row_stride < 1 || row_stride > kMaxStride))
      return bad(LBGEMM_ERR_INVALID_ARG, "a stride of the output does not hold its row");
    if (!aligned(codes, 16) || (N > 1 && code_stride % 16) || !aligned(row_scales, 4))
      return bad(LBGEMM_ERR_ALIGNMENT,
                 "codes and their stride must be 16-byte, row scales 4-byte aligned");
    CallDevice dev;
    st = call_device(&dev);
    if (st != LBGEMM_OK) return st;
    W4QuantParams p;
    p.rows = N;
    p.k = K;
    p.group = group;
    p.w = W;
    p.w_stride = w_stride;
    p.codes = static_cast<uint8_t*>(codes);
    p.code_stride = code_stride;
    p.scales = static_cast<uint8_t*>(scales);
    p.scale_stride = scale_stride;
    p.row_scales = row_scales;
    p.row_stride = row_stride;
    const cudaError_t e = launch_w4_quantize(dtype, p, as_stream(stream));
    if (e != cudaSuccess) return report_cuda_error(e, "4-bit quantiser launch");
    count_launches(1);
    return LBGEMM_OK;
  } catch (...) {
    return report_error(LBGEMM_ERR_CUDA, "internal error");
  }
}

lbgemm_status lbgemm_w4_linear(int dtype, int64_t M, int64_t N, int64_t K, int64_t group,
                               const void* X, int64_t x_stride, const void* codes,
                               const void* scales, const float* row_scales, void* Y,
                               int64_t y_stride, void* stream) {
  try {
    lbgemm_status st = check_dtype(dtype, false);
    if (st == LBGEMM_OK) st = check_group(K, group);
    if (st != LBGEMM_OK) return st;
    if (M < 0 || M > kMostRows || N < 0 || N > kMostRows)
      return bad(LBGEMM_ERR_INVALID_ARG, "%lld tokens, %lld rows", (long long)M, (long long)N);
    if (M * N > (int64_t(1) << 45))  // (the kernels count tiles in 32 bits)
      return bad(LBGEMM_ERR_INVALID_ARG, "%lld tokens by %lld rows are too many tiles",
                 (long long)M, (long long)N);
    if (M == 0 || N == 0) return LBGEMM_OK;
    st = check_rows("X", X, x_stride, M, K, dtype);
    if (st == LBGEMM_OK) st = check_w4("W", codes, scales, row_scales);
    if (st != LBGEMM_OK) return st;
    if (!Y) return bad(LBGEMM_ERR_INVALID_ARG, "Y is a null pointer");
    if (y_stride > kMaxStride || (M > 1 && y_stride < N))
      return bad(LBGEMM_ERR_INVALID_ARG, "Y: row stride %lld does not hold %lld elements",
                 (long long)y_stride, (long long)N);
    if (!aligned(Y, 16)) return bad(LBGEMM_ERR_ALIGNMENT, "Y must be 16-byte aligned");
    CallDevice dev;
    st = call_device(&dev);
    if (st != LBGEMM_OK) return st;
    W4LinearParams p;
    p.m = M;
    p.n = N;
    p.k = K;
    p.group = (int)group;
    p.x = X;
    p.x_stride = M > 1 ? x_stride : K;
    p.w = {static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), row_scales};
    p.y = Y;
    p.y_stride = y_stride;
    p.status = dev.status;
    cudaStream_t s = as_stream(stream);
    return with_scratch(dev, w4_linear_scratch(p, dev.sm_count), s, "4-bit linear layer launch",
                        [&](void* scratch, int* launches) {
                          return launch_w4_linear(dtype, p, scratch, dev.sm_count, launches, s);
                        });
  } catch (...) {
    return report_error(LBGEMM_ERR_CUDA, "internal error");
  }
}

lbgemm_status lbgemm_moe_route(int dtype, int64_t tokens, int64_t experts, int64_t top_k,
                               const void* logits, int64_t stride, int renormalize, int32_t* ids,
                               float* weights, void* stream) {
  try {
    lbgemm_status st = check_dtype(dtype, true);
    if (st != LBGEMM_OK) return st;
    if (tokens < 0 || tokens > kMostRows)
      return bad(LBGEMM_ERR_INVALID_ARG, "%lld tokens", (long long)tokens);
    if (experts < 1 || experts > 1024 || top_k < 1 || top_k > 32 || top_k > experts)
      return bad(LBGEMM_ERR_INVALID_ARG, "%lld of %lld experts (up to 32 of up to 1024)",
                 (long long)top_k, (long long)experts);
    if (tokens == 0) return LBGEMM_OK;
    if (!logits || !ids || !weights)
      return bad(LBGEMM_ERR_INVALID_ARG, "logits, ids or weights are a null pointer");
    if (stride > kMaxStride || (tokens > 1 && stride < experts))
      return bad(LBGEMM_ERR_INVALID_ARG, "logits: row stride %lld does not hold %lld experts",
                 (long long)stride, (long long)experts);
    if (!aligned(logits, elem_size(dtype)) || !aligned(ids, 4) || !aligned(weights, 4))
      return bad(LBGEMM_ERR_ALIGNMENT, "logits, ids and weights must be aligned to their elements");
    CallDevice dev;
    st = call_device(&dev);
    if (st != LBGEMM_OK) return st;
    RouteParams p;
    p.tokens = tokens;
    p.experts = (int)experts;
    p.top_k = (int)top_k;
    p.renormalize = renormalize != 0;
    p.logits = logits;
    p.stride = stride;
    p.ids = ids;
    p.weights = weights;
    const cudaError_t e = launch_moe_route(dtype, p, as_stream(stream));
    if (e != cudaSuccess) return report_cuda_error(e, "router launch");
    count_launches(1);
    return LBGEMM_OK;
  } catch (...) {
    return report_error(LBGEMM_ERR_CUDA, "internal error");
  }
}

lbgemm_status lbgemm_moe_w4(int dtype, int64_t tokens, int64_t hidden, int64_t inter,
                            int64_t experts, int64_t top_k, int64_t group, const void* X,
                            int64_t x_stride, const int32_t* ids, const float* weights,
                            const void* up_codes, const void* up_scales,
                            const float* up_row_scales, const void* down_codes,
                            const void* down_scales, const float* down_row_scales, void* Y,
                            int64_t y_stride, void* stream) {
  try {
    lbgemm_status st = check_dtype(dtype, false);
    if (st == LBGEMM_OK) st = check_group(hidden, group);
    if (st == LBGEMM_OK) st = check_group(inter, group);
    if (st != LBGEMM_OK) return st;
    if (experts < 1 || experts > 1024 || top_k < 1 || top_k > 32)
      return bad(LBGEMM_ERR_INVALID_ARG, "%lld choices among %lld experts (up to 32, up to 1024)",
                 (long long)top_k, (long long)experts);
    if (tokens < 0 || tokens > (int64_t(1) << 24) / top_k)
      return bad(LBGEMM_ERR_INVALID_ARG, "%lld tokens of %lld choices (up to 2^24 together)",
                 (long long)tokens, (long long)top_k);
    if (experts * std::max(2 * inter, hidden) > kMostRows)
      return bad(LBGEMM_ERR_INVALID_ARG, "the experts have more than 2^30 rows");
    if (tokens == 0) return LBGEMM_OK;
    st = check_rows("X", X, x_stride, tokens, hidden, dtype);
    if (st == LBGEMM_OK) st = check_rows("Y", Y, y_stride, tokens, hidden, dtype);
    if (st == LBGEMM_OK) st = check_w4("up", up_codes, up_scales, up_row_scales);
    if (st == LBGEMM_OK) st = check_w4("down", down_codes, down_scales, down_row_scales);
    if (st != LBGEMM_OK) return st;
    if (!ids || !weights)
      return bad(LBGEMM_ERR_INVALID_ARG, "ids or weights are a null pointer");
    if (!aligned(ids, 4) || !aligned(weights, 4))
      return bad(LBGEMM_ERR_ALIGNMENT, "ids and weights must be 4-byte aligned");
    CallDevice dev;
    st = call_device(&dev);
    if (st != LBGEMM_OK) return st;
    MoeParams p;
    p.tokens = tokens;
    p.hidden = (int)hidden;
    p.inter = (int)inter;
    p.experts = (int)experts;
    p.top_k = (int)top_k;
    p.group = (int)group;
    p.x = X;
    p.x_stride = tokens > 1 ? x_stride : hidden;
    p.ids = ids;
    p.weights = weights;
    p.up = {static_cast<const uint8_t*>(up_codes), static_cast<const uint8_t*>(up_scales),
            up_row_scales};
    p.down = {static_cast<const uint8_t*>(down_codes), static_cast<const uint8_t*>(down_scales),
              down_row_scales};
    p.y = Y;
    p.y_stride = y_stride;
    p.status = dev.status;
    cudaStream_t s = as_stream(stream);
    return with_scratch(dev, moe_w4_scratch(p, dev.sm_count), s, "experts launch",
                        [&](void* scratch, int* launches) {
                          return launch_moe_w4(dtype, p, scratch, dev.sm_count, launches, s);
                        });
  } catch (...) {
    return report_error(LBGEMM_ERR_CUDA, "internal error");
  }
}

lbgemm_status lbgemm_residual_norm(int dtype, int64_t tokens, int64_t width, const void* X,
                                   int64_t x_stride, const void* Y, int64_t y_stride,
                                   const void* w_post, const void* gate, int64_t gate_stride,
                                   float residual_scale, float block_scale, const void* w_next,
                                   float eps, void* X_out, int64_t x_out_stride, void* N_out,
                                   int64_t n_out_stride, void* stream) {
  try {
    lbgemm_status st =
        check_norm(dtype, tokens, width, X, x_stride, Y, y_stride, w_post, gate, gate_stride,
                   residual_scale, block_scale, w_next, eps);
    if (st != LBGEMM_OK) return st;
    if ((w_next != nullptr) != (N_out != nullptr) && tokens > 0)
      return bad(LBGEMM_ERR_INVALID_ARG, "N_out is given exactly where w_next is");
    if (!X_out && tokens > 0 && (Y || !N_out))
      return bad(LBGEMM_ERR_INVALID_ARG, "X_out is a null pointer");
    if (X_out) st = check_rows("X_out", X_out, x_out_stride, tokens, width, dtype);
    if (st == LBGEMM_OK && N_out)
      st = check_rows("N_out", N_out, n_out_stride, tokens, width, dtype);
    if (st != LBGEMM_OK || tokens == 0) return st;
    CallDevice dev;
    st = call_device(&dev);
    if (st != LBGEMM_OK) return st;
    ResidualNormParams p;
    p.tokens = tokens;
    p.width = (int)width;
    p.x = X;
    p.y = Y;
    p.post = w_post;
    p.gate = gate;
    p.next = w_next;
    p.x_stride = x_stride;
    p.y_stride = y_stride;
    p.gate_stride = gate_stride;
    p.a = residual_scale;
    p.b = block_scale;
    p.eps = eps;
    p.x_out = X_out;
    p.n_out = N_out;
    p.x_out_stride = x_out_stride;
    p.n_out_stride = n_out_stride;
    p.status = dev.status;
    const cudaError_t e = launch_residual_norm(dtype, p, dev.sm_count, as_stream(stream));
    if (e != cudaSuccess) return report_cuda_error(e, "residual norm launch");
    count_launches(1);
    return LBGEMM_OK;
  } catch (...) {
    return report_error(LBGEMM_ERR_CUDA, "internal error");
  }
}

lbgemm_status lbgemm_residual_norm_backward(
    int dtype, int64_t tokens, int64_t width, const void* dX_out, int64_t dx_out_stride,
    const void* dN, int64_t dn_stride, const void* X, int64_t x_stride, const void* Y,
    int64_t y_stride, const void* w_post, const void* gate, int64_t gate_stride,
    float residual_scale, float block_scale, const void* w_next, float eps, void* dX,
    int64_t dx_stride, void* dY, int64_t dy_stride, void* dgate, int64_t dgate_stride,
    float* dw_post, float* dw_next, void* stream) {
  try {
    lbgemm_status st =
        check_norm(dtype, tokens, width, X, x_stride, Y, y_stride, w_post, gate, gate_stride,
                   residual_scale, block_scale, w_next, eps);
    if (st != LBGEMM_OK) return st;
    if ((w_post != nullptr) != (dw_post != nullptr) || (w_next != nullptr) != (dw_next != nullptr))
      return bad(LBGEMM_ERR_INVALID_ARG, "dw_post and dw_next are given exactly where the weights are");
    const bool row_gates = gate && gate_stride != 0;
    if (tokens > 0) {
      if ((w_next != nullptr) != (dN != nullptr))
        return bad(LBGEMM_ERR_INVALID_ARG, "dN is given exactly where w_next is");
      if (!dX_out && !dN) return bad(LBGEMM_ERR_INVALID_ARG, "no gradient of an output is given");
      if ((Y != nullptr) != (dY != nullptr))
        return bad(LBGEMM_ERR_INVALID_ARG, "dY is given exactly where Y is");
      if (dX_out) st = check_rows("dX_out", dX_out, dx_out_stride, tokens, width, dtype);
      if (st == LBGEMM_OK && dN) st = check_rows("dN", dN, dn_stride, tokens, width, dtype);
      if (st == LBGEMM_OK) st = check_rows("dX", dX, dx_stride, tokens, width, dtype);
      if (st == LBGEMM_OK && dY) st = check_rows("dY", dY, dy_stride, tokens, width, dtype);
      if (st != LBGEMM_OK) return st;
    }
    if ((gate != nullptr) != (dgate != nullptr) && (tokens > 0 || !row_gates))
      return bad(LBGEMM_ERR_INVALID_ARG, "dgate is given exactly where gate is");
    if (row_gates && dgate) {
      if (dgate_stride < width)
        return bad(LBGEMM_ERR_INVALID_ARG, "dgate has a row for every row of gates");
      st = check_rows("dgate", dgate, dgate_stride, tokens, width, dtype);
      if (st != LBGEMM_OK) return st;
    } else if (!aligned(dgate, 16)) {
      return bad(LBGEMM_ERR_ALIGNMENT, "dgate must be 16-byte aligned");
    }
    if (!aligned(dw_post, 16) || !aligned(dw_next, 16))
      return bad(LBGEMM_ERR_ALIGNMENT, "dw_post and dw_next must be 16-byte aligned");
    ResidualNormParams p;
    p.tokens = tokens;
    p.width = (int)width;
    p.x = X;
    p.y = Y;
    p.post = w_post;
    p.gate = gate;
    p.next = w_next;
    p.x_stride = x_stride;
    p.y_stride = y_stride;
    p.gate_stride = gate_stride;
    p.a = residual_scale;
    p.b = block_scale;
    p.eps = eps;
    p.dx_out = dX_out;
    p.dn = dN;
    p.dx_out_stride = dx_out_stride;
    p.dn_stride = dn_stride;
    p.dx = dX;
    p.dy = dY;
    p.dgate = dgate;
    p.dx_stride = dx_stride;
    p.dy_stride = dy_stride;
    p.dgate_stride = dgate_stride;
    p.dpost = dw_post;
    p.dnext = dw_next;
    if (tokens == 0 && !dw_post && !dw_next && !(dgate && !row_gates)) return LBGEMM_OK;
    CallDevice dev;
    st = call_device(&dev);
    if (st != LBGEMM_OK) return st;
    p.status = dev.status;
    cudaStream_t s = as_stream(stream);
    return with_scratch(dev, residual_norm_scratch(dtype, p, dev.sm_count), s,
                        "residual norm backward launch", [&](void* scratch, int* launches) {
                          return launch_residual_norm_backward(
                              dtype, p, dev.sm_count, static_cast<float*>(scratch), launches, s);
                        });
  } catch (...) {
    return report_error(LBGEMM_ERR_CUDA, "internal error");
  }
}

}  // extern "C"
