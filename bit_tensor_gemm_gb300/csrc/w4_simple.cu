// w4_simple.cu -- products with 4-bit weights, a warp a sum.
#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "ffn.h"
#include "w4_codes.cuh"
#include "w4_kernels.h"

namespace lbg {
namespace {

template <typename T>
__device__ __forceinline__ float2 floats(uint32_t p) {
  const T* h = reinterpret_cast<const T*>(&p);
  return make_float2(to_f32(h[0]), to_f32(h[1]));
}

// x . row, by a warp
template <typename T>
__device__ float row_dot(const T* x, const W4& w, int64_t row, int k, int group) {
  const int lane = threadIdx.x % 32;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(w.codes + row * (k / 2));
  const uint8_t* scales = w.scales + row * (k / group);
  float sum = 0.0f;
  for (int o = lane; o < k / 8; o += 32) {
    float f[8];
    unpack8(load8_raw(x + o * 8), f);
    W4Scale<T> sc, same;
    w4_scales(scales[o * 8 / group], 0, sc, same);
    uint32_t v[4];
    w4_word(codes[o], sc, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = floats<T>(v[j]);
      sum += a.x * f[2 * j] + a.y * f[2 * j + 1];
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  return sum * w.row_scales[row];
}

constexpr int kWarps = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) linear_kernel(const W4LinearParams p) {
  const int64_t items = p.m * p.n;
  for (int64_t i = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; i < items;
       i += (int64_t)gridDim.x * kWarps) {
    const int64_t m = i / p.n, n = i - m * p.n;
    const float v = row_dot(static_cast<const T*>(p.x) + m * p.x_stride, p.w, n, (int)p.k, p.group);
    if (threadIdx.x % 32 == 0) static_cast<T*>(p.y)[m * p.y_stride + n] = from_f32<T>(v);
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) up_kernel(const MoeParams p, T* h) {
  const int64_t items = p.tokens * p.top_k * p.inter;
  for (int64_t i = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; i < items;
       i += (int64_t)gridDim.x * kWarps) {
    const int64_t pick = i / p.inter, c = i - pick * p.inter;
    const int e = p.ids[pick];
    if (e < 0 || e >= p.experts) continue;
    const T* x = static_cast<const T*>(p.x) + pick / p.top_k * p.x_stride;
    const int64_t row = (int64_t)e * 2 * p.inter + 2 * c;
    const float g = row_dot(x, p.up, row, p.hidden, p.group);
    const float u = row_dot(x, p.up, row + 1, p.hidden, p.group);
    if (threadIdx.x % 32 == 0) h[i] = from_f32<T>(g / (1.0f + expf(-g)) * u);
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) down_kernel(const MoeParams p, const T* h) {
  const int64_t items = p.tokens * p.hidden;
  for (int64_t i = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; i < items;
       i += (int64_t)gridDim.x * kWarps) {
    const int64_t t = i / p.hidden, c = i - t * p.hidden;
    float v = 0.0f;
    for (int j = 0; j < p.top_k; ++j) {
      const int64_t pick = t * p.top_k + j;
      const int e = p.ids[pick];
      if (e < 0 || e >= p.experts) {
        if (e >= p.experts) atomicOr(p.status, kStatusBadIndex);
        continue;
      }
      v += p.weights[pick] *
           row_dot(h + pick * p.inter, p.down, (int64_t)e * p.hidden + c, p.inter, p.group);
    }
    if (threadIdx.x % 32 == 0) static_cast<T*>(p.y)[t * p.y_stride + c] = from_f32<T>(v);
  }
}

template <typename T>
cudaError_t moe_typed(const MoeParams& p, void* scratch, int sm_count, cudaStream_t s) {
  up_kernel<T><<<8 * sm_count, 32 * kWarps, 0, s>>>(p, static_cast<T*>(scratch));
  down_kernel<T><<<8 * sm_count, 32 * kWarps, 0, s>>>(p, static_cast<const T*>(scratch));
  return cudaGetLastError();
}

}  // namespace

size_t w4_linear_scratch(W4LinearParams*, int) { return 0; }
cudaError_t launch_w4_linear(int dtype, const W4LinearParams& p, void*, int sm_count,
                             int* launches, cudaStream_t s) {
  *launches += 1;
  if (w4_rows_take_linear(p, sm_count)) return launch_w4_rows_linear(dtype, p, sm_count, s);
  if (dtype == LBGEMM_BF16)
    linear_kernel<__nv_bfloat16><<<8 * sm_count, 32 * kWarps, 0, s>>>(p);
  else
    linear_kernel<__half><<<8 * sm_count, 32 * kWarps, 0, s>>>(p);
  return cudaGetLastError();
}
size_t moe_w4_scratch(MoeParams* p, int) { return (size_t)p->tokens * p->top_k * p->inter * 2; }
cudaError_t launch_moe_w4(int dtype, const MoeParams& p, void* scratch, int sm_count,
                          int* launches, cudaStream_t s) {
  if (w4_rows_take_moe(p, sm_count))
    return launch_w4_rows_moe(dtype, p, scratch, sm_count, launches, s);
  *launches += 2;
  return dtype == LBGEMM_BF16 ? moe_typed<__nv_bfloat16>(p, scratch, sm_count, s)
                              : moe_typed<__half>(p, scratch, sm_count, s);
}

}  // namespace lbg
