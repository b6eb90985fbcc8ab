// w4_quantize.cu -- weights into 4-bit codes with a scale for every group and
// row (the steps are in include/lbgemm.h).  Done once for a set of weights: 11008 x 4096 in 60 us
// of bf16 and 59 of fp32 (1.9 and 3.5 TB/s), 128000 x 4096 in 0.65 and 0.63 ms.
//
// A block a row: its largest size, then groups of 32, 64 or 128 elements by 4, 8
// or 16 lanes of 8 elements each, which make one word of codes a lane.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "ffn.h"

namespace lbg {
namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) w4_quantize_kernel(const W4QuantParams p) {
  __shared__ float tops[kThreads / 32];
  const int64_t row = blockIdx.x;
  const T* w = static_cast<const T*>(p.w) + row * p.w_stride;
  const int lane = threadIdx.x % 32;
  const int octets = (int)(p.k / 8);
  float top = 0.0f;  // NaN and infinity of any element stay (compared as bits)
  for (int o = threadIdx.x; o < octets; o += kThreads) {
    float f[8];
    unpack8(load8_raw(w + (int64_t)o * 8), f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(f[i]) & 0x7fffffffu));
  }
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
  if (lane == 0) tops[threadIdx.x / 32] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i)
    top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(tops[i])));
  const bool finite = top < INFINITY;
  const float size = finite ? __fmul_rn(top, 1.0f / 3136.0f) : NAN;
  if (threadIdx.x == 0) p.row_scales[row * p.row_stride] = size;
  const bool any = finite && size > 0.0f;

  const int lanes = (int)p.group / 8;
  uint32_t* codes = reinterpret_cast<uint32_t*>(p.codes + row * p.code_stride);
  for (int first = threadIdx.x - lane; first < octets; first += kThreads) {
    const int o = first + lane;  // (octets is a multiple of a group's lanes, not of 32)
    float f[8] = {};
    if (o < octets) unpack8(load8_raw(w + (int64_t)o * 8), f);
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(f[i]));
    for (int off = lanes / 2; off >= 1; off >>= 1)
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
    if (o >= octets) continue;
    const __nv_fp8_storage_t s8 =
        any ? __nv_cvt_float_to_fp8(__fdiv_rn(__fmul_rn(most, 1.0f / 7.0f), size), __NV_SATFINITE,
                                    __NV_E4M3)
            : 0;
    const float step = __fmul_rn(
        __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3))), any ? size : 0.0f);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = step > 0.0f ? rintf(__fdiv_rn(f[i], step)) : 0.0f;
      const int c = (int)fminf(fmaxf(q, -7.0f), 7.0f);
      word |= (uint32_t)(c & 15) << (4 * (i / 2) + 16 * (i % 2));
    }
    codes[o] = word;
    if (o % lanes == 0) p.scales[row * p.scale_stride + o / lanes] = s8;
  }
}

}  // namespace

cudaError_t launch_w4_quantize(int dtype, const W4QuantParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)p.rows;
  if (dtype == LBGEMM_BF16)
    w4_quantize_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
  else if (dtype == LBGEMM_F16)
    w4_quantize_kernel<__half><<<grid, kThreads, 0, s>>>(p);
  else
    w4_quantize_kernel<float><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace lbg
