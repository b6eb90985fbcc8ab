// moe_route.cu -- the top experts of every token and their weights.
//
//   ids[t][j]: the j-th largest of a token's logits, the lower index first among
//   equals; weights[t][j] = exp(l - top) / sum exp(l' - top), the sum over the
//   chosen experts or over all.
//
// A warp a token: the logits sit in registers as sortable 32-bit keys, and each
// of the top_k rounds is two warp reductions (the largest key; the lowest expert
// that has it), so ties are settled by value and index and by nothing else.
// Bound by the launch up to thousands of tokens.
#include <cuda_runtime.h>

#include <cfloat>

#include "attn_common.cuh"
#include "ffn.h"

namespace lbg {
namespace {

constexpr int kWarps = 4;

// A key that orders as the numbers do (0: never chosen).  NaN and -inf are never
// chosen, +inf counts as the largest finite number, -0 as 0.
__device__ __forceinline__ float usable(float x) {
  if (!(x > -INFINITY)) return -INFINITY;
  return fminf(x, FLT_MAX) + 0.0f;
}
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x == -INFINITY) return 0;
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float number_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// PER: experts a lane holds, expert 32 i + lane in place i.
template <typename T, int PER>
__global__ void __launch_bounds__(32 * kWarps) moe_route_kernel(const RouteParams p) {
  const int lane = threadIdx.x % 32;
  const int64_t token = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  if (token >= p.tokens) return;
  const T* row = static_cast<const T*>(p.logits) + token * p.stride;
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = 32 * i + lane;
    key[i] = e < p.experts ? key_of(usable(to_f32(row[e]))) : 0;
  }
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) best = max(best, key[i]);
  const uint32_t first = __reduce_max_sync(0xffffffffu, best);
  const float top = number_of(first);
  float all = 0.0f;
  if (!p.renormalize) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i]) all += expf(number_of(key[i]) - top);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
  }
  // lane j keeps the j-th choice
  int id = -1;
  uint32_t chosen = 0;
  for (int j = 0; j < p.top_k; ++j) {
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    if (most == 0) break;
    uint32_t at = 0xffffffffu;
    if (best == most) {
#pragma unroll
      for (int i = PER - 1; i >= 0; --i)
        if (key[i] == most) at = 32 * i + lane;
    }
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == j) id = (int)at, chosen = most;
    if (lane == (at & 31)) {
      best = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (32 * i + lane == at) key[i] = 0;
        best = max(best, key[i]);
      }
    }
  }
  float w = chosen ? expf(number_of(chosen) - top) : 0.0f;
  if (p.renormalize) {
    all = w;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
  }
  if (lane < p.top_k) {
    p.ids[token * p.top_k + lane] = id;
    p.weights[token * p.top_k + lane] = id < 0 ? 0.0f : w / all;
  }
}

template <typename T>
cudaError_t launch_typed(const RouteParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)((p.tokens + kWarps - 1) / kWarps);
  const int per = (p.experts + 31) / 32;
  if (per <= 1)
    moe_route_kernel<T, 1><<<grid, 32 * kWarps, 0, s>>>(p);
  else if (per <= 2)
    moe_route_kernel<T, 2><<<grid, 32 * kWarps, 0, s>>>(p);
  else if (per <= 4)
    moe_route_kernel<T, 4><<<grid, 32 * kWarps, 0, s>>>(p);
  else if (per <= 8)
    moe_route_kernel<T, 8><<<grid, 32 * kWarps, 0, s>>>(p);
  else if (per <= 16)
    moe_route_kernel<T, 16><<<grid, 32 * kWarps, 0, s>>>(p);
  else
    moe_route_kernel<T, 32><<<grid, 32 * kWarps, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_route(int dtype, const RouteParams& p, cudaStream_t s) {
  if (dtype == LBGEMM_BF16) return launch_typed<__nv_bfloat16>(p, s);
  if (dtype == LBGEMM_F16) return launch_typed<__half>(p, s);
  return launch_typed<float>(p, s);
}

}  // namespace lbg
