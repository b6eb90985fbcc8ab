// moe_route.cu -- the top experts of every token and their weights.
//
//   ids[t][j]: the j-th largest of a token's logits, the lower index first among
//   equals; weights[t][j] = exp(l - top) / sum exp(l' - top), the sum over the
//   chosen experts or over all.
//
// A warp a token: the logits sit in registers as sortable 32-bit keys, and each
// of the top_k rounds takes the largest by warp reductions, so ties are settled by
// value and index and by nothing else.  A 16-bit logit leaves room for the expert in
// its key's low bits, and one reduction a round finds both; of fp32 logits a second
// one finds the lowest expert that has the largest key (16384 tokens, 8 of 128: 9.5 us in
// 16 bits, 12.2 in fp32).  Bound by the launch up to thousands of tokens, then by logic
// operations.
#include <cuda_runtime.h>

#include <cfloat>

#include "attn_common.cuh"
#include "ffn.h"

namespace lbg {
namespace {

constexpr int kWarps = 4;

// Low bits of a key that the type's numbers leave free: it has 8 exponent bits and
// T's mantissa bits.
template <typename T>
constexpr int kFree = 0;
template <>
constexpr int kFree<__nv_bfloat16> = 16;
template <>
constexpr int kFree<__half> = 13;

// A key that orders as the numbers do (0: never chosen), the lower expert first among
// equals where there is room.  NaN and -inf are never chosen, +inf counts as the largest
// finite fp32 number (which no 16-bit number is, so there its key is inf's own), -0 as 0.
template <typename T>
__device__ __forceinline__ uint32_t key_of(T logit, int expert) {
  constexpr uint32_t low = (1u << kFree<T>) - 1;
  float x = to_f32(logit);
  if (!(x > -INFINITY)) return 0;
  if (low == 0) x = fminf(x, FLT_MAX);
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t key = u & 0x80000000u ? ~u : u | 0x80000000u;
  return low ? (key & ~low) | (low - expert) : key;
}
template <typename T>
__device__ __forceinline__ float number_of(uint32_t key) {
  constexpr uint32_t low = (1u << kFree<T>) - 1;
  return fminf(__uint_as_float(key & 0x80000000u ? key & 0x7fffffffu & ~low : ~(key | low)),
               FLT_MAX);
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
    key[i] = e < p.experts ? key_of(row[e], e) : 0;
  }
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) best = max(best, key[i]);
  const uint32_t first = __reduce_max_sync(0xffffffffu, best);
  const float top = number_of<T>(first);
  float all = 0.0f;
  if (!p.renormalize) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i]) all += expf(number_of<T>(key[i]) - top);
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
    if (kFree<T> > 0) {
      constexpr uint32_t low = (1u << kFree<T>) - 1;
      at = low - (most & low);
    } else {
      if (best == most) {
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
          if (key[i] == most) at = 32 * i + lane;
      }
      at = __reduce_min_sync(0xffffffffu, at);
    }
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
  float w = chosen ? expf(number_of<T>(chosen) - top) : 0.0f;
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
