// kv4_cache.cu -- the paged cache of keys and values in 4 bits: quantising
// vectors as they are written, and reading them back.
//
//   scale = bf16(max|x| * (1/7)),  code = clamp(rne(x / scale), -7, 7),  value = code * scale
//
// Bound by HBM: a vector of D channels is read once (2 D or 4 D bytes) and
// written as D / 2 + 2 bytes, or the other way round.
#include <cuda_runtime.h>

#include <algorithm>

#include "attn.h"
#include "attn_common.cuh"

namespace lbg {
namespace {

constexpr int kThreads = 256;

// Where a vector of the cache lives.  which: 0 key, 1 value.
struct Place {
  uint8_t* codes;
  __nv_bfloat16* scale;
};
__device__ __forceinline__ Place place_of(const Kv4Cache& c, int64_t page, int64_t at, int head,
                                          int which) {
  uint8_t* block = c.base + (page * c.heads + head) * kv4_block_bytes(c.dim, c.page_size);
  Place pl;
  pl.codes = block + (which * c.page_size + at) * (c.dim / 2);
  pl.scale = reinterpret_cast<__nv_bfloat16*>(block + c.page_size * c.dim) +
             which * c.page_size + at;
  return pl;
}

// One lane group of LPH = dim / 8 lanes per vector; vector index = (token *
// 2 + which) * heads + head.
struct Vector {
  int64_t token;
  int head, which;
};
__device__ __forceinline__ Vector vector_of(const Kv4CopyParams& p, int64_t i) {
  Vector v;
  const int64_t row = i / p.cache.heads;
  v.head = (int)(i - row * p.cache.heads);
  v.token = row >> 1;
  v.which = (int)(row & 1);
  return v;
}

template <typename T, int LPH>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const Kv4CopyParams p, int64_t count) {
  const int lane = threadIdx.x % LPH;
  const int64_t index = (int64_t)blockIdx.x * (kThreads / LPH) + threadIdx.x / LPH;
  const Vector v = vector_of(p, index < count ? index : count - 1);
  const int64_t slot = p.slots[v.token];
  bool live = index < count && slot >= 0;
  const int64_t page = slot / p.cache.page_size;
  if (live && page >= p.cache.pages) {
    atomicOr(p.status, kStatusBadIndex);
    live = false;
  }
  const T* src = static_cast<const T*>(v.which ? p.v : p.k) +
                 v.token * (v.which ? p.v_stride : p.k_stride) + v.head * (LPH * 8) + lane * 8;
  float x[8];
  load8(src, x);
  // the largest magnitude as a bit pattern: NaNs order above infinity, so a
  // NaN channel makes the scale NaN
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
  for (int off = LPH / 2; off >= 1; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  const __nv_bfloat16 scale = __float2bfloat16_rn(__uint_as_float(top) * (1.0f / 7.0f));
  const float s = __bfloat162float(scale);
  const bool ok = s > 0.0f && s <= 3.4e38f;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -7.0f), 7.0f);
    word |= ((uint32_t)(int)(ok ? q : 0.0f) & 15u) << (4 * i);
  }
  if (!live) return;
  const Place pl = place_of(p.cache, page, slot - page * p.cache.page_size, v.head, v.which);
  reinterpret_cast<uint32_t*>(pl.codes)[lane] = word;
  if (lane == 0) *pl.scale = scale;
}

template <typename T, int LPH>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4CopyParams p, int64_t count) {
  const int lane = threadIdx.x % LPH;
  const int64_t index = (int64_t)blockIdx.x * (kThreads / LPH) + threadIdx.x / LPH;
  if (index >= count) return;
  const Vector v = vector_of(p, index);
  const int64_t slot = p.slots[v.token];
  const int64_t page = slot / p.cache.page_size;
  float x[8] = {};
  if (slot >= 0 && page >= p.cache.pages) {
    atomicOr(p.status, kStatusBadIndex);
  } else if (slot >= 0) {
    const Place pl = place_of(p.cache, page, slot - page * p.cache.page_size, v.head, v.which);
    const uint32_t word = reinterpret_cast<const uint32_t*>(pl.codes)[lane];
    const float s = __bfloat162float(*pl.scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)nibble_value(word >> (4 * i)) * s;
  }
  T* dst = static_cast<T*>(v.which ? p.v : p.k) +
           v.token * (v.which ? p.v_stride : p.k_stride) + v.head * (LPH * 8) + lane * 8;
  store8(dst, x);
}

template <typename T>
void launch_typed(bool write, const Kv4CopyParams& p, cudaStream_t s) {
  const int64_t count = p.tokens * 2 * p.cache.heads;
  const int lph = p.cache.dim / 8;
  const unsigned blocks = (unsigned)((count + kThreads / lph - 1) / (kThreads / lph));
  if (lph == 8) {
    if (write) kv4_write_kernel<T, 8><<<blocks, kThreads, 0, s>>>(p, count);
    else kv4_read_kernel<T, 8><<<blocks, kThreads, 0, s>>>(p, count);
  } else {
    if (write) kv4_write_kernel<T, 16><<<blocks, kThreads, 0, s>>>(p, count);
    else kv4_read_kernel<T, 16><<<blocks, kThreads, 0, s>>>(p, count);
  }
}

cudaError_t launch_copy(bool write, int dtype, const Kv4CopyParams& p, cudaStream_t s) {
  if (dtype == LBGEMM_BF16) launch_typed<__nv_bfloat16>(write, p, s);
  else if (dtype == LBGEMM_F16) launch_typed<__half>(write, p, s);
  else launch_typed<float>(write, p, s);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_write(int dtype, const Kv4CopyParams& p, int, cudaStream_t s) {
  return launch_copy(true, dtype, p, s);
}

cudaError_t launch_kv4_read(int dtype, const Kv4CopyParams& p, int, cudaStream_t s) {
  return launch_copy(false, dtype, p, s);
}

}  // namespace lbg
