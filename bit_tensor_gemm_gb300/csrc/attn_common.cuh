// attn_common.cuh -- element conversions shared by the attention operators.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace lbg {

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) {
  return __half2float(x);
}
template <>
__device__ __forceinline__ float to_f32<float>(float x) {
  return x;
}

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) {
  return __float2half_rn(x);
}
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}

// Eight consecutive elements at a 16-byte-aligned address (16-bit types) or
// 32 bytes at one (fp32), as loaded: 16 or 32 bytes in registers.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) == 4 ? 2 : 1];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load8_raw(const T* p) {
  Raw8<T> r;
  r.v[0] = reinterpret_cast<const uint4*>(p)[0];
  if constexpr (sizeof(T) == 4) r.v[1] = reinterpret_cast<const uint4*>(p)[1];
  return r;
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&f)[8]) {
  const T* h = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = to_f32(h[i]);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  Raw8<T> r;
  T* h = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = from_f32<T>(f[i]);
  reinterpret_cast<uint4*>(p)[0] = r.v[0];
  if constexpr (sizeof(T) == 4) reinterpret_cast<uint4*>(p)[1] = r.v[1];
}

// Four consecutive elements: 8 bytes (16-bit types) or 16 (fp32).
template <typename T>
struct Raw4 {
  uint2 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&f)[4]) {
  Raw4<T> r;
  if constexpr (sizeof(T) == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r.v[0] = make_uint2(v.x, v.y);
    r.v[1] = make_uint2(v.z, v.w);
  } else {
    r.v[0] = *reinterpret_cast<const uint2*>(p);
  }
  const T* h = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = to_f32(h[i]);
}

template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&f)[4]) {
  Raw4<T> r;
  T* h = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = from_f32<T>(f[i]);
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<uint4*>(p) = make_uint4(r.v[0].x, r.v[0].y, r.v[1].x, r.v[1].y);
  else
    *reinterpret_cast<uint2*>(p) = r.v[0];
}

// ---- two fp32 numbers in one operation ------------------------------------------
using float2x = uint64_t;
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

}  // namespace lbg
