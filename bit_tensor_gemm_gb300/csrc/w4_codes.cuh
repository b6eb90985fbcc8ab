// w4_codes.cuh -- 4-bit weights as 16-bit floats.
//
// A code is a signed number of 3 bits and sign (or -8), a group scale an e4m3
// number of 4 significant bits: their product has at most 7 and is exact in bf16
// and (its size being 2^-9 .. 8 * 448) in fp16.  The matrix products run on these
// exact numbers; the fp32 scale of a row multiplies its sum.
//
// In a word of eight codes element 2j sits in bits 4j .. and 2j + 1 in bits 16 +
// 4j .., so one shift and one three-input operation give two neighbouring codes
// as the top mantissa bits of halves between 16 and 32:
//   ((w << s) & mask) ^ (16.0 with the sign bit of the code turned) = 16 + (code + 8)
// and one multiply-add with (scale, -24 scale) takes the 24 out, exactly: 24
// scale has 6 significant bits.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace lbg {

// (a & b) ^ c in one operation.
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

template <typename T>
struct W4Math;

template <>
struct W4Math<__nv_bfloat16> {
  static constexpr int kUp = 3;  // a code's place in 16.0's mantissa
  static constexpr uint32_t kMask = 0x00780078u, kBase = 0x41c041c0u;
  __device__ static __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
  }
  __device__ static __forceinline__ uint32_t twice(float x) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(d) : "f"(x));
    return d;
  }
};
template <>
struct W4Math<__half> {
  static constexpr int kUp = 6;
  static constexpr uint32_t kMask = 0x03c003c0u, kBase = 0x4e004e00u;
  __device__ static __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
  }
  __device__ static __forceinline__ uint32_t twice(float x) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(d) : "f"(x));
    return d;
  }
};

// An e4m3 scale (s, s) and (-24 s, -24 s) as pairs of T.
struct W4Scale {
  uint32_t s, off;
};
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)byte));
  return __half2float(__ushort_as_half((uint16_t)h));
}
template <typename T>
__device__ __forceinline__ W4Scale w4_scale(uint32_t byte) {
  const float s = e4m3_value(byte & 0xffu);
  return {W4Math<T>::twice(s), W4Math<T>::twice(-24.0f * s)};
}

// Eight weights of a word, as four pairs in order.
template <typename T>
__device__ __forceinline__ void w4_word(uint32_t w, const W4Scale& sc, uint32_t (&out)[4]) {
  using M = W4Math<T>;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int up = M::kUp - 4 * j;
    const uint32_t at = up >= 0 ? w << (up & 31) : w >> (-up & 31);
    out[j] = M::fma(and_xor(at, M::kMask, M::kBase), sc.s, sc.off);
  }
}

}  // namespace lbg
