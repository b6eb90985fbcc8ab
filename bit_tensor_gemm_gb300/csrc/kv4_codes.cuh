// kv4_codes.cuh -- 4-bit codes as halves, and the range of the weights, shared
// by the two attention kernels.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

namespace lbg {

// The reference of a row's weights moves when one exceeds kFar, and is set for
// a largest product of at least kLeastTop.
constexpr float kFar = 1.2676506e30f;       // 2^100
constexpr int kLevel = 11;  // the largest product is put at 2^11
// ... by the reference alone where a row's largest product with a value scale is
// within 2^-60 .. 2^60 of its largest weight; past that the reference stops, so
// that weights and their sum stay normal fp32 numbers, and products take a power of
// two of the row besides, in the careful form of a step only.
constexpr int kSpan = 60;
constexpr float kSpanLeast = 8.6736174e-19f, kSpanMost = 1.1529215e18f;  // 2^-60, 2^60

// Codes 0 and 4 of a word (HIGH: 1 and 5) as two halves in units of kCodeUnit;
// codes 2, 6 and 3, 7 are those of the word >> 8.  One three-input logical
// operation, (w & mask) ^ eight, makes subnormals (code + 8) 2^-24, or 16 times
// that (left to the compiler it became two: 45.1 -> 37.8 us over 131072 tokens);
// a multiply-add brings them to normal numbers and takes the 8 out, exactly.
// MMAs would take the subnormals exactly too, but line products up by their
// operands' exponents before they drop digits: a subnormal's leading zeros then
// cost up to 8 digits of a score (log-sums off by 6.7e-7 of themselves).
constexpr float kCodeUnit = 1.0f / 512.0f;
template <bool HIGH>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
  uint32_t c;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;"
      : "=r"(c)
      : "r"(w), "r"(HIGH ? 0x00F000F0u : 0x000F000Fu), "r"(HIGH ? 0x00800080u : 0x00080008u));
  const uint32_t up = HIGH ? 0x68006800u : 0x78007800u;  // 2^11, 2^15
  const uint32_t eight = 0xA400A400u;                    // -8 kCodeUnit
  const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&c),
                            *reinterpret_cast<const __half2*>(&up),
                            *reinterpret_cast<const __half2*>(&eight));
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace lbg
