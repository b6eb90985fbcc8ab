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
constexpr float kLeastTop = 8.2718061e-25f;  // 2^-80

// Codes 0 and 4 of a word (HIGH: 1 and 5) as two subnormal halves: (code + 8)
// 2^-24, or 16 times that.  Codes 2, 6 and 3, 7 are those of the word >> 8.
// One three-input operation, (w & mask) ^ eight: left to the compiler it became
// two (45.1 -> XX us over 131072 tokens).
template <bool HIGH>
__device__ __forceinline__ uint32_t codes8(uint32_t w) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;"
      : "=r"(d)
      : "r"(w), "r"(HIGH ? 0x00F000F0u : 0x000F000Fu), "r"(HIGH ? 0x00800080u : 0x00080008u));
  return d;
}
// The same without the 8: code 2^-24, or 16 times that (exact).
template <bool HIGH>
__device__ __forceinline__ uint32_t codes0(uint32_t w) {
  const uint32_t c = codes8<HIGH>(w), eight = HIGH ? 0x00800080u : 0x00080008u;
  const __half2 v =
      __hsub2(*reinterpret_cast<const __half2*>(&c), *reinterpret_cast<const __half2*>(&eight));
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace lbg
