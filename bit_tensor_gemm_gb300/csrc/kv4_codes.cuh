// kv4_codes.cuh -- 4-bit codes as halves, and the range of the weights, shared
// by the two attention kernels.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

namespace lbg {

// The reference of a row's weights moves when one exceeds kFar, or a product of a
// weight and a value scale fp16's range; then
constexpr float kFar = 1.2676506e30f;  // 2^100
constexpr int kLevel = 11;             // the largest product is put at 2^11
// ... by the reference alone where a row's largest product with a value scale is
// within 2^-30 .. 2^30 of its largest weight; past that the reference stops, and
// products take a power of two of the row besides, in the careful form of a step
// only.  So weights and sums of one row never stand more than 2^60 apart for their
// values' sake, wherever they are brought to one reference, and stay normal fp32
// numbers.  The same where scores are too large (kFarScore) for a reference that is
// a few binades beside them.
constexpr int kSpan = 30;
constexpr float kSpanLeast = 9.3132257e-10f, kSpanMost = 1.0737418e9f;  // 2^-30, 2^30
constexpr float kFarScore = 4194304.0f;                                  // 2^22: ulps of 1/2

__device__ __forceinline__ float power_of_two(int e) {  // of a normal number
  return __uint_as_float((uint32_t)(127 + e) << 23);
}

// Of a warp's numbers, none negative: the largest, the smallest.
__device__ __forceinline__ float warp_most(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}
__device__ __forceinline__ float warp_least(float x) {
  return __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(x)));
}

// The exponent of the power of two that brings queries whose largest is `most`
// to 2^14 .. 2^15 (0 for zeros): -113 .. 126.
__device__ __forceinline__ int query_power(float most) {
  return most > 0.0f ? min(14 - ((int)(__float_as_uint(most) >> 23) - 127), 126) : 0;
}
// Whether the rows of a tile take powers of their own: the smallest of their
// largest elements would stay below 1, or the tile's power be too far from 1 to be
// a factor of the keys' scales.
__device__ __forceinline__ bool far_queries(float most, float least) {
  const int k = query_power(most);
  return k < -64 || least < power_of_two(-k);
}
// Then the tile's exponent that goes into that factor, and a row's, at most 126
// above it (a row whose scores are 2^-126 of another's has scores of 0).
__device__ __forceinline__ int far_tile_power(float most) { return min(max(query_power(most), -64), 64); }
__device__ __forceinline__ int far_row_power(float row_most, int tile) {
  return min(query_power(row_most), tile + 126);
}

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
