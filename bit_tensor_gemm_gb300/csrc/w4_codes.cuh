// w4_codes.cuh -- 4-bit weights as 16-bit floats.
//
// A code is a signed number of 3 bits and sign (or -8), a group scale an e4m3
// number of 4 significant bits: their product has at most 7 and is exact in bf16
// and (its size being 2^-9 .. 8 * 448) in fp16.  The matrix products run on these
// exact numbers; the fp32 scale of a row multiplies its sum.
//
// In a word of eight codes element 2j sits in bits 4j .. and 2j + 1 in bits 16 +
// 4j .., so a shift and a three-input operation give two neighbouring codes as
// mantissa bits of a pair of halves:
//   ((w >> s) & mask) ^ (base with the codes' sign bit turned) = base + unit (code + 8)
// Logic and shifts run at half the rate of other operations and bound the kernels
// for few tokens, so shifts are spared:
//   bf16  code at mantissa bit 3: 16 + (code + 8), and fma(v, s, -24 s) is exact
//         (24 s has 6 significant bits); pair 0 is taken where it stands, as 128 +
//         (code + 8), and costs an addition of -136 before the product instead;
//   fp16  has mantissa bits for two codes where they stand: 1024 + (code + 8) with
//         an addition of -1032, and 1024 + 16 (code + 8) with fma(v, s / 16, -72 s)
//         (8 significant bits): one shift for the word.
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
  __device__ static __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
  }
  __device__ static __forceinline__ uint32_t mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ static __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
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
  __device__ static __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
  }
  __device__ static __forceinline__ uint32_t mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ static __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
};

// An e4m3 scale as pairs of T: s, and what the fma above takes beside it (bf16: -24 s;
// fp16: s / 16 and -72 s).  s / 16 is exact in fp16 (s is a multiple of 2^-9).
template <typename T>
struct W4Scale;
template <>
struct W4Scale<__nv_bfloat16> {
  uint32_t s, off;
};
template <>
struct W4Scale<__half> {
  uint32_t s, low, off;
};
// Of two bytes, the scales of two rows.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t first, uint32_t second) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(first | second << 8)));
  return h;
}
__device__ __forceinline__ void w4_scales(uint32_t first, uint32_t second,
                                          W4Scale<__nv_bfloat16>& a, W4Scale<__nv_bfloat16>& b) {
  using M = W4Math<__nv_bfloat16>;
  const uint32_t h = e4m3_pair(first, second);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  a.s = M::twice(f.x);
  b.s = M::twice(f.y);
  a.off = M::mul(a.s, 0xc1c0c1c0u);
  b.off = M::mul(b.s, 0xc1c0c1c0u);
}
__device__ __forceinline__ void w4_scales(uint32_t first, uint32_t second, W4Scale<__half>& a,
                                          W4Scale<__half>& b) {
  using M = W4Math<__half>;
  const uint32_t h = e4m3_pair(first, second);
  a.s = __byte_perm(h, h, 0x1010);
  b.s = __byte_perm(h, h, 0x3232);
  a.low = M::mul(a.s, 0x2c002c00u);
  b.low = M::mul(b.s, 0x2c002c00u);
  a.off = M::mul(a.s, 0xd480d480u);
  b.off = M::mul(b.s, 0xd480d480u);
}

// Eight weights of a word, as four pairs in order.
__device__ __forceinline__ void w4_word(uint32_t w, const W4Scale<__nv_bfloat16>& sc,
                                        uint32_t (&out)[4]) {
  using M = W4Math<__nv_bfloat16>;
  out[0] = M::mul(M::add(and_xor(w, 0x000f000fu, 0x43084308u), 0xc308c308u), sc.s);
#pragma unroll
  for (int j = 1; j < 4; ++j)
    out[j] = M::fma(and_xor(w >> (4 * j - 3), 0x00780078u, 0x41c041c0u), sc.s, sc.off);
}
__device__ __forceinline__ void w4_word(uint32_t w, const W4Scale<__half>& sc, uint32_t (&out)[4]) {
  using M = W4Math<__half>;
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const uint32_t v = j == 0 ? w : w >> 8;
    out[j] = M::mul(M::add(and_xor(v, 0x000f000fu, 0x64086408u), 0xe408e408u), sc.s);
    out[j + 1] = M::fma(and_xor(v, 0x00f000f0u, 0x64806480u), sc.low, sc.off);
  }
}

// silu(gate) * up = gate / (1 + exp(-gate)) * up, the same in both kernels.  By e =
// exp(-|gate| / 2), as exp(-gate) passes fp32's range at 88.7, where a large up still makes an
// ordinary number of silu(gate): with one e at the gate and one at up no factor leaves the
// range before the product does, and e and 1 + e^2 stay where the fast instructions are good
// to 2^-22 of themselves (e, by its rounded argument, to |gate| 2^-24).  The result is rounded
// to T, 2^-12 at best.  (4096 tokens, 6 of 64 experts: 351 us, with exp(-gate) 349, with expf
// and a true division 401.)
//
// That rounding is the one place where a mixture holds less than fp32: the result is an operand
// of the second product's MMAs, which take 16 bits.  Errors against 64 bits, of the output's
// size: 2.4e-3 in bf16, 1.7e-3 being the output's own rounding; 3.1e-4 and 2.2e-4 in fp16.  In
// two parts (T(h) and T(h - T(h)), an MMA for each) only the latter is left, at 1.05 times the
// time for 24 tokens (6 of 64 experts of 2048 / 1024: 67.3 -> 70.8 us), 1.11 for 64 (79 -> 88),
// 1.17 for 4096 (355 -> 414) and 1.30 where inter is 4096 (8 experts, 327 -> 425).  That is
// more than the error is worth to a caller whose tokens are of T: one part.
__device__ __forceinline__ float silu_times(float gate, float up) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(gate) * -0.72134752f));  // log2(e) / 2
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e, e, 1.0f)));
  const float s = gate < 0.0f ? e : 1.0f;
  return gate * s * r * (up * s);
}

}  // namespace lbg
