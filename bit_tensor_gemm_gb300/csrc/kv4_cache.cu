// kv4_cache.cu -- the paged cache of keys and values in 4 bits: quantising
// vectors as they are written, and reading them back.
//
//   scale = bf16(max|x| * (1/7)),  code = clamp(rne(x / scale), -7, 7),  value = code * scale
//
// Bound by HBM: a vector of D channels is read once (2 D or 4 D bytes) and
// written as D / 2 + 2 bytes, or the other way round.  A group of D / 8 lanes
// takes a vector, 8 channels a lane (16 bytes of a 16-bit type), and four
// vectors at a time, so that enough loads are on their way.
// Measured, bf16, 30011 tokens of 8 heads of 128: written in 38 us (155 MB), read
// in 26 (155 MB, 33 of them from L2).  The write is bound by its instructions
// (issue 65 %): a division a channel, in pairs.
#include <cuda_runtime.h>

#include <algorithm>

#include "attn.h"
#include "attn_common.cuh"
#include "kv4_codes.cuh"

namespace lbg {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;  // heads of a lane group's token that are in flight

// A lane group takes kAtOnce heads of the keys or the values of a token: item i
// of a block is (token, key or value, chunk of heads) in this order; a block has
// `per_block` consecutive tokens.  What a slot's page and place cost to find is
// so paid once for kAtOnce vectors.
struct Item {
  int64_t token;
  int which, head, heads;  // 0 keys, 1 values; first head and their number
  int64_t stride;          // bytes from a head's block to the next
  uint8_t* codes;          // of the first head (nullptr: the token has no slot)
  __nv_bfloat16* scale;
};
__device__ __forceinline__ Item item_of(const Kv4CopyParams& p, uint32_t i, int dim) {
  Item it;
  const Kv4Cache& c = p.cache;
  const uint32_t row = p.by_chunks(i);
  it.head = (int)(i - row * p.by_chunks.d) * kAtOnce;
  it.heads = min(kAtOnce, c.heads - it.head);
  it.token = (int64_t)blockIdx.x * p.per_block + (row >> 1);
  it.which = (int)(row & 1);
  it.codes = nullptr;
  it.scale = nullptr;
  it.stride = kv4_block_bytes(dim, c.page_size);
  const int64_t slot = __ldg(p.slots + it.token);
  if (slot < 0) return it;
  if (slot >= c.pages * c.page_size) {
    atomicOr(p.status, kStatusBadIndex);
    return it;
  }
  // (slots below 2^31 are divided by multiplication)
  const int64_t page = slot <= INT32_MAX ? (int64_t)p.by_page((uint32_t)slot) : slot / c.page_size;
  const int64_t at = slot - page * c.page_size;
  uint8_t* block = c.base + (page * c.heads + it.head) * it.stride;
  it.codes = block + (it.which * c.page_size + at) * (dim / 2);
  it.scale = reinterpret_cast<__nv_bfloat16*>(block + c.page_size * dim) + it.which * c.page_size + at;
  return it;
}
__device__ __forceinline__ uint32_t items_of_block(const Kv4CopyParams& p) {
  const int64_t tokens = min((int64_t)p.per_block, p.tokens - (int64_t)blockIdx.x * p.per_block);
  return (uint32_t)tokens * 2 * p.by_chunks.d;
}
template <typename T>
__device__ __forceinline__ T* tensor_at(const Kv4CopyParams& p, const Item& it, int dim) {
  return static_cast<T*>(it.which ? p.v : p.k) + it.token * (it.which ? p.v_stride : p.k_stride) +
         it.head * dim;
}

// The largest magnitude of eight elements, as an fp32 bit pattern in which NaNs
// order above infinity (so a NaN channel makes the scale NaN).
template <typename T>
__device__ __forceinline__ uint32_t magnitude(const Raw8<T>& r) {
  uint32_t top = 0;
  if constexpr (sizeof(T) == 2) {
    // the halves' bit patterns without their signs, two at a time
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
    uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    const uint16_t h = (uint16_t)max(m & 0xffffu, m >> 16);
    top = __float_as_uint(to_f32(*reinterpret_cast<const T*>(&h)));
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, w[i] & 0x7fffffffu);
  }
  return top;
}

// The codes of eight elements over scale s, as a word.
template <typename T>
__device__ __forceinline__ uint32_t codes_of(const Raw8<T>& r, float s) {
  float x[8];
  unpack8(r, x);
  if (sizeof(T) == 2 && s >= 7.8886091e-31f && s <= 3.4e38f) {  // 2^-100 and finite
    // x / s, correctly rounded, from the correctly rounded reciprocal y: q = x y,
    // then q + (x - s q) y (Markstein, "Computation of elementary functions on the
    // IBM RISC System/6000 processor", 1990).  The remainder is exact here (no
    // underflow above 2^-100); |x / s| < 7.02 needs no clamp.  Adding and taking
    // away 1.5 2^23 rounds to a whole number, half to even; + 8 makes it 1 .. 15,
    // and four of those are put together as fp32 numbers below 2^16.
    const float y = __frcp_rn(s);
    const uint64_t y2 = pair(y, y), s2 = pair(-s, -s);
    uint64_t word = 0;  // elements 0..3 and 4..7
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      const uint64_t x2 = pair(x[i], x[i + 4]);
      uint64_t q = mul2(x2, y2);
      q = fma2(fma2(s2, q, x2), y2, q);
      q = add2(add2(q, pair(12582912.0f, 12582912.0f)), pair(-12582904.0f, -12582904.0f));
      word = i == 3 ? q : fma2(word, pair(16.0f, 16.0f), q);
    }
    float lo, hi;
    unpair(add2(word, pair(8388608.0f, 8388608.0f)), lo, hi);  // whole numbers in the low bits
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410) ^ 0x88888888u;
  }
  uint32_t word = 0;
  const bool ok = s > 0.0f && s <= 3.4e38f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -7.0f), 7.0f);
    word |= ((uint32_t)(int)(ok ? q : 0.0f) & 15u) << (4 * i);
  }
  return word;
}

template <typename T, int LPH>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const Kv4CopyParams p) {
  constexpr int GROUPS = kThreads / LPH, DIM = LPH * 8;
  const int lane = threadIdx.x % LPH;
  const uint32_t count = items_of_block(p);
  // (the lanes of a warp shuffle together: a group without an item takes the
  // last one again and stores nothing)
  for (uint32_t first = 0; first < count; first += GROUPS) {
    const uint32_t i = first + threadIdx.x / LPH;
    const Item it = item_of(p, min(i, count - 1), DIM);
    const T* src = tensor_at<T>(p, it, DIM) + lane * 8;
    Raw8<T> raw[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) raw[u] = load8_raw(src + (u < it.heads ? u : 0) * DIM);
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      uint32_t top = magnitude(raw[u]);
#pragma unroll
      for (int off = LPH / 2; off >= 1; off >>= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
      const __nv_bfloat16 scale = __float2bfloat16_rn(__uint_as_float(top) * (1.0f / 7.0f));
      const uint32_t word = codes_of(raw[u], __bfloat162float(scale));
      if (i >= count || u >= it.heads || it.codes == nullptr) continue;
      reinterpret_cast<uint32_t*>(it.codes + u * it.stride)[lane] = word;
      if (lane == 0)
        *reinterpret_cast<__nv_bfloat16*>(reinterpret_cast<uint8_t*>(it.scale) + u * it.stride) = scale;
    }
  }
}

template <typename T, int LPH>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4CopyParams p) {
  constexpr int GROUPS = kThreads / LPH, DIM = LPH * 8;
  const int lane = threadIdx.x % LPH;
  const uint32_t count = items_of_block(p);
  for (uint32_t i = threadIdx.x / LPH; i < count; i += GROUPS) {
    const Item it = item_of(p, i, DIM);
    uint32_t word[kAtOnce];
    float scale[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      word[u] = 0;
      scale[u] = 0.0f;
      if (it.codes != nullptr && u < it.heads) {
        word[u] = __ldg(reinterpret_cast<const uint32_t*>(it.codes + u * it.stride) + lane);
        scale[u] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
            reinterpret_cast<const uint8_t*>(it.scale) + u * it.stride));
      }
    }
    T* dst = tensor_at<T>(p, it, DIM) + lane * 8;
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (u >= it.heads) continue;
      float x[8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // codes 0, 4 and 1, 5; then 2, 6 and 3, 7
        const uint32_t w = k ? word[u] >> 8 : word[u];
        const uint32_t lo = codes_f16<false>(w), hi = codes_f16<true>(w);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        // (the codes' unit first: exact, whatever the scale)
        x[2 * k] = a.x * (1.0f / kCodeUnit) * scale[u];
        x[2 * k + 4] = a.y * (1.0f / kCodeUnit) * scale[u];
        x[2 * k + 1] = b.x * (1.0f / kCodeUnit) * scale[u];
        x[2 * k + 5] = b.y * (1.0f / kCodeUnit) * scale[u];
      }
      store8(dst + u * DIM, x);
    }
  }
}

template <typename T>
cudaError_t launch_typed(bool write, Kv4CopyParams p, cudaStream_t s) {
  const int lph = p.cache.dim / 8;
  const int chunks = (p.cache.heads + kAtOnce - 1) / kAtOnce;
  p.per_block = std::max(1, kThreads / lph / (2 * chunks));  // an item for every lane group
  p.by_chunks = FastDiv((uint32_t)chunks);
  p.by_page = FastDiv((uint32_t)p.cache.page_size);
  const unsigned blocks = (unsigned)((p.tokens + p.per_block - 1) / p.per_block);
  if (lph == 8) {
    if (write) kv4_write_kernel<T, 8><<<blocks, kThreads, 0, s>>>(p);
    else kv4_read_kernel<T, 8><<<blocks, kThreads, 0, s>>>(p);
  } else {
    if (write) kv4_write_kernel<T, 16><<<blocks, kThreads, 0, s>>>(p);
    else kv4_read_kernel<T, 16><<<blocks, kThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_copy(bool write, int dtype, const Kv4CopyParams& p, cudaStream_t s) {
  if (dtype == LBGEMM_BF16) return launch_typed<__nv_bfloat16>(write, p, s);
  if (dtype == LBGEMM_F16) return launch_typed<__half>(write, p, s);
  return launch_typed<float>(write, p, s);
}

}  // namespace

cudaError_t launch_kv4_write(int dtype, const Kv4CopyParams& p, cudaStream_t s) {
  return launch_copy(true, dtype, p, s);
}

cudaError_t launch_kv4_read(int dtype, const Kv4CopyParams& p, cudaStream_t s) {
  return launch_copy(false, dtype, p, s);
}

}  // namespace lbg
