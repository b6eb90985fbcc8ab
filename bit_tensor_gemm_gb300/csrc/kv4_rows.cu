// kv4_rows.cu -- attention over the 4-bit cache for few query rows (a decoding
// step, drafted tokens): tiles of 8 or 16 rows (query tokens x heads of a
// group), streaming the cache once.
//
// Bound by HBM: D + 4 bytes per cached token and head against 4 D flops a
// row.  What an SM must keep up with at the copy rate is about 24 bytes a
// cycle, which is 47 codes to turn into floats, so the design keeps the
// instructions per code low:
//   - warp MMAs with the cached tokens (keys) or channels (values) as the 16
//     rows and the query rows as the 8 columns, so 8 rows cost no padding;
//   - a code becomes a float by one shift and one logical operation on two
//     codes at once: n = code + 8 placed in the mantissa of 16.0 is 16 + n.
//     For keys the constant 24 is taken out of the product by starting the
//     accumulators at -24 sum(q); for values it is subtracted, since there the
//     products add up over thousands of tokens and the constant would cost
//     digits;
//   - the order of channels in a product is free, so a lane's codes are used
//     in the order in which they lie in memory;
//   - the running maximum, and the largest weight seen, move only when a score
//     or weight exceeds them 2^8 or 2^4 times, so almost no step rescales its
//     accumulators.
// Every warp streams its own tokens (32 a step) through its own ring of bulk
// copies, with no barrier between warps until the end.
#include <cuda_runtime.h>

#include <atomic>

#include "kv4_attention.cuh"
#include "ptx.cuh"

namespace lbg {
namespace {

constexpr int kWarps = 4, kStages = 3, kStep = 32;
constexpr float kLeastTop = 2.4074124e-35f;  // 2^-115: 2^11 over it is finite

template <int DIM>
struct Ring {
  static constexpr int kCodes = kStep * DIM / 2;     // bytes of keys (or values) of a step
  static constexpr int kBytes = 2 * kCodes + 4 * kStep;
  static constexpr int kTotal = kWarps * kStages * kBytes;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes i and i + 4 of a word as two 16-bit floats 16 + (code + 8).  The
// nibble goes to the top four bits of the mantissa of 16.0 (7 bits in bf16,
// 10 in fp16), its sign bit flipped by the constant.
template <bool BF16, int I>
__device__ __forceinline__ uint32_t codes24(uint32_t w) {
  constexpr int SHIFT = 4 * I - (BF16 ? 3 : 6);
  constexpr uint32_t MASK = BF16 ? 0x00780078u : 0x03C003C0u;
  constexpr uint32_t SET = BF16 ? 0x41C041C0u : 0x4E004E00u;
  const uint32_t s = SHIFT >= 0 ? w >> (SHIFT >= 0 ? SHIFT : 0) : w << (SHIFT < 0 ? -SHIFT : 0);
  return (s & MASK) ^ SET;
}
// The same as the codes themselves, in fp16.
template <int I>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
  const uint32_t c = codes24<false, I>(w);
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&c), __half2half2(__half(24.0f)));
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Element order inside a warp (lane = 4 g + c):
//   keys    MMA row g of a 16-token tile is token 2 g + e(g), row g + 8 the
//           other token of that pair, e(g) = parity of the low two bits of g:
//           so a lane's two tokens share one 32-bit word of scales, and reads
//           of keys and values by the lanes of a phase fall on different
//           banks (values: two lanes a bank, the least that 8-byte reads of
//           64-byte rows allow).  A lane holds the channels c DIM/4 ... of its
//           tokens; word w, code i and i + 4 make one register.
//   values  lane (g, c) holds the channels g DIM/8 ... of the tokens of MMA
//           rows 2c, 2c + 1, 2c + 8, 2c + 9; MMA tile i, row g is channel
//           g DIM/8 + 2 i, row g + 8 the one after it.
template <typename T, int DIM, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 4 : 3)
    kv4_rows_kernel(const Kv4AttnParams p) {
  constexpr bool BF16 = sizeof(T) == 2 && __is_same(T, __nv_bfloat16);
  constexpr int KW = DIM / 32;   // 32-bit words of a key that a lane holds
  constexpr int VW = DIM / 64;   // of a value
  constexpr int MT = DIM / 16;   // MMA tiles of channels
  constexpr int R = 8 * NT;
  using Rg = Ring<DIM>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ float merge_m[kWarps][R], merge_l[kWarps][R];
  __shared__ int abort_flag;

  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, c = lane % 4;
  const int tile = (int)(blockIdx.x / (unsigned)p.max_chunks);
  const int chunk = (int)(blockIdx.x - (unsigned)tile * p.max_chunks);
  const int head = blockIdx.y, b = blockIdx.z;
  const RowTile t = row_tile(p, b, tile);
  if (chunk >= t.chunks) return;
  const int begin = t.base + chunk * p.chunk;
  const int end = min(t.last, begin + p.chunk);

  const uint32_t bar0 = smem_addr(&bars[warp][0]);
  const uint32_t ring = smem_addr(smem) + (uint32_t)(warp * kStages * Rg::kBytes);
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane < kStages) mbar_init(bar0 + 8 * lane, 1);
  fence_barrier_init();
  __syncthreads();

  // ---- copies: this warp's step s covers the 32 tokens from
  // begin + (s kWarps + warp) 32.  One copy per piece (keys, values, two
  // arrays of scales) and run of tokens in one page: the whole step when
  // pages are multiples of 32, else 16 tokens.
  const int steps = max(0, (end - begin - warp * kStep + kWarps * kStep - 1) / (kWarps * kStep));
  const int runs = p.cache.page_size % kStep ? 2 : 1, run_tokens = kStep / runs;
  const int my_run = lane >> 2, piece = lane & 3;
  const bool copies = lane < 4 * runs;
  const int32_t* table = p.page_table + (int64_t)b * p.table_width;
  const int page16 = (int)(p.cache.page_size / 16);
  const uint32_t piece_bytes =
      (uint32_t)(piece < 2 ? run_tokens * (DIM / 2) : run_tokens * 2);
  const uint32_t piece_dst = (uint32_t)(piece < 2 ? piece * Rg::kCodes + my_run * run_tokens * (DIM / 2)
                                                  : 2 * Rg::kCodes + (piece - 2) * 2 * kStep +
                                                        my_run * run_tokens * 2);
  const int64_t block_bytes = kv4_block_bytes(DIM, p.cache.page_size);
  const int64_t piece_src = (int64_t)p.cache.page_size * (piece < 2 ? piece * (DIM / 2)
                                                                    : DIM + (piece - 2) * 2);
  auto step_token = [&](int s) { return begin + (s * kWarps + warp) * kStep; };
  // page number of this lane's run in step s (-1: no copy)
  auto page_of = [&](int s) -> int {
    const int token = step_token(s) + my_run * run_tokens;
    if (!copies || s >= steps || token >= end) return -1;
    const int page = __ldg(table + p.by_page16((uint32_t)token / 16));
    if (page >= 0 && page < p.cache.pages) return page;
    atomicOr(p.status, kStatusBadIndex);
    return -1;
  };
  auto issue = [&](int s, int page) {
    const uint32_t stage = (uint32_t)(s % kStages), bar = bar0 + 8 * stage;
    uint32_t total = page >= 0 ? piece_bytes : 0;
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    if (lane == 0) mbar_arrive_expect_tx(bar, total);
    __syncwarp();
    if (page >= 0) {
      const uint32_t group = (uint32_t)(step_token(s) + my_run * run_tokens) / 16;
      const int inside = (int)(group - p.by_page16(group) * page16) * 16;
      const uint8_t* src = p.cache.base + ((int64_t)page * p.cache.heads + head) * block_bytes +
                           piece_src + inside * (piece < 2 ? DIM / 2 : 2);
      bulk_load(ring + stage * Rg::kBytes + piece_dst, src, piece_bytes, bar);
    }
  };
  int next_page = page_of(0);
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    const int page = next_page;
    next_page = page_of(s + 1);
    if (s < steps) issue(s, page);
  }

  // ---- queries: B fragments, column g of tile nt is row t.r0 + 8 nt + g
  uint32_t q[NT][MT][2];
  float bias[NT][2];   // -24 sum(q) of columns 2c, 2c + 1
  int seen_to[NT][2];  // one past the last token that columns 2c, 2c + 1 see
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + g;
    uint32_t raw[DIM / 8];  // DIM / 4 elements: two a word
#pragma unroll
    for (int i = 0; i < DIM / 8; ++i) raw[i] = 0;
    if (r < t.rows) {
      const int row = t.r0 + r, i = (int)p.by_group((uint32_t)row);
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const T*>(p.q) + (int64_t)(t.q0 + i) * p.q_stride +
          (int64_t)(head * p.group + row - i * p.group) * DIM + c * (DIM / 4));
#pragma unroll
      for (int i4 = 0; i4 < DIM / 32; ++i4)
        reinterpret_cast<uint4*>(raw)[i4] = __ldg(src + i4);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < DIM / 8; ++i) {
      const T* h = reinterpret_cast<const T*>(&raw[i]);
      sum += to_f32(h[0]) + to_f32(h[1]);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
    for (int e = 0; e < 2; ++e) bias[nt][e] = -24.0f * __shfl_sync(0xffffffffu, sum, 4 * (2 * c + e));
    // channels (d, d + 4) of a word of codes make a register
#pragma unroll
    for (int w = 0; w < KW; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        q[nt][2 * w + i / 2][i % 2] =
            __byte_perm(raw[4 * w + i / 2], raw[4 * w + 2 + i / 2], i % 2 ? 0x7632 : 0x5410);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      seen_to[nt][e] = last_seen(p, t, (int)p.by_group((uint32_t)(t.r0 + 8 * nt + 2 * c + e)));
  }
  // steps wholly inside [all_from, all_to) need no mask
  const int i_last = (int)p.by_group((uint32_t)(t.r0 + t.rows - 1));
  const int all_to = min(end, last_seen(p, t, (int)p.by_group((uint32_t)t.r0)));
  const int all_from = p.window ? max(t.first, first_seen(p, last_seen(p, t, i_last))) : 0;

  const float to_log2 = p.scale * kLog2e;
  const int eg = (g ^ (g >> 1)) & 1;        // e(g)
  const int tok_a = 2 * g + eg, tok_b = 2 * g + 1 - eg;
  const uint32_t sel_a = eg ? 0x3244u : 0x1044u, sel_b = eg ? 0x1044u : 0x3244u;
  const int cp = c & 1;
  // values: byte offsets of the tokens of rows 2c, 2c + 1, 2c + 8, 2c + 9
  const uint32_t v_off[4] = {(uint32_t)(4 * c + cp) * (DIM / 2), (uint32_t)(4 * c + 3 - cp) * (DIM / 2),
                             (uint32_t)(4 * c + 1 - cp) * (DIM / 2), (uint32_t)(4 * c + 2 + cp) * (DIM / 2)};

  // per column: the running maximum m (lagging by at most 2^8), the sum l of
  // the weights 2^(t - m), and the unit of o: weights enter the value product
  // in fp16 as (weight x value scale) 2^11 / wtop, where wtop has been the
  // largest such weight of this column and is followed when one exceeds it
  // 2^4 times: at most 2^15, and normal down to 2^-25 of the largest,
  // whatever scores and scales look like
  float o[MT][NT][4], m[NT][2], l[NT][2], wtop[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[nt][e] = -3.0e38f;
      l[nt][e] = 0.0f;
      wtop[nt][e] = kLeastTop;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][nt][k] = 0.0f;
  }

  bool ok = true;
  for (int s = 0; s < steps; ++s) {
    const uint32_t stage = (uint32_t)(s % kStages);
    ok = ok && mbar_wait(bar0 + 8 * stage, (uint32_t)(s / kStages) & 1u, &abort_flag, p.status);
    if (!ok) {  // a wait ran out: let the copies in flight land (again with a limit)
      volatile int go_on = 0;
      for (int k = 0; k < kStages && s + k < steps; ++k)
        mbar_wait(bar0 + 8 * ((s + k) % kStages), (uint32_t)((s + k) / kStages) & 1u, &go_on,
                  p.status, kWaitLimitNs / 8);
      break;
    }
    const uint8_t* buf = smem + (warp * kStages + stage) * Rg::kBytes;
    const int token0 = step_token(s);
    const bool masked = token0 < all_from || token0 + kStep > all_to;

    float sc[2][NT][4];  // scores of the step's two 16-token tiles, in log2 units
    float vs[2][2];      // value scales of the lane's tokens
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint8_t* kp = buf + mt * 16 * (DIM / 2) + c * (DIM / 8);
      uint32_t ka[KW], kb[KW];
      if constexpr (KW == 4) {
        *reinterpret_cast<uint4*>(ka) = *reinterpret_cast<const uint4*>(kp + tok_a * (DIM / 2));
        *reinterpret_cast<uint4*>(kb) = *reinterpret_cast<const uint4*>(kp + tok_b * (DIM / 2));
      } else {
        *reinterpret_cast<uint2*>(ka) = *reinterpret_cast<const uint2*>(kp + tok_a * (DIM / 2));
        *reinterpret_cast<uint2*>(kb) = *reinterpret_cast<const uint2*>(kp + tok_b * (DIM / 2));
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        sc[mt][nt][0] = sc[mt][nt][2] = bias[nt][0];
        sc[mt][nt][1] = sc[mt][nt][3] = bias[nt][1];
      }
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        {
          const uint32_t a0 = codes24<BF16, 0>(ka[w]), a1 = codes24<BF16, 0>(kb[w]);
          const uint32_t a2 = codes24<BF16, 1>(ka[w]), a3 = codes24<BF16, 1>(kb[w]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816<BF16>(sc[mt][nt], a0, a1, a2, a3, q[nt][2 * w][0], q[nt][2 * w][1]);
        }
        {
          const uint32_t a0 = codes24<BF16, 2>(ka[w]), a1 = codes24<BF16, 2>(kb[w]);
          const uint32_t a2 = codes24<BF16, 3>(ka[w]), a3 = codes24<BF16, 3>(kb[w]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816<BF16>(sc[mt][nt], a0, a1, a2, a3, q[nt][2 * w + 1][0], q[nt][2 * w + 1][1]);
        }
      }
      const uint8_t* scales = buf + 2 * Rg::kCodes + mt * 32 + g * 4;
      const uint32_t ks2 = *reinterpret_cast<const uint32_t*>(scales);
      const uint32_t vs2 = *reinterpret_cast<const uint32_t*>(scales + 2 * kStep);
      const float ks_a = __uint_as_float(__byte_perm(ks2, 0, sel_a)) * to_log2;
      const float ks_b = __uint_as_float(__byte_perm(ks2, 0, sel_b)) * to_log2;
      vs[mt][0] = __uint_as_float(__byte_perm(vs2, 0, sel_a));
      vs[mt][1] = __uint_as_float(__byte_perm(vs2, 0, sel_b));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        sc[mt][nt][0] *= ks_a;
        sc[mt][nt][1] *= ks_a;
        sc[mt][nt][2] *= ks_b;
        sc[mt][nt][3] *= ks_b;
      }
    }
    if (masked) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const int ta = token0 + mt * 16 + tok_a, tb = token0 + mt * 16 + tok_b;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int to = min(end, seen_to[nt][e]), from = max(t.first, first_seen(p, seen_to[nt][e]));
            if (ta >= to || ta < from) sc[mt][nt][e] = -INFINITY;
            if (tb >= to || tb < from) sc[mt][nt][2 + e] = -INFINITY;
          }
      }
    }
    // the running maximum, moved when it must (o keeps its digits: its unit moves)
    bool move = false;
    float high[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        high[nt][e] = fmaxf(fmaxf(sc[0][nt][e], sc[0][nt][2 + e]), fmaxf(sc[1][nt][e], sc[1][nt][2 + e]));
        move |= high[nt][e] > m[nt][e] + 8.0f;
      }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int off = 4; off <= 16; off <<= 1)
            high[nt][e] = fmaxf(high[nt][e], __shfl_xor_sync(0xffffffffu, high[nt][e], off));
          const float next = fmaxf(m[nt][e], high[nt][e]);
          const float keep = ex2(m[nt][e] - next);
          m[nt][e] = next;
          l[nt][e] *= keep;
          wtop[nt][e] *= keep;
        }
    }
    // weights: sc becomes weight x value scale
    move = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float most = 0.0f;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const float pa = ex2(sc[mt][nt][e] - m[nt][e]), pb = ex2(sc[mt][nt][2 + e] - m[nt][e]);
          l[nt][e] += pa + pb;
          float wa = pa * vs[mt][0], wb = pb * vs[mt][1];
          if (masked) {  // what a row does not see has weight 0 whatever its scale
            if (sc[mt][nt][e] == -INFINITY) wa = 0.0f;
            if (sc[mt][nt][2 + e] == -INFINITY) wb = 0.0f;
          }
          sc[mt][nt][e] = wa;
          sc[mt][nt][2 + e] = wb;
          most = fmaxf(most, fmaxf(fabsf(wa), fabsf(wb)));
        }
        high[nt][e] = most;
        move |= most > 16.0f * wtop[nt][e] || wtop[nt][e] < kLeastTop;
      }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int off = 4; off <= 16; off <<= 1)
            high[nt][e] = fmaxf(high[nt][e], __shfl_xor_sync(0xffffffffu, high[nt][e], off));
          const float next = fminf(fmaxf(fmaxf(wtop[nt][e], high[nt][e]), kLeastTop), 3.0e38f);
          const float f = wtop[nt][e] / next;
          wtop[nt][e] = next;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[i][nt][e] *= f;
            o[i][nt][2 + e] *= f;
          }
        }
    }
    // their products with the values
    float to_unit[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) to_unit[nt][e] = __fdividef(2048.0f, wtop[nt][e]);
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t b0[NT], b1[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        b0[nt] = transpose8x8(pack_f16(sc[mt][nt][0] * to_unit[nt][0], sc[mt][nt][1] * to_unit[nt][1]));
        b1[nt] = transpose8x8(pack_f16(sc[mt][nt][2] * to_unit[nt][0], sc[mt][nt][3] * to_unit[nt][1]));
      }
      const uint8_t* vp = buf + Rg::kCodes + mt * 16 * (DIM / 2) + g * (DIM / 16);
      uint32_t v[4][VW];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (VW == 2)
          *reinterpret_cast<uint2*>(v[k]) = *reinterpret_cast<const uint2*>(vp + v_off[k]);
        else
          v[k][0] = *reinterpret_cast<const uint32_t*>(vp + v_off[k]);
      }
#pragma unroll
      for (int w = 0; w < VW; ++w)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // the four codes of this half word, of two tokens side by side
          const uint32_t x = __byte_perm(v[0][w], v[1][w], half ? 0x7632 : 0x5410);
          const uint32_t y = __byte_perm(v[2][w], v[3][w], half ? 0x7632 : 0x5410);
          const int i = w * 4 + half * 2;
          {
            const uint32_t a0 = codes_f16<0>(x), a1 = codes_f16<1>(x);
            const uint32_t a2 = codes_f16<0>(y), a3 = codes_f16<1>(y);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<false>(o[i][nt], a0, a1, a2, a3, b0[nt], b1[nt]);
          }
          {
            const uint32_t a0 = codes_f16<2>(x), a1 = codes_f16<3>(x);
            const uint32_t a2 = codes_f16<2>(y), a3 = codes_f16<3>(y);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<false>(o[i + 1][nt], a0, a1, a2, a3, b0[nt], b1[nt]);
          }
        }
    }
    __syncwarp();  // every lane has read the stage
    const int page = next_page;
    next_page = page_of(s + kStages + 1);
    if (s + kStages < steps) issue(s + kStages, page);
  }

  // ---- join the warps: o, l relative to the common maximum
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1)
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
      if (g == 0) {
        merge_m[warp][8 * nt + 2 * c + e] = m[nt][e];
        merge_l[warp][8 * nt + 2 * c + e] = l[nt][e];
      }
    }
  __syncthreads();  // (also: every ring is drained or abandoned)
  if (abort_flag) return;
  float* mo = reinterpret_cast<float*>(smem);  // [warp][row][DIM]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * nt + 2 * c + e;
      float all = merge_m[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) all = fmaxf(all, merge_m[w][r]);
      const float f = ex2(m[nt][e] - all) * (wtop[nt][e] * (1.0f / 2048.0f));
      float* dst = mo + (warp * R + r) * DIM + g * (DIM / 8);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        dst[2 * i] = o[i][nt][e] * f;
        dst[2 * i + 1] = o[i][nt][2 + e] * f;
      }
    }
  __syncthreads();
  const bool whole = t.chunks == 1;
  const int64_t unit_at = unit_of(p, b, head, tile, chunk);
  for (int i = threadIdx.x; i < R * (DIM / 4); i += kWarps * 32) {
    const int r = i / (DIM / 4), d = i % (DIM / 4) * 4;
    if (r >= t.rows) continue;
    float all = merge_m[0][r], sum = 0.0f;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) all = fmaxf(all, merge_m[w][r]);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sum += merge_l[w][r] * ex2(merge_m[w][r] - all);
      const float4 x = *reinterpret_cast<const float4*>(mo + (w * R + r) * DIM + d);
      v.x += x.x;
      v.y += x.y;
      v.z += x.z;
      v.w += x.w;
    }
    const bool none = sum == 0.0f;
    const float inv = none ? 0.0f : 1.0f / sum;
    v.x *= inv;
    v.y *= inv;
    v.z *= inv;
    v.w *= inv;
    const float lse = none ? -INFINITY : all + log2f(sum);
    if (whole) {
      const int64_t at = out_row(p, t, head, t.r0 + r);
      T h[4] = {from_f32<T>(v.x), from_f32<T>(v.y), from_f32<T>(v.z), from_f32<T>(v.w)};
      *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + at * DIM + d) =
          *reinterpret_cast<const uint2*>(h);
      if (p.lse && d == 0) p.lse[at] = lse * kLn2;
    } else {
      *reinterpret_cast<float4*>(p.share_o + (unit_at * p.tile_rows + r) * DIM + d) = v;
      if (d == 0) p.share_lse[unit_at * p.tile_rows + r] = lse;
    }
  }
}

template <typename T, int DIM, int NT>
cudaError_t launch_tile(const Kv4AttnParams& p, cudaStream_t s) {
  const int merge = kWarps * 8 * NT * DIM * 4;
  const int smem = Ring<DIM>::kTotal > merge ? Ring<DIM>::kTotal : merge;
  auto kernel = kv4_rows_kernel<T, DIM, NT>;
  static std::atomic<uint64_t> set{0};  // devices on which the kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(set.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    set |= uint64_t(1) << dev;
  }
  const dim3 grid((unsigned)(p.max_chunks * p.row_tiles), (unsigned)p.cache.heads,
                  (unsigned)p.batch);
  kernel<<<grid, kWarps * 32, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const Kv4AttnParams& p, cudaStream_t s) {
  if (p.cache.dim == 64)
    return p.tile_rows == 8 ? launch_tile<T, 64, 1>(p, s) : launch_tile<T, 64, 2>(p, s);
  return p.tile_rows == 8 ? launch_tile<T, 128, 1>(p, s) : launch_tile<T, 128, 2>(p, s);
}

}  // namespace

cudaError_t launch_kv4_rows(int dtype, const Kv4AttnParams& p, cudaStream_t s) {
  return dtype == LBGEMM_BF16 ? launch_typed<__nv_bfloat16>(p, s) : launch_typed<__half>(p, s);
}

}  // namespace lbg
