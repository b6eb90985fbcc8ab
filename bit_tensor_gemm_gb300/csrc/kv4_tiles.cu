// kv4_tiles.cu -- attention over the 4-bit cache for many query rows (prompts,
// chunks of prompts): tiles of 256 rows on the tensor cores, tcgen05.mma with
// scores, weights and sums in tensor memory.
//
// A CTA (one an SM) holds the queries of two 128-row tiles X = 0, 1 in shared
// memory and walks over the cached tokens in steps of 128:
//
//   converters (4 warps for keys, 3 for values)
//                          codes of a step -> fp16 in shared memory, for S = Q
//                          K^T and O += P V, each once for both tiles
//   one warp               the MMAs: O_X += P_X V of step j - 1, then S_X = Q_X
//                          K^T of step j, for X = 0, then 1
//   softmax (4 warps an X) weights 2^(t - ref) from S_X, times the value scales
//                          as fp16 back to tensor memory, over the S they came
//                          from.  A thread takes four rows' pairs of columns
//                          (the layout of a warp MMA's sums): with a thread a
//                          row each scale was read once a row, and these reads
//                          alone held shared memory for 2048 cycles a step
//
// While the tensor cores work for one tile, the other tile's softmax runs.
// The floor is the MMAs, 4 x 128 x DIM flops per row and step (2150 cycles for
// DIM = 128); the converters' and softmax's instructions must fit beside them,
// which is why both scales stay factors of columns, the weights need no maximum
// (the reference moves only when a product with a value scale leaves fp16's
// range, as in kv4_rows.cu), and arithmetic goes in pairs (f32x2).
// Measured: 4096 queries of 32 heads over 16384 tokens (962 GFLOP) 1.02 ms, 0.94
// PFLOP/s; 7 prompts of up to 1100 tokens, DIM = 64, 139 us.  A step takes 5000
// cycles: what bounds it is the chain score MMA - weights - value MMA of a half,
// with one softmax warp of a half on each of the SM's quarters (issue 48 %, MMAs
// 40 %, exponentials 20 % of their rates); with 128 channels tensor memory is full
// with two halves' scores and sums, so a third half to fill the gaps has no room
// (with 64, a quarter of its columns is free).
#include <cuda_runtime.h>

#include <atomic>

#include "kv4_attention.cuh"
#include "kv4_codes.cuh"
#include "ptx.cuh"

namespace lbg {
namespace {

// Warps 0..3, 4..7 softmax, 8..11 keys, 12 MMAs, 13..15 values.  Launched with
// 128 registers a thread (512 threads: all of the SM's); the softmax warps then
// go up to 152 and the others down to 104: 152 + 152 + 104 + 104 = 4 x 128 in
// each quarter of the register file.  The block has no more than it was launched
// with, and a warp waits without a limit for what it asks: the launch checks that
// the compiler did give the kernel 128 (a block of 17 warps once got 96, and
// waited for ever).
constexpr int kThreads = 512, kSoftmaxThreads = 256;
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 152, kOtherRegs = 104;
static_assert(kSoftmaxThreads * kSoftmaxRegs + (kThreads - kSoftmaxThreads) * kOtherRegs <=
                  kThreads * kLaunchRegs,
              "the shares of a block's registers");
constexpr int kStep = kStepTokens;
constexpr int kMinSteps = 4;
// In steps (see find_run).  A tile's queries, its first scores, its results and
// the wait for its other half take 8 us, three steps: 7 prompts of up to 1100
// tokens (416 tiles of 2 to 24 steps) 184 us with 0, 167 with 1, 145 with 2, 138
// with 3.
constexpr int kTileCost = 3;
constexpr int kScaleSlots = 4;

template <int DIM>
struct Smem {
  static constexpr int kTile = kStep * DIM * 2;  // bytes of 128 rows of fp16
  static constexpr int kQ = 0;                   // [2] queries
  static constexpr int kK = kQ + 2 * kTile;      // [2] keys
  static constexpr int kV = kK + 2 * kTile;      // [2] values
  static constexpr int kScales = kV + 2 * kTile; // [4][2][128] fp32: keys' x factor, values'
  static constexpr int kState = kScales + kScaleSlots * 2 * kStep * 4;  // [12][256] fp32
  static constexpr int kUnits = kState + 12 * 256 * 4;  // [256] fp32, and whether they are in use
  static constexpr int kBars = kUnits + 256 * 4 + 16;
  static constexpr int kNumBars = 8 + kScaleSlots + 1 + 8;
  static constexpr int kMisc = (kBars + 8 * kNumBars + 15) / 16 * 16;
  static constexpr int kMost = kMisc + 16, kLeast = kMisc + 80;  // [8] fp32 each, read as float4
  static_assert(kMost % 16 == 0 && kLeast % 16 == 0 && kScales % 16 == 0 && kState % 16 == 0 &&
                    kUnits % 16 == 0 && kBars % 16 == 0,
                "wide accesses to shared memory");
  static constexpr int kBytes = kMisc + 128 + 1024;  // slack to align to 1024
};

// Chunk j (16 bytes) of row r of a 128-byte-swizzled block of rows of 128 bytes.
__device__ __forceinline__ uint32_t swizzled(int r, int j) {
  return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4));
}

// Descriptor of an operand whose rows (tokens) are the K dimension and whose
// 64 elements of a row the other one: blocks of 64 elements `block` bytes
// apart, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_rows_k(uint32_t addr, uint32_t block) {
  uint64_t d = smem_desc_sw128(addr);
  d &= ~((uint64_t)0x3FFF << 16);
  d |= (uint64_t)(block >> 4) << 16;
  return d;
}

// 16 TMEM lanes x 32 columns: register 4 b + i of lane (g, c) is column 8 b + 2 c +
// i % 2 of TMEM lane g + 8 (i / 2).
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// 16 TMEM lanes x 16 columns of pairs of halves: register 2 b + i of lane (g, c) is
// column 4 b + c of TMEM lane g + 8 i.
__device__ __forceinline__ void tmem_ld_16x16h(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_16x16h(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}
// Wait for this thread's TMEM loads; the registers that they fill pass through
// it, so that nothing uses them before.
template <int N>
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[N]) {
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
}

template <typename V, V N>
struct Const {
  static constexpr V value = N;
};

constexpr int kFirstLevel = 5;
constexpr float kNoRef = -3.0e38f;  // the reference of a row that has seen nothing
constexpr float kGone = 1000.0f;    // binades after which nothing is left of a weight

// 16 bytes that this SM reads once: past the L1, which is small beside this much
// shared memory.
__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Walks the steps of a run: which tile, head and step of the tile.
struct Cursor {
  int seq_tile, head, off;
  RowTile t;
  __device__ __forceinline__ void start(const Kv4AttnParams& p, const Run& run) {
    seq_tile = run.seq_tile;
    head = run.head;
    off = run.off;
    t = row_tile(p, seq_tile);
  }
  // to the next tile of the row of steps (the caller knows that there is one)
  __device__ __forceinline__ void next_tile(const Kv4AttnParams& p) {
    off = 0;
    if (++head == p.cache.heads) {
      head = 0;
      t = next_row_tile(p, &seq_tile);
    }
  }
};

// The steps of a tile that the rows of half X see: [from, to) within the tile.
struct HalfTile {
  int rows, from, to;
};
__device__ __forceinline__ HalfTile half_tile(const Kv4AttnParams& p, const RowTile& t, int x) {
  HalfTile h;
  h.rows = min(128, t.rows - 128 * x);
  h.from = h.to = 0;
  if (h.rows <= 0) {
    h.rows = 0;
    return h;
  }
  const int r0 = t.r0 + 128 * x;
  const int i0 = (int)p.by_group((uint32_t)r0), i1 = (int)p.by_group((uint32_t)(r0 + h.rows - 1));
  const int last = min(t.last, last_seen(p, t, i1));
  const int first = max(t.first, first_seen(p, last_seen(p, t, i0)));
  if (last > first) {
    h.from = (first - t.base) / kStep;
    h.to = (last - t.base + kStep - 1) / kStep;
  }
  return h;
}

// What shared memory has of a softmax thread's four rows beside its registers, in
// arrays 256 floats apart: [2] ref and [2] l of the two rows at hand; of all four [4]
// the tokens of the step that the row sees (from the low half to the high half) and
// [4] the exponents of the powers of two that its products take besides (kSpan);
// then [256] the tile's rows' own units of the scores, and whether these are in use.
__device__ __forceinline__ uint32_t row_sees(const float* state, int row) {
  return reinterpret_cast<const uint32_t*>(state + 4 * 256)[row * 256];
}

// Where a reference has moved: the sums (at `to`, when they hold anything: S of this
// step was committed after O += P V of the step before) and this step's weights so
// far, `q` chunks, times f.
template <int DIM>
__device__ __forceinline__ void follow_reference(uint32_t ts, uint32_t to, int q, bool sums,
                                                 const float (&f)[2]) {
  tmem_st_wait();
  if (sums) {
#pragma unroll 1
    for (int n = 0; n < DIM / 32; ++n) {
      uint32_t v[16];
      tmem_ld_16x32(to + 32 * n, v);
      tmem_ld_wait_for(v);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f[k / 2 % 2]);
      tmem_st_16x32(to + 32 * n, v);
    }
  }
#pragma unroll 1
  for (int n = 0; n < q; ++n) {
    uint32_t v[8];
    tmem_ld_16x16h(ts + 16 * n, v);
    tmem_ld_wait_for(v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // (in fp32: a factor may be below fp16's range)
      const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&v[k]));
      v[k] = pack_f16(w.x * f[k % 2], w.y * f[k % 2]);
    }
    tmem_st_16x16h(ts + 16 * n, v);
  }
}

// The careful form of the weights of 32 tokens (chunk q of the step) and two of a
// thread's rows, 2 h and 2 h + 1, 16 TMEM lanes, whose S begins at `ts`
// (warp-uniform call); ks: the chunk's scales of this thread's first columns.  True,
// with nothing done, where one of the warp's rows is too far from the ordinary for it
// (far_weights).  Both are functions of their own, so that their registers are not
// the loop's, and apart from one another, as every tile begins with this one.
template <int DIM>
__device__ __noinline__ bool careful_weights(uint32_t ts, uint32_t to, const float* ks, int q,
                                             bool sums, float* state, int h) {
  const int c4 = threadIdx.x % 4;
  float s8[2][8], ref[2], f[2];
  bool moved = false, far = state[13 * 256 - threadIdx.x] != 0.0f;
  uint32_t sv[16], pw[8];
  tmem_ld_16x32(ts + 32 * q, sv);
  tmem_ld_wait_for(sv);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t seen = row_sees(state, 2 * h + i);
    const int upto = (int)(seen >> 16) - 32 * q - 2 * c4, from = (int)(seen & 0xffffu) - 32 * q - 2 * c4;
    const float rf = state[i * 256];
    float high = -INFINITY, top = -INFINITY;  // of t; of log2 |2^t vs|
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int token = n / 2 * 8 + n % 2;
      const bool see = token < upto && token >= from;
      s8[i][n] = see ? __uint_as_float(sv[n / 2 * 4 + i * 2 + n % 2]) * ks[token] : -INFINITY;
      high = fmaxf(high, s8[i][n]);
      const float v = fabsf(ks[kStep + token]);
      if (see && v < INFINITY) top = fmaxf(top, s8[i][n] + __log2f(v));
    }
#pragma unroll
    for (int d = 1; d < 4; d *= 2) {  // (the four lanes of a row agree)
      high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, d));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    }
    ref[i] = rf;
    if (high > -INFINITY) {
      // products past the span of the weights (below it, weights just grow), scores
      // or a reference too large to be a few binades apart, weights out of range
      const float over = top - high;
      far |= !(over <= (float)kSpan && over >= -75.0f) || fabsf(high) >= kFarScore;
      if (rf == kNoRef) {
        ref[i] = top - kFirstLevel;
      } else {
        far |= fabsf(rf) >= kFarScore || high - rf > 99.0f;
        if (top - rf > 14.9f) ref[i] = rf + ceilf(top - kLevel - rf);  // (binades: an exact factor)
      }
    }
    far |= state[(8 + 2 * h + i) * 256] != 0.0f;
    f[i] = rf == kNoRef ? 0.0f : ex2(rf - ref[i]);
    moved |= rf != kNoRef && ref[i] != rf;
  }
  if (__any_sync(0xffffffffu, far)) return true;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float total = 0.0f;
#pragma unroll
    for (int n = 0; n < 8; n += 2) {
      float w2[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float pj = ex2(s8[i][n + e] - ref[i]);
        const bool see = s8[i][n + e] != -INFINITY;
        total += see ? pj : 0.0f;
        // what a row does not see has weight 0 whatever its scale
        w2[e] = see ? pj * ks[kStep + n / 2 * 8 + e] : 0.0f;
      }
      pw[n + i] = pack_f16(w2[0], w2[1]);
    }
    state[i * 256] = ref[i];
    state[(2 + i) * 256] = state[(2 + i) * 256] * f[i] + total;
  }
  tmem_st_16x16h(ts + 16 * q, pw);
  if (__any_sync(0xffffffffu, moved)) follow_reference<DIM>(ts, to, q, sums, f);
  return false;
}

// The same for rows of every kind: the largest product goes to its level by the
// reference as far as kSpan allows it beside the largest weight, past that by a
// power of two of the row; scores are in units of the rows' own.  True where a row's
// next step needs this form again.
template <int DIM>
__device__ __noinline__ bool far_weights(uint32_t ts, uint32_t to, const float* ks, int q,
                                         bool sums, float* state, int h) {
  const int c4 = threadIdx.x % 4;
  float* shifts = state + (8 + 2 * h) * 256;
  const float* units = state + 12 * 256 - threadIdx.x % 32 + threadIdx.x % 32 / 4 + 16 * h;
  float f[2];
  bool moved = false, wide = state[13 * 256 - threadIdx.x] != 0.0f;
  uint32_t sv[16], pw[8];
  tmem_ld_16x32(ts + 32 * q, sv);
  tmem_ld_wait_for(sv);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t seen = row_sees(state, 2 * h + i);
    const int upto = (int)(seen >> 16) - 32 * q - 2 * c4, from = (int)(seen & 0xffffu) - 32 * q - 2 * c4;
    const float rf = state[i * 256], shift = shifts[i * 256], unit = units[i * 8];
    float sum = state[(2 + i) * 256];            // this lane's columns only
    float high = -INFINITY, over = -INFINITY;  // of t; of log2 |2^(t - high) vs|
    float s8[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int token = n / 2 * 8 + n % 2;
      const bool see = token < upto && token >= from;
      s8[n] = see ? __uint_as_float(sv[n / 2 * 4 + i * 2 + n % 2]) * ks[token] * unit : -INFINITY;
      high = fmaxf(high, s8[n]);
    }
#pragma unroll
    for (int d = 1; d < 4; d *= 2) {
      high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, d));
      sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float v = fabsf(ks[kStep + n / 2 * 8 + n % 2]);
      if (v < INFINITY && s8[n] > -INFINITY) over = fmaxf(over, s8[n] - high + __log2f(v));
    }
#pragma unroll
    for (int d = 1; d < 4; d *= 2) over = fmaxf(over, __shfl_xor_sync(0xffffffffu, over, d));
    float ref = rf, next_shift = shift;
    if (rf == kNoRef || high - rf + over + shift > 14.9f) {
      // (the largest weight of what is there is at most its sum)
      const float most = rf == kNoRef ? high : fmaxf(high, rf + __log2f(sum));
      const float level = rf == kNoRef ? (float)kFirstLevel : (float)kLevel;
      over += high - most;
      const float follow = over > -INFINITY ? fminf(fmaxf(over, -(float)kSpan), (float)kSpan) : 0.0f;
      const bool huge = fabsf(most) >= kFarScore;
      const float need = huge ? most : most + follow - level;
      // (by binades, so that what is there scales exactly; not where that is gone)
      if (high > -INFINITY)
        ref = huge || rf == kNoRef || need - rf > kGone ? need : rf + ceilf(need - rf);
      next_shift = over > -INFINITY
                       ? fminf(fmaxf(rintf(huge ? level - over : follow - over), -126.0f), 100.0f)
                       : 0.0f;
    } else if (high - rf > 99.0f) {
      // weights out of range, products not: these stay where they are
      ref = fabsf(high) >= kFarScore ? high
            : high - rf > kGone      ? high - kSpan
                                     : rf + ceilf(high - kSpan - rf);
      next_shift = fminf(shift + rintf(ref - rf), 100.0f);
    }
    const float fl = rf == kNoRef ? 0.0f : ex2(rf - ref);
    f[i] = rf == kNoRef ? 0.0f : ex2(rf - ref + (next_shift - shift));
    moved |= rf != kNoRef && (ref != rf || next_shift != shift);
    wide |= next_shift != 0.0f;
    const float power = ex2(next_shift);
    float total = 0.0f;
#pragma unroll
    for (int n = 0; n < 8; n += 2) {
      float w2[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float pj = ex2(s8[n + e] - ref);
        const bool see = s8[n + e] != -INFINITY;
        total += see ? pj : 0.0f;
        w2[e] = see ? pj * ks[kStep + n / 2 * 8 + e] * power : 0.0f;
      }
      pw[n + i] = pack_f16(w2[0], w2[1]);
    }
    state[i * 256] = ref;
    state[(2 + i) * 256] = state[(2 + i) * 256] * fl + total;
    shifts[i * 256] = next_shift;
  }
  tmem_st_16x16h(ts + 16 * q, pw);
  if (__any_sync(0xffffffffu, moved)) follow_reference<DIM>(ts, to, q, sums, f);
  return wide;
}

template <typename T, int DIM>
__global__ void __launch_bounds__(kThreads, 1)
    kv4_tiles_kernel(const __grid_constant__ Kv4AttnParams p) {
  using S = Smem<DIM>;
  constexpr int kBlock = kStep * 128;
  constexpr uint32_t kIdescS = instr_desc(128, kStep);
  constexpr uint32_t kIdescO = instr_desc(128, DIM) | (1u << 16);  // B's rows are the K dimension
  constexpr uint32_t kColO = 256;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem), bar0 = sbase + S::kBars;
  auto k_full = [&](int i) { return bar0 + 8u * i; };
  auto k_empty = [&](int i) { return bar0 + 8u * (2 + i); };
  auto v_full = [&](int i) { return bar0 + 8u * (4 + i); };
  auto v_empty = [&](int i) { return bar0 + 8u * (6 + i); };
  auto scale_full = [&](int i) { return bar0 + 8u * (8 + i); };
  const uint32_t q_full = bar0 + 8u * (8 + kScaleSlots);
  auto s_full = [&](int x) { return q_full + 8u + 8u * x; };
  auto p_full = [&](int x) { return q_full + 24u + 8u * x; };
  auto o_full = [&](int x) { return q_full + 40u + 8u * x; };
  const uint32_t drain = q_full + 56u, taken = q_full + 64u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);
  float* factor_slot = reinterpret_cast<float*>(smem + S::kMisc + 8);
  float* most_slots = reinterpret_cast<float*>(smem + S::kMost);
  float* least_slots = reinterpret_cast<float*>(smem + S::kLeast);
  float* units = reinterpret_cast<float*>(smem + S::kUnits);
  float* scales = reinterpret_cast<float*>(smem + S::kScales);
  // the present tile, for the MMAs and converters: steps, and those each half sees
  volatile int* piece = reinterpret_cast<volatile int*>(smem + S::kMisc + 48);  // count, from, to, from, to

  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full(i), 128);
      mbar_init(k_empty(i), 1);
      mbar_init(v_full(i), 96);
      mbar_init(v_empty(i), 1);
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 128);
      mbar_init(o_full(i), 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) mbar_init(scale_full(i), 128 + 96);
    mbar_init(q_full, 256);
    mbar_init(taken, 128 + 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  const Run run = find_run<kThreads>(p, kMinSteps, kTileCost);  // (with a barrier of the block)
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (p.joins > 0 && !p.by_tile && threadIdx.x == 0) p.join[blockIdx.x].last_cta = -1;

  bool dead = false;
  auto wait = [&](uint32_t bar, uint32_t phase) {
    if (!dead) dead = !mbar_wait(bar, phase & 1u, abort_flag, p.status);
  };
  // the same for all lanes of a warp, which go on together
  auto warp_wait = [&](uint32_t bar, uint32_t phase) {
    wait(bar, phase);
    dead = __any_sync(0xffffffffu, dead);
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 12) {
      // ---------------- the MMAs ----------------
      // The whole warp walks, lane 0 issues: what it passes stays warp-uniform and
      // the descriptors of a step are sums of few registers and constants.
      if (run.count > 0) {
        const uint64_t q_desc = smem_desc_sw128(sbase + S::kQ), k_desc = smem_desc_sw128(sbase + S::kK);
        const uint64_t v_desc = smem_desc_rows_k(sbase + S::kV, kBlock);
        uint32_t step = 0, tile = 0;     // of the run: steps so far, tiles so far
        uint32_t n_p0 = 0, n_p1 = 0;     // weights of each half consumed so far
        // O_X += P_X V of run step sv (`with_o`), S_X = Q_X K^T of run step sj (`with_s`)
        auto issue = [&](int X, uint32_t sv, bool with_o, bool first, bool last, uint32_t sj,
                         bool with_s) {
          if (with_o) warp_wait(p_full(X), X ? n_p1++ : n_p0++);
          if (dead) return;
          tc_fence_after();
          if (lane == 0) {
            if (with_o) {
              const uint64_t v = v_desc + (sv & 1) * (S::kTile >> 4);
#pragma unroll
              for (int k = 0; k < kStep / 16; ++k)
                mma_f16_ts(tmem + kColO + 128 * X, tmem + 128 * X + 8 * k, v + k * (2048 >> 4),
                           kIdescO, k > 0 ? 1u : first ? 0u : 1u);
              if (last) mma_commit(o_full(X));
            }
            if (with_s) {
              const uint64_t q0 = q_desc + X * (S::kTile >> 4), k0 = k_desc + (sj & 1) * (S::kTile >> 4);
#pragma unroll
              for (int k = 0; k < DIM / 16; ++k) {
                const uint64_t at = ((k / 4) * kBlock + (k % 4) * 32) >> 4;
                mma_f16(tmem + 128 * X, q0 + at, k0 + at, kIdescS, k > 0 ? 1u : 0u);
              }
              mma_commit(s_full(X));
            }
            // (half 1 goes last: both halves have then used the step's values, keys)
            if (X == 1 && sv != ~0u) mma_commit(v_empty(sv & 1));
            if (X == 1 && sj != ~0u) mma_commit(k_empty(sj & 1));
          }
          __syncwarp();
        };
        for (int done = 0; done < run.count; ++tile) {
          warp_wait(q_full, tile);
          const int count = dead ? 1 : piece[0];
          const int from0 = piece[1], to0 = piece[2], from1 = piece[3], to1 = piece[4];
          __syncwarp();
          if (lane == 0) mbar_arrive(taken);
          for (int j = 0; j <= count; ++j) {
            // run steps of the values and the keys (~0: none)
            const uint32_t sv = j > 0 ? step + j - 1 : ~0u, sj = j < count ? step + j : ~0u;
            if (j > 0) warp_wait(v_full(sv & 1), sv >> 1);
            if (j < count) warp_wait(k_full(sj & 1), sj >> 1);
#pragma unroll 1
            for (int X = 0; X < 2; ++X) {
              const int from = X ? from1 : from0, to = X ? to1 : to0;
              issue(X, sv, j > from && j <= to, j - 1 == from, j == to, sj, j >= from && j < to);
            }
          }
          step += count;
          done += count;
        }
        // every MMA and commit has ended before the block does (with a limit, also
        // after a wait that ran out)
        volatile int go_on = 0;
        if (lane == 0) {
          mma_commit(drain);
          mbar_wait(drain, 0, &go_on, p.status);
        }
        __syncwarp();
      }
    } else {
      // ---------------- converters ----------------
      // Warps 8..11 keys, 13..15 values; the next step's codes are on their way to
      // registers while the MMAs use this one's.
      // Groups of TPL tokens go to the warps in turn; a lane takes 32 codes (16
      // bytes) of a token, the lanes of a phase of 8 different tokens of 8 (no
      // bank conflicts).
      {
        const bool values = warp > 12;
        const int warps = values ? 3 : 4;
        constexpr int LPT = DIM / 32, TPL = 32 / LPT, GROUPS = kStep / TPL;
        constexpr int LOADS = (GROUPS + 2) / 3, SCALES = 2;
        const int cw = warp - (values ? 13 : 8), ctid = cw * 32 + lane, chunk = lane / TPL;
        const int page_size = (int)p.cache.page_size;
        const uint32_t page16 = (uint32_t)page_size / 16;
        const uint8_t* codes_at = p.cache.base + (values ? (int64_t)page_size * (DIM / 2) : 0) +
                                  chunk * 16 + lane % TPL % 16 * (DIM / 2);
        const uint8_t* scales_at = p.cache.base + (int64_t)page_size * (DIM + (values ? 2 : 0));
        // where the loads stand: `ahead` steps into the run; lane l < 8 has the
        // offsets of the codes and scales of the step's tokens 16 l and on (-1: none)
        Cursor c = {};
        int ahead = 0;
        int64_t codes_off, scales_off;
        auto find = [&]() {
          codes_off = scales_off = -1;
          const int token = c.t.base + c.off * kStep + lane * 16;
          // (no row sees any of it: past the last token, or before a window, where the
          // sequence may have given its pages back)
          if (ahead >= run.count || lane >= 8 || token >= c.t.last || token + 16 <= c.t.first) return;
          const uint32_t group = (uint32_t)token / 16, in_table = p.by_page16(group);
          const int page = __ldg(p.page_table + (int64_t)c.t.b * p.table_width + in_table);
          if ((uint32_t)page >= (uint32_t)p.cache.pages) {
            atomicOr(p.status, kStatusBadIndex);
            return;
          }
          const int64_t block =
              ((int64_t)page * p.cache.heads + c.head) * kv4_block_bytes(DIM, page_size);
          const uint32_t inside = (group - in_table * page16) * 16;
          codes_off = block + inside * (DIM / 2);
          scales_off = block + inside * 2;
        };
        uint4 raw[LOADS];
        uint32_t raw_s[SCALES];
        // loads the codes of the step found, and finds the next one
        auto load = [&]() {
#pragma unroll
          for (int i = 0; i < LOADS; ++i) {
            const int first = (cw + warps * i) * TPL;  // token of the step
            const int64_t off = __shfl_sync(0xffffffffu, codes_off, first / 16 % 8);
            raw[i] = make_uint4(0, 0, 0, 0);
            if (first < kStep && off >= 0)
              raw[i] = load_once(codes_at + off + first % 16 * (DIM / 2));
          }
#pragma unroll
          for (int i = 0; i < SCALES; ++i) {
            const int token = ctid + 32 * warps * i;
            const int64_t off = __shfl_sync(0xffffffffu, scales_off, token / 16 % 8);
            raw_s[i] = 0;
            if (token < kStep && off >= 0)
              raw_s[i] = __ldg(reinterpret_cast<const uint16_t*>(scales_at + off) + token % 16);
          }
          if (++ahead < run.count && ++c.off == c.t.steps) c.next_tile(p);
          find();
        };
        if (run.count > 0) {
          c.start(p, run);
          find();
          load();
        }
        uint32_t tile = 0;
        int left = 0;  // (keys) steps of the present tile still to convert
        float factor = 1.0f;
        for (int s = 0; s < run.count; ++s) {
          if (!values && left-- == 0) {
            wait(q_full, tile++);
            left = dead ? run.count : piece[0] - 1;
            factor = *reinterpret_cast<volatile float*>(factor_slot);
            mbar_arrive(taken);
          }
          const int st = s & 1, use = s >> 1;
#pragma unroll
          for (int i = 0; i < SCALES; ++i) {
            const int token = ctid + 32 * warps * i;
            if (token < kStep)
              scales[((s % kScaleSlots) * 2 + (values ? 1 : 0)) * kStep + token] =
                  __uint_as_float(raw_s[i] << 16) * factor;
          }
          mbar_arrive(scale_full(s % kScaleSlots));
          if (use > 0) wait(values ? v_empty(st) : k_empty(st), use - 1);
          const uint32_t dst = sbase + (values ? S::kV : S::kK) + st * S::kTile;
#pragma unroll
          for (int i = 0; i < LOADS; ++i) {
            const int r = (cw + warps * i) * TPL + lane % TPL;
            if (r >= kStep) continue;
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t w8 = w[k] >> 8;
              const int at = chunk * 4 + k;
              st_shared_v4(dst + (at / 8) * kBlock + swizzled(r, at % 8), (int)codes_f16<false>(w[k]),
                           (int)codes_f16<true>(w[k]), (int)codes_f16<false>(w8), (int)codes_f16<true>(w8));
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(values ? v_full(st) : k_full(st));
          __syncwarp();
          load();
        }
      }
    }
  } else {
    // ---------------- softmax ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int x = warp / 4, r = threadIdx.x;  // half; row of the 256 (queries and results)
    const int g = lane / 4, c4 = lane % 4;    // scores: rows g + 8 i of the warp's 32, i < 4
    const uint32_t lane_base = (uint32_t)(32 * (warp % 4)) << 16;
    const uint32_t ts = tmem + lane_base + 128 * x, to_ = tmem + lane_base + kColO + 128 * x;
    // What a tile is, is looked up again where it is needed (hidden from the
    // compiler, which would keep it in registers throughout and spill others).
    auto hide = [](int v) {
      asm volatile("" : "+r"(v));
      return v;
    };
    int seq_tile = run.seq_tile, head = run.head, off = run.off;
    uint32_t step = 0, n_s = 0, n_o = 0;
    for (int done = 0, tile = 0; done < run.count; ++tile) {
      int count, from, upto, all_from, all_to, token_base;
      {
      const RowTile t = row_tile(p, hide(seq_tile));
      count = min(t.steps - off, run.count - done);
      const HalfTile h = half_tile(p, t, x);
      const bool live = r < t.rows;
      const int qi = (int)p.by_group((uint32_t)(t.r0 + min(r, t.rows - 1)));
      // ---- queries to shared memory: fp16 times the tile's power of two (its
      // largest element goes to 2^14 .. 2^15), in the codes' order; where a row would
      // be too small by it, every row its own, and scores are brought to their unit in
      // the careful form of a step (as in kv4_rows.cu).  (Every MMA of the tile before
      // has ended.)  The MMAs' warp and the keys' converters have
      // taken over the tile before: of one that sees nothing this half waited for
      // nothing, and several in a row would run away from those that walk them.
      {
        if (tile > 0) warp_wait(taken, tile - 1);
        const T* src = static_cast<const T*>(p.q) + (int64_t)(t.q0 + qi) * p.q_stride +
                       (int64_t)(head * p.group + t.r0 + min(r, t.rows - 1) - qi * p.group) * DIM;
        // (kept for the second use as far as registers go: the L1 beside this much
        // shared memory keeps little)
        constexpr int KEEP = 8;
        Raw8<T> raw[KEEP];
#pragma unroll
        for (int i = 0; i < KEEP; ++i) raw[i] = load8_raw(src + 8 * i);
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < DIM / 8; ++i) {
          float v[8];
          unpack8(i < KEEP ? raw[i % KEEP] : load8_raw(src + 8 * i), v);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (fabsf(v[k]) < INFINITY) most = fmaxf(most, fabsf(v[k]));
        }
        const float row_most = most;
        float least = most > 0.0f ? most : INFINITY;  // of rows that are not 0
        most = warp_most(most);
        least = warp_least(least);
        asm volatile("bar.sync 1, 256;" ::: "memory");  // (the slots' last readers are done)
        if (lane == 0) {
          most_slots[warp] = most;
          least_slots[warp] = least;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 a = *reinterpret_cast<const float4*>(most_slots + i);
          const float4 b = *reinterpret_cast<const float4*>(least_slots + i);
          most = fmaxf(most, fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)));
          least = fminf(least, fminf(fminf(b.x, b.y), fminf(b.z, b.w)));
        }
        const bool wide = far_queries(most, least);
        const int k_tile = wide ? far_tile_power(most) : query_power(most);
        const int k_row = wide ? far_row_power(row_most, k_tile) : k_tile;
        const float up = power_of_two(k_row);
        units[r] = power_of_two(k_tile - k_row);
        if (r == 0) {
          const HalfTile h1 = half_tile(p, t, 1);  // (this thread's is half 0)
          piece[0] = count;
          piece[1] = min(max(h.from - off, 0), count);
          piece[2] = min(max(h.to - off, piece[1]), count);
          piece[3] = min(max(h1.from - off, 0), count);
          piece[4] = min(max(h1.to - off, piece[3]), count);
          units[256] = wide ? 1.0f : 0.0f;
          *factor_slot = power_of_two(-k_tile) * (p.scale * kLog2e / kCodeUnit);
        }
        const uint32_t dst = sbase + S::kQ + x * S::kTile;
#pragma unroll
        for (int i = 0; i < DIM / 8; ++i) {
          float v[8];
          unpack8(i < KEEP ? raw[i % KEEP] : load8_raw(src + 8 * i), v);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = live ? v[k] * up : 0.0f;
          st_shared_v4(dst + (i / 8) * kBlock + swizzled(r % 128, i % 8), (int)pack_f16(v[0], v[4]),
                       (int)pack_f16(v[1], v[5]), (int)pack_f16(v[2], v[6]),
                       (int)pack_f16(v[3], v[7]));
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
      }
      // ---- the steps that this half sees, and the tokens that all its rows see
      from = min(max(h.from - off, 0), count);
      upto = min(max(h.to - off, from), count);
      token_base = t.base + off * kStep;
      const int hr0 = t.r0 + 128 * x;
      all_to = min(t.last, last_seen(p, t, (int)p.by_group((uint32_t)hr0)));
      all_from = max(t.first, first_seen(p, last_seen(p, t, (int)p.by_group(
                                                (uint32_t)(hr0 + max(h.rows, 1) - 1)))));
      }
      // Per row: weights 2^(t - ref), l their sum.  A weight times a value scale goes
      // into the value product in fp16; `ref` puts the largest of the first 32 of
      // those at 2^5, and moves (up, by whole binades, so that what is there scales
      // exactly) when one exceeds 2^15, or a weight 2^100, which then goes to 2^11:
      // fp16 rounds them by 2^-11 of themselves or 2^-30 (2^-36 once it has moved) of the
      // largest, whichever is more.  (2^11 from the start: rows then moved after every
      // other chunk of the first steps, 1250 us instead of 1099 for 4096 queries over
      // 16384 tokens.)  Until a row has seen a token its reference is kNoRef: its first
      // weight overflows and so sets it.
      float ref[4], l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ref[i] = kNoRef;
        l[i] = 0.0f;
      }
      float* state = reinterpret_cast<float*>(smem + S::kState) + threadIdx.x;
      uint32_t* seen = reinterpret_cast<uint32_t*>(state + 4 * 256);
      float* shifts = state + 8 * 256;
#pragma unroll
      for (int i = 0; i < 4; ++i) shifts[i * 256] = 0.0f;
      bool was_masked = true;  // (and `seen` to be set)
      // The steps before `from` were not waited for: with the first scores there,
      // every earlier step has its scales, so the barrier of a slot of scales is in
      // this step's phase or past it, and its parity says which.
      if (from < upto) warp_wait(s_full(x), n_s);
      // every step takes the careful form: rows have units of their own, or products
      // of a row a power of two besides
      bool wide = state[13 * 256 - threadIdx.x] != 0.0f;
      for (int j = from; j < upto; ++j) {
        const uint32_t slot = (step + j) % kScaleSlots;
        warp_wait(scale_full(slot), (step + j) / kScaleSlots);
        warp_wait(s_full(x), n_s++);
        if (dead) break;
        tc_fence_after();
        const int token0 = token_base + j * kStep;
        const bool masked = token0 < all_from || token0 + kStep > all_to;
        // tokens of the step that row i sees
        if (masked) {
          const RowTile t = row_tile(p, hide(seq_tile));
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const int row = min(32 * warp + g + 8 * i, t.rows - 1);
            const int sees = last_seen(p, t, (int)p.by_group((uint32_t)(t.r0 + row)));
            const int lo = max(t.first, first_seen(p, sees)) - token0;
            const int hi = min(t.last, sees) - token0;
            seen[i * 256] =
                (uint32_t)min(max(lo, 0), kStep) | (uint32_t)min(max(hi, 0), kStep) << 16;
          }
          was_masked = true;
        } else if (was_masked) {
          was_masked = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) seen[i * 256] = (uint32_t)kStep << 16;
        }
        // 32 tokens and the thread's four rows (rows 2 h, 2 h + 1 in sv[h]) at a time; P
        // overwrites S that is done with.  (Not unrolled further: the loops of all
        // roles have to stay in the SM's instruction cache; unrolled, a kernel of
        // 1.85 ms waited for instructions half its time.  The next lot's scores
        // loaded ahead gained nothing: the other half's warps fill that time.)
        auto weights = [&](auto masked_, int q, const float* ks) {
          constexpr bool MASKED = decltype(masked_)::value;
          uint32_t sv[2][16], pw[2][8];
          tmem_ld_16x32(ts + 32 * q, sv[0]);
          tmem_ld_16x32(ts + (16u << 16) + 32 * q, sv[1]);
          tmem_ld_wait_for(sv[0]);
          tmem_ld_wait_for(sv[1]);
          uint64_t sum[4] = {0, 0, 0, 0};
          __half2 most = __half2half2(__half(0.0f));
          bool again = wide;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const uint64_t k2 = *reinterpret_cast<const uint64_t*>(ks + 8 * b);
            const uint64_t v2 = *reinterpret_cast<const uint64_t*>(ks + kStep + 8 * b);
            if (MASKED) {  // a scale that is not a number may stand in a masked place
              float a, c;
              unpair(v2, a, c);
              again |= !(fabsf(a) < INFINITY) || !(fabsf(c) < INFINITY);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float x0, x1;
              unpair(fma2(pair(__uint_as_float(sv[i / 2][4 * b + i % 2 * 2]),
                               __uint_as_float(sv[i / 2][4 * b + i % 2 * 2 + 1])),
                          k2, pair(-ref[i], -ref[i])),
                     x0, x1);
              if (MASKED) {
                const uint32_t see = seen[i * 256], lo = see & 0xffffu, hi = see >> 16;
                const uint32_t n = 32 * q + 8 * b + 2 * c4;
                if (n < lo || n >= hi) x0 = -INFINITY;
                if (n + 1 < lo || n + 1 >= hi) x1 = -INFINITY;
              }
              const uint64_t p2 = pair(ex2(x0), ex2(x1));
              sum[i] = add2(sum[i], p2);
              unpair(mul2(p2, v2), x0, x1);
              const uint32_t h = pack_f16(x0, x1);
              most = __hmax2_nan(most, __habs2(*reinterpret_cast<const __half2*>(&h)));
              pw[i / 2][2 * b + i % 2] = h;
            }
          }
          again |= !__hble2(most, __half2half2(__half(32768.0f)));  // (or no number)
          float part[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float a, b;
            unpair(sum[i], a, b);
            part[i] = a + b;
          }
          again |= fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])) > kFar;
          if (__any_sync(0xffffffffu, again)) {
            // weights out of range, or odd scales beside a mask: once more, with care
            const bool odd = __any_sync(0xffffffffu, wide);
            wide = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                state[i * 256] = ref[2 * h + i];
                state[(2 + i) * 256] = l[2 * h + i];
              }
              const uint32_t lanes = h ? 16u << 16 : 0u;
              if (odd || careful_weights<DIM>(ts + lanes, to_ + lanes, ks, q, j > from, state, h))
                wide |= far_weights<DIM>(ts + lanes, to_ + lanes, ks, q, j > from, state, h);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                ref[2 * h + i] = state[i * 256];
                l[2 * h + i] = state[(2 + i) * 256];
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) l[i] += part[i];
            tmem_st_16x16h(ts + 16 * q, pw[0]);
            tmem_st_16x16h(ts + (16u << 16) + 16 * q, pw[1]);
          }
        };
        auto chunks = [&](auto masked_) {
          const float* ks = scales + slot * 2 * kStep + 2 * c4;
#pragma unroll 1
          for (int q = 0; q < 4; ++q, ks += 32) weights(masked_, q, ks);
        };
        if (masked) chunks(Const<bool, true>{});
        else chunks(Const<bool, false>{});
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full(x));
      }
      // ---- the rows' results
      // (a thread a row again: row `lane` of the warp's 32 is row i = lane / 8 of
      // the lanes 4 (lane % 8) ..)
      const RowTile t = row_tile(p, hide(seq_tile));
      const bool whole = count == t.steps, live = r < t.rows;
      float l_row = 0.0f, ref_row = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        const float a = __shfl_sync(0xffffffffu, l[i], 4 * (lane % 8));
        const float b = __shfl_sync(0xffffffffu, ref[i], 4 * (lane % 8));
        if (lane / 8 == i) {
          l_row = a;
          ref_row = b;
        }
      }
      __syncwarp();
      const float unit = ex2(-(reinterpret_cast<const float*>(smem + S::kState) + 8 * 256)
                                  [lane / 8 * 256 + threadIdx.x - lane + 4 * (lane % 8)]);
      const bool none = l_row == 0.0f;
      const float inv = none ? 0.0f : (1.0f / kCodeUnit) / l_row;
      const float lse = none ? -INFINITY : ref_row + log2f(l_row);
      if (upto > from) {
        warp_wait(o_full(x), n_o++);
        tc_fence_after();
      }
      if (p.joins > 0 && off == 0 && (!whole || p.by_tile) && threadIdx.x == 0) {
        const int64_t last = (run.pos + done + tile * kTileCost + t.steps - 1) / run.per;  // the CTA of its last step
        p.join[p.by_tile ? seq_tile * p.cache.heads + head : (int)blockIdx.x] =
            Kv4Join{seq_tile, head, (int)blockIdx.x, whole ? -1 : (int)last};
      }
      const int64_t share = ((int64_t)blockIdx.x * 2 + (off == 0)) * p.tile_rows + r;
      const int64_t at = out_row(p, t, head, t.r0 + min(r, t.rows - 1));
      if (t.rows > 128 * x && !dead) {
#pragma unroll 1
        for (int q = 0; q < DIM / 32; ++q) {
          uint32_t v[32];
          if (upto > from) {
            tmem_ld32(to_ + 32 * q, v);
            tmem_ld_wait_for(v);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // columns 8 i .. of the accumulator are channels 0, 4, 1, 5, 2, 6, 3, 7 of
            // eight, in units of kCodeUnit
            float ch[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int d = k / 2 + (k & 1) * 4;
              ch[d] = none ? 0.0f
                           : __uint_as_float(v[8 * i + k]) * inv * unit;
            }
            if (!live) continue;
            if (whole) store8(static_cast<T*>(p.o) + at * DIM + 32 * q + 8 * i, ch);
            else store8(p.share_o + share * DIM + 32 * q + 8 * i, ch);
          }
        }
        if (live) {
          if (whole) {
            if (p.lse) p.lse[at] = lse * kLn2;
          } else {
            p.share_lse[share] = lse;
          }
        }
      }
      step += count;
      done += count;
      off = 0;
      if (done < run.count && ++head == p.cache.heads) {
        head = 0;
        next_row_tile(p, &seq_tile);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int DIM>
cudaError_t launch_tile(const Kv4AttnParams& p, cudaStream_t s) {
  auto kernel = kv4_tiles_kernel<T, DIM>;
  static std::atomic<uint64_t> set{0};  // devices on which the kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(set.load() >> dev & 1)) {
    cudaFuncAttributes has = {};
    e = cudaFuncGetAttributes(&has, kernel);
    if (e != cudaSuccess) return e;
    if (has.numRegs < kLaunchRegs) return cudaErrorLaunchOutOfResources;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<DIM>::kBytes);
    if (e != cudaSuccess) return e;
    set |= uint64_t(1) << dev;
  }
  kernel<<<p.ctas, kThreads, Smem<DIM>::kBytes, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_tiles(int dtype, const Kv4AttnParams& p, cudaStream_t s) {
  if (dtype == LBGEMM_BF16)
    return p.cache.dim == 64 ? launch_tile<__nv_bfloat16, 64>(p, s)
                             : launch_tile<__nv_bfloat16, 128>(p, s);
  return p.cache.dim == 64 ? launch_tile<__half, 64>(p, s) : launch_tile<__half, 128>(p, s);
}

}  // namespace lbg
