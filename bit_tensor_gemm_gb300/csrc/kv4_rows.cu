// kv4_rows.cu -- attention over the 4-bit cache for few query rows (a decoding
// step, drafted tokens): tiles of 8 or 16 rows (query tokens x heads of a
// group), streaming the cache once.
//
// The floor is HBM: D + 4 bytes per cached token and head against 4 D flops a
// row.  What an SM must keep up with at the copy rate is about 24 bytes a
// cycle, which is 47 codes to turn into floats, so the design keeps the
// instructions per code low:
//   - warp MMAs with the cached tokens (keys) or channels (values) as the 16
//     rows and the query rows as the 8 columns, so 8 rows cost no padding;
//   - two codes become two fp16 by a logical operation and a multiply-add (and a
//     shift for every second pair; kv4_codes.cuh);
//   - queries enter as fp16 times a power of two of their tile, in the order of
//     channels in which a lane's codes lie in memory (the order is free);
//   - the reference of the weights moves only when one leaves fp16's range, so
//     almost no step rescales its accumulators.
// A CTA streams 128 tokens a step through a ring of bulk copies; each of its
// four warps takes 32 of them, with a reference and sum of its own until the
// end.  The warps issue the copies in turn.  Three CTAs an SM with four stages
// (16 rows: two): with four CTAs of three stages, which left 128 registers and
// spilled, 131072 tokens took 44.4 us, 41.4 so.
// Measured: one row group over 131072 tokens of 8 heads (138 MB) 42.8 us, 3.2
// TB/s; 64 sequences of up to 8192 tokens (296 MB) 83 us, 3.6 TB/s.  In there,
// by clock: 7.4 us until the first tokens are worked on (finding the run, the
// pages, the queries: all first passes through their instructions), 1.5 us a
// step of an SM's three CTAs (5.1 TB/s; each instruction waits for the one
// before it too often for 12 warps to fill the SM: issue 37 %), 1.5 us for the
// warps' sums, 5 us for the join.
#include <cuda_runtime.h>

#include <atomic>

#include "kv4_attention.cuh"
#include "kv4_codes.cuh"
#include "ptx.cuh"

namespace lbg {
namespace {

// By what power of two a row's largest product is to be multiplied for its level,
// 2^(kLevel - 1) .. 2^kLevel, where `top` is that product over its largest weight.
__device__ __forceinline__ int to_level(float top) {
  return kLevel - 1 - ((int)(__float_as_uint(top) >> 23) - 127);
}
// What its products take besides its reference, which is `below` its largest score
// (of a row within the span to_level, but for scores that are too large to hold
// it): an even number, -126 .. 126.
__device__ __forceinline__ int top_shift(float below, float top) {
  return top > 0.0f ? min(max((to_level(top) - __float2int_rn(below)) & ~1, -126), 126) : 0;
}

constexpr int kWarps = 4, kStages = 4, kTokens = 32, kStep = kStepTokens;
constexpr int kMinSteps = 3;  // of a CTA's run
// in steps (see find_run).  64 sequences of up to 8192 tokens: 97.7 us with 0, 85.8
// with 1, 81.1 with 2, 81.6 with 3, 82.2 with 4 (and 24 drafts of 5 tokens
// 19.6, 17.1, 17.8, 18.2, 21.7).
constexpr int kTileCost = 2;
static_assert(kWarps * kTokens == kStep, "a warp's share of a step");
template <int DIM>
struct Ring {
  static constexpr int kCodes = kStep * DIM / 2;     // bytes of keys (or values) of a step
  static constexpr int kBytes = 2 * kCodes + 4 * kStep;
  static constexpr int kTotal = kStages * kBytes;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same into new accumulators: d = a b.
__device__ __forceinline__ void mma16816_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Four 8 x 8 matrices of halves, transposed: lane l gives the address of row
// l % 8 of matrix l / 8 and gets rows 2 (l % 4) and + 1 of column l / 4 of each.
__device__ __forceinline__ void load_transposed(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Element order inside a warp (lane = 4 g + c):
//   keys    MMA row g of a 16-token tile is token 2 g + e(g), row g + 8 the
//           other token of that pair, e(g) = parity of the low two bits of g:
//           so a lane's two tokens share one 32-bit word of scales, and the
//           key reads of a phase fall on different banks.  A lane holds the
//           channels c DIM/4 ... of its tokens; of a word, codes i and i + 4
//           make one register.
//   values  transposing loads give a lane half word g of the 16-byte chunk q of
//           the tokens of MMA rows 2c, 2c + 1 (then 2c + 8, 2c + 9) side by
//           side: four codes each.  MMA tile 2 q + j, row g is channel 32 q +
//           4 g + 2 j, row g + 8 the one after it.
template <typename T, int DIM, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 3 : 2)
    kv4_rows_kernel(const Kv4AttnParams p) {
  constexpr int KW = DIM / 32;   // 32-bit words of a key that a lane holds
  constexpr int MT = DIM / 16;   // MMA tiles of channels
  constexpr int R = 8 * NT;
  using Rg = Ring<DIM>;
  constexpr int ROW = DIM + 4;  // floats from a row to the next in the merge buffer
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2][kStages];  // full, empty
  __shared__ float merge_ref[kWarps][R], merge_l[kWarps][R], row_unit[kWarps][R];
  __shared__ int abort_flag;

  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, c = lane % 4;
  const uint32_t full = smem_addr(&bars[0][0]), empty = smem_addr(&bars[1][0]);
  if (threadIdx.x < kStages) {
    mbar_init(full + 8 * threadIdx.x, 1);
    mbar_init(empty + 8 * threadIdx.x, kWarps);
  }
  if (threadIdx.x == 0) abort_flag = 0;
  fence_barrier_init();
  // the kernel that joins shares may be scheduled once every CTA has begun
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Run run = find_run<kWarps * 32>(p, kMinSteps, kTileCost);  // (with a barrier of the block)
  if (p.joins > 0 && !p.by_tile && threadIdx.x == 0) p.join[blockIdx.x].last_cta = -1;
  if (run.count == 0) return;

  // ---- copies.  Step s of the run: one copy per piece (keys, values, two
  // arrays of scales: lane % 4) and stretch of tokens that certainly lie in one
  // page (lane / 4).  Warp w issues steps w, w + 4, ...: the first ones at once, step
  // s + 3 when it begins step s, into the slot that step s - 1 leaves.
  static_assert(kWarps == kStages, "every warp issues one of the first steps");
  const uint32_t ring = smem_addr(smem);
  const int page_size = (int)p.cache.page_size;
  const int stretch =
      page_size % 128 == 0 ? 128 : page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : 16;
  const int piece = lane & 3, stretch_at = (lane >> 2) * stretch;  // its first token in a step
  const uint32_t page16 = (uint32_t)page_size / 16;
  const uint32_t row_bytes = piece < 2 ? DIM / 2 : 2;
  const uint32_t piece_dst = ring +
                             (piece < 2 ? piece * Rg::kCodes : 2 * Rg::kCodes + (piece - 2) * 2 * kStep) +
                             stretch_at * row_bytes;
  const int64_t block_bytes = kv4_block_bytes(DIM, page_size);
  const uint8_t* piece_src =
      p.cache.base + (int64_t)page_size * (piece < 2 ? piece * (DIM / 2) : DIM + (piece - 2) * 2);
  // where the next step that this warp issues stands, and its lane's source
  int is_tile = run.seq_tile, is_head = run.head, is_off = run.off, is_step = 0;
  RowTile is = row_tile(p, is_tile);
  const uint8_t* is_src = nullptr;
  auto advance = [&](int by) {  // to a step `by` further on, and its page
    is_step += by;
    is_src = nullptr;
    if (is_step >= run.count) return;
    is_off += by;
    while (is_off >= is.steps) {
      is_off -= is.steps;
      if (++is_head == p.cache.heads) {
        is_head = 0;
        is = next_row_tile(p, &is_tile);  // (there is one: the run goes on)
      }
    }
    const int token = is.base + is_off * kStep + stretch_at;
    // (none of it seen: past the last token, or before a window, where the sequence
    // may have given its pages back)
    if (stretch_at >= kStep || token >= is.last || token + stretch <= is.first) return;
    const uint32_t group = (uint32_t)token / 16, in_table = p.by_page16(group);
    const int page = __ldg(p.page_table + (int64_t)is.b * p.table_width + in_table);
    if ((uint32_t)page >= (uint32_t)p.cache.pages) {
      atomicOr(p.status, kStatusBadIndex);
      return;
    }
    is_src = piece_src + ((int64_t)page * p.cache.heads + is_head) * block_bytes +
             (group - in_table * page16) * 16 * row_bytes;
  };
  auto issue = [&]() {
    const uint32_t slot = (uint32_t)(is_step % kStages), bar = full + 8 * slot;
    const uint32_t lanes = __popc(__ballot_sync(0xffffffffu, is_src != nullptr));  // four a stretch
    if (lane == 0) mbar_arrive_expect_tx(bar, lanes / 4 * stretch * (DIM + 4));
    __syncwarp();
    if (is_src) bulk_load(piece_dst + slot * Rg::kBytes, is_src, stretch * row_bytes, bar);
  };
  advance(warp);
  if (is_step < run.count) issue();
  advance(kWarps);  // to the first step that this warp issues in the loop

  const int eg = (g ^ (g >> 1)) & 1;        // e(g)
  const int tok_a = 2 * g + eg, tok_b = 2 * g + 1 - eg;
  const uint32_t sel_a = eg ? 0x3244u : 0x1044u, sel_b = eg ? 0x1044u : 0x3244u;
  // values: this lane's row of the transposing loads
  const int v_row = lane & 7, v_e = (v_row ^ (v_row >> 1)) & 1;
  const uint32_t v_lane =
      (uint32_t)((2 * v_row + (lane & 8 ? 1 - v_e : v_e)) * (DIM / 2) + (lane & 16)) +
      (uint32_t)(Rg::kCodes + warp * kTokens * (DIM / 2));

  bool dead = false;  // a wait ran out: no more waits and sums, but every barrier
  int seq_tile = run.seq_tile, head = run.head, off = run.off, done = 0, tile = 0;
  RowTile t = row_tile(p, seq_tile);
  while (true) {
    const int piece_steps = min(t.steps - off, run.count - done);
    const int end = t.last;
    // ---- queries: B fragments, column g of tile nt is row t.r0 + 8 nt + g
    uint32_t q[NT][MT][2];
    int seen_to[NT][2];  // one past the last token that columns 2c, 2c + 1 see
    // The tile's power of two: its largest element goes to 2^14 .. 2^15, so that
    // in fp16 every element keeps its digits down to 2^-28 of that.  Where a row
    // would stay below 1 by it, or the power is too far from 1 to be a factor of the
    // keys' scales, every row has its own (own_units): its scores are then brought
    // to their unit in the careful form of a step.  Either way an element is off by
    // at most 2^-25 of its row's largest.
    uint32_t raw[NT][DIM / 8];  // DIM / 4 elements of row 8 nt + g: two a word
    float row_most[NT], most = 0.0f, least = INFINITY;  // least: of rows that are not 0
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g;
#pragma unroll
      for (int i = 0; i < DIM / 8; ++i) raw[nt][i] = 0;
      if (r < t.rows) {
        const int row = t.r0 + r, i = (int)p.by_group((uint32_t)row);
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const T*>(p.q) + (int64_t)(t.q0 + i) * p.q_stride +
            (int64_t)(head * p.group + row - i * p.group) * DIM + c * (DIM / 4));
#pragma unroll
        for (int i4 = 0; i4 < DIM / 32; ++i4)
          reinterpret_cast<uint4*>(raw[nt])[i4] = __ldg(src + i4);
      }
      const T* x = reinterpret_cast<const T*>(raw[nt]);
      row_most[nt] = 0.0f;
#pragma unroll
      for (int i = 0; i < DIM / 4; ++i) {
        const float a = fabsf(to_f32(x[i]));
        if (a < INFINITY) row_most[nt] = fmaxf(row_most[nt], a);
      }
#pragma unroll
      for (int x = 2; x >= 1; x >>= 1)
        row_most[nt] = fmaxf(row_most[nt], __shfl_xor_sync(0xffffffffu, row_most[nt], x));
      most = fmaxf(most, row_most[nt]);
      if (row_most[nt] > 0.0f) least = fminf(least, row_most[nt]);
    }
    most = warp_most(most);
    least = warp_least(least);
    const bool own_units = far_queries(most, least);
    const int k = own_units ? far_tile_power(most) : query_power(most);
    // the accumulators' unit (but for the rows' own) times scale log2(e)
    const float factor = power_of_two(-k) * (p.scale * kLog2e / kCodeUnit);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const T* x = reinterpret_cast<const T*>(raw[nt]);
      const int k_row = own_units ? far_row_power(row_most[nt], k) : k;
      const float up = power_of_two(k_row);
      if (own_units && c == 0) row_unit[warp][8 * nt + g] = power_of_two(k - k_row);
      // channels (d, d + 4) of a word of codes make a register
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 h = __floats2half2_rn(to_f32(x[8 * w + i]) * up, to_f32(x[8 * w + i + 4]) * up);
          q[nt][2 * w + i / 2][i % 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        seen_to[nt][e] = last_seen(p, t, (int)p.by_group((uint32_t)(t.r0 + 8 * nt + 2 * c + e)));
    }
    // steps wholly inside [all_from, all_to) need no mask
    const int i_last = (int)p.by_group((uint32_t)(t.r0 + t.rows - 1));
    const int all_to = min(end, last_seen(p, t, (int)p.by_group((uint32_t)t.r0)));
    const int all_from = p.window ? max(t.first, first_seen(p, last_seen(p, t, i_last))) : 0;

    // Per column: the weights are 2^(t - ref), l their sum, and weight x value
    // scale goes into the value product in fp16.  `ref` is such that the largest
    // of those products so far was 2^10 .. 2^11 when it was set (and moves when
    // one exceeds 2^15, or a weight 2^100): fp16 then holds them with all its digits
    // down to 2^-24 of the largest, whatever scores and scales look like.  (A
    // channel in which every larger product has code 0 keeps what lies above
    // 2^-34 of the row's largest.)
    // m, wtop: the largest score, and the largest product relative to 2^m.
    // shifts: halves of the columns' top_shift in force, 7 bits each, and own_units;
    // where it is not 0, every step takes the careful form.
    constexpr uint32_t kOwnUnits = 1u << 28;
    uint32_t shifts = own_units ? kOwnUnits : 0;
    auto shift_of = [&](int nt, int e) { return (int)(shifts << (25 - 7 * (2 * nt + e))) >> 25 << 1; };
    float o[MT][NT][4], ref[NT][2], l[NT][2], m[NT][2], wtop[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ref[nt][e] = m[nt][e] = -3.0e38f;
        l[nt][e] = wtop[nt][e] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.0f;
    }

    for (int s = done; s < done + piece_steps; ++s) {
      const uint32_t slot = (uint32_t)(s % kStages);
      if (s > 0 && s + kStages - 1 == is_step && !dead) {
        const int old = s - 1;  // the step whose slot this is
        if (is_step < run.count) {
          dead = !mbar_wait(empty + 8 * (old % kStages), (uint32_t)(old / kStages) & 1u, &abort_flag,
                            p.status);
          dead = __any_sync(0xffffffffu, dead);  // (the lanes go on together)
          if (!dead) issue();
        }
        advance(kWarps);
      }
      if (!dead)
        dead = !mbar_wait(full + 8 * slot, (uint32_t)(s / kStages) & 1u, &abort_flag, p.status);
      dead = __any_sync(0xffffffffu, dead);
      const int token0 = t.base + (off + s - done) * kStep + warp * kTokens;
      if (token0 < end && !dead) {
        const uint8_t* buf = smem + slot * Rg::kBytes;
        float acc[2][NT][4];     // q . (key codes) of the two 16-token tiles
        float ks[2][2], vs[2][2];  // scales of the lane's tokens (keys': times factor)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const uint8_t* kp = buf + (warp * kTokens + mt * 16) * (DIM / 2) + c * (DIM / 8);
          uint32_t ka[KW], kb[KW];
          float odd[NT][4];
          if constexpr (KW == 4) {
            *reinterpret_cast<uint4*>(ka) = *reinterpret_cast<const uint4*>(kp + tok_a * (DIM / 2));
            *reinterpret_cast<uint4*>(kb) = *reinterpret_cast<const uint4*>(kp + tok_b * (DIM / 2));
          } else {
            *reinterpret_cast<uint2*>(ka) = *reinterpret_cast<const uint2*>(kp + tok_a * (DIM / 2));
            *reinterpret_cast<uint2*>(kb) = *reinterpret_cast<const uint2*>(kp + tok_b * (DIM / 2));
          }
#pragma unroll
          for (int w = 0; w < KW; ++w)
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // codes 0, 1 (with 4, 5), then 2, 3 (with 6, 7)
              const uint32_t wa = i ? ka[w] >> 8 : ka[w], wb = i ? kb[w] >> 8 : kb[w];
              const uint32_t a0 = codes_f16<false>(wa), a1 = codes_f16<false>(wb);
              const uint32_t a2 = codes_f16<true>(wa), a3 = codes_f16<true>(wb);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                // (two chains of sums: an MMA waits for the one before it in its chain)
                float(&d)[4] = i ? odd[nt] : acc[mt][nt];
                if (w == 0)
                  mma16816_new(d, a0, a1, a2, a3, q[nt][i][0], q[nt][i][1]);
                else
                  mma16816(d, a0, a1, a2, a3, q[nt][2 * w + i][0], q[nt][2 * w + i][1]);
              }
            }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[mt][nt][r] += odd[nt][r];
          const uint8_t* scales = buf + 2 * Rg::kCodes + (warp * kTokens + mt * 16) * 2 + g * 4;
          const uint32_t ks2 = *reinterpret_cast<const uint32_t*>(scales);
          const uint32_t vs2 = *reinterpret_cast<const uint32_t*>(scales + 2 * kStep);
          ks[mt][0] = __uint_as_float(__byte_perm(ks2, 0, sel_a)) * factor;
          ks[mt][1] = __uint_as_float(__byte_perm(ks2, 0, sel_b)) * factor;
          vs[mt][0] = __uint_as_float(__byte_perm(vs2, 0, sel_a));
          vs[mt][1] = __uint_as_float(__byte_perm(vs2, 0, sel_b));
        }
        // scores that are masked, by bit (mt NT + nt) 4 + register
        uint32_t hidden = 0;
        if (token0 < all_from || token0 + kTokens > all_to) {
#pragma unroll
          for (int i = 0; i < 8 * NT; ++i) {
            const int token = token0 + i / (4 * NT) * 16 + (i & 2 ? tok_b : tok_a);
            const int to = seen_to[i / 4 % NT][i & 1];
            if (token >= min(end, to) || token < max(t.first, first_seen(p, to))) hidden |= 1u << i;
          }
        }
        // weights, and weights x value scales as B fragments of the value product
        uint32_t pw[2][NT][2];
        float part[NT][2];
        __half2 most2 = __half2half2(__half(0.0f));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float sum[2];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              const float pa = ex2(fmaf(acc[mt][nt][e], ks[mt][0], -ref[nt][e]));
              const float pb = ex2(fmaf(acc[mt][nt][2 + e], ks[mt][1], -ref[nt][e]));
              sum[mt] = pa + pb;
              w[mt][e] = pa * vs[mt][0];
              w[mt][2 + e] = pb * vs[mt][1];
            }
            part[nt][e] = sum[0] + sum[1];
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const __half2 h = __floats2half2_rn(w[mt][2 * r], w[mt][2 * r + 1]);
              most2 = __hmax2(most2, __habs2(h));
              pw[mt][nt][r] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        // masked scores, or weights out of range: once more, with care
        bool again = (hidden | shifts) != 0 || !__hble2(most2, __half2half2(__half(32768.0f)));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) again |= part[nt][0] > kFar || part[nt][1] > kFar;
        if (__any_sync(0xffffffffu, again)) {
          if (shifts & kOwnUnits) {
            __syncwarp();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float unit = row_unit[warp][8 * nt + 2 * c + e];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  float& s4 = acc[i / 2][nt][(i & 1) * 2 + e];
                  s4 = s4 * ks[i / 2][i & 1] * unit;
                }
              }
            ks[0][0] = ks[0][1] = ks[1][0] = ks[1][1] = 1.0f;
          }
          bool far = shifts != 0;  // a row whose products take a power of two besides
          float down[NT][2];       // by how many binades each row's reference falls
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float t4[4];  // scores
              float high = m[nt][e];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const bool hide = hidden >> ((i / 2 * NT + nt) * 4 + (i & 1) * 2 + e) & 1;
                t4[i] = hide ? -INFINITY : acc[i / 2][nt][(i & 1) * 2 + e] * ks[i / 2][i & 1];
                high = fmaxf(high, t4[i]);
              }
#pragma unroll
              for (int x = 4; x <= 16; x <<= 1)
                high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, x));
              // (by square roots of the weights: a weight itself is 0 below 2^-126, its
              // product with a large scale may yet be the largest)
              float root = ex2(0.5f * (m[nt][e] - high));
              float top = wtop[nt][e] * root * root;
              const float before = top;
#pragma unroll
              for (int i = 0; i < 4; ++i) {  // (a NaN is passed over)
                root = ex2(0.5f * (t4[i] - high));
                top = fmaxf(top, fabsf(root * vs[i / 2][i & 1] * root));
              }
#pragma unroll
              for (int x = 4; x <= 16; x <<= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
              float next = ref[nt][e];
              const float lead = fminf(fmaxf(top, kSpanLeast), kSpanMost);
              far |= top != lead && top > 0.0f;
              // (the eight lanes of a column agree on all of this)
              if (high > m[nt][e] || top > before) next = high - (float)to_level(lead);
              m[nt][e] = high;
              wtop[nt][e] = top;
              down[nt][e] = ref[nt][e] - next;
              ref[nt][e] = next;
              l[nt][e] *= ex2(down[nt][e]);
              part[nt][e] = 0.0f;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float w = ex2(t4[i] - next);
                part[nt][e] += w;
                // what a row does not see has weight 0 whatever its scale
                acc[i / 2][nt][(i & 1) * 2 + e] = t4[i] == -INFINITY ? 0.0f : w * vs[i / 2][i & 1];
              }
            }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) far |= fabsf(m[nt][e]) >= kFarScore && wtop[nt][e] > 0.0f;
          if (__any_sync(0xffffffffu, far)) {
            uint32_t next_shifts = shifts & kOwnUnits;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int shift = top_shift(m[nt][e] - ref[nt][e], wtop[nt][e]);
                next_shifts |= (uint32_t)(shift >> 1 & 127) << 7 * (2 * nt + e);
                // (o hardly grows: what was the largest product is not more now)
                down[nt][e] = fminf(down[nt][e] + (float)(shift - shift_of(nt, e)), 100.0f);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i / 2][nt][(i & 1) * 2 + e] *= power_of_two(shift);
              }
            shifts = next_shifts;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float f = ex2(down[nt][e]);
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[i][nt][e] *= f;
                o[i][nt][2 + e] *= f;
              }
            }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                pw[mt][nt][r] = pack_f16(acc[mt][nt][2 * r], acc[mt][nt][2 * r + 1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) l[nt][e] += part[nt][e];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t b[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            b[nt][0] = transpose8x8(pw[mt][nt][0]);
            b[nt][1] = transpose8x8(pw[mt][nt][1]);
          }
#pragma unroll
          for (int u = 0; u < DIM / 64; ++u) {
            uint32_t v[4];
            load_transposed(v, ring + slot * Rg::kBytes + v_lane + mt * 16 * (DIM / 2) + u * 32);
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // MMA tile 4 u + i: codes 0, 1, then 2, 3 of a chunk
              const uint32_t x = i & 1 ? v[i & 2] >> 8 : v[i & 2];
              const uint32_t y = i & 1 ? v[(i & 2) + 1] >> 8 : v[(i & 2) + 1];
              const uint32_t a0 = codes_f16<false>(x), a1 = codes_f16<true>(x);
              const uint32_t a2 = codes_f16<false>(y), a3 = codes_f16<true>(y);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(o[4 * u + i][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
            }
          }
        }
      }
      __syncwarp();  // every lane has read its part of the slot
      if (lane == 0) mbar_arrive(empty + 8 * slot);
    }

    // ---- join the warps: o, l relative to the largest reference
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x <= 16; x <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
        if (g == 0) {
          merge_ref[warp][8 * nt + 2 * c + e] = ref[nt][e];
          merge_l[warp][8 * nt + 2 * c + e] = l[nt][e];
        }
      }
    // a buffer [row][MMA tile][g][2] that the warps add to in turn, rows 4 floats
    // apart from a multiple of 32: the accesses of a phase fall on different banks
    float* mo = reinterpret_cast<float*>(smem + Rg::kTotal);
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      __syncthreads();
      if (w != warp) continue;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * nt + 2 * c + e;
          float all = merge_ref[0][r];
#pragma unroll
          for (int i = 1; i < kWarps; ++i) all = fmaxf(all, merge_ref[i][r]);
          const float f =
              ex2(ref[nt][e] - all) * power_of_two(-shift_of(nt, e));
          float2* dst = reinterpret_cast<float2*>(mo + r * ROW + 2 * g);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            float2 v = make_float2(o[i][nt][e] * f, o[i][nt][2 + e] * f);
            if (w > 0) {
              v.x += dst[8 * i].x;
              v.y += dst[8 * i].y;
            }
            dst[8 * i] = v;
          }
        }
    }
    __syncthreads();
    const bool whole = piece_steps == t.steps;
    const int64_t share = ((int64_t)blockIdx.x * 2 + (off == 0)) * p.tile_rows;
    if (p.joins > 0 && off == 0 && (!whole || p.by_tile) && threadIdx.x == 0) {
      const int64_t last = (run.pos + done + tile * kTileCost + t.steps - 1) / run.per;  // the CTA of its last step
      p.join[p.by_tile ? seq_tile * p.cache.heads + head : (int)blockIdx.x] =
          Kv4Join{seq_tile, head, (int)blockIdx.x, whole ? -1 : (int)last};
    }
    // a thread takes 4 channels of a row: 32 q + 4 g8 and on, tiles 2 q and 2 q + 1
    for (int i = threadIdx.x; i < R * (DIM / 4); i += kWarps * 32) {
      const int r = i / (DIM / 4), d = i % (DIM / 4) * 4, chunk_q = d / 32, g8 = d / 4 % 8;
      if (r >= t.rows) continue;
      float all = merge_ref[0][r], sum = 0.0f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) all = fmaxf(all, merge_ref[w][r]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += merge_l[w][r] * ex2(merge_ref[w][r] - all);
      const float* src = mo + r * ROW + 32 * chunk_q + 2 * g8;
      const float2 x = *reinterpret_cast<const float2*>(src);
      const float2 y = *reinterpret_cast<const float2*>(src + 16);
      const bool none = sum == 0.0f;
      const float inv = none ? 0.0f : (1.0f / kCodeUnit) / sum;
      const float lse = none ? -INFINITY : all + log2f(sum);
      if (whole) {
        const int64_t at = out_row(p, t, head, t.r0 + r);
        T h[4] = {from_f32<T>(x.x * inv), from_f32<T>(x.y * inv), from_f32<T>(y.x * inv),
                  from_f32<T>(y.y * inv)};
        *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + at * DIM + d) =
            *reinterpret_cast<const uint2*>(h);
        if (p.lse && d == 0) p.lse[at] = lse * kLn2;
      } else {
        *reinterpret_cast<float4*>(p.share_o + (share + r) * DIM + d) =
            make_float4(x.x * inv, x.y * inv, y.x * inv, y.y * inv);
        if (d == 0) p.share_lse[share + r] = lse;
      }
    }
    done += piece_steps;
    if (done == run.count) break;
    ++tile;
    __syncthreads();  // the merge buffers are free again
    off = 0;
    if (++head == p.cache.heads) {
      head = 0;
      t = next_row_tile(p, &seq_tile);
    }
  }
  if (dead) {  // let the copies in flight land (again with a limit)
    volatile int go_on = 0;
    for (int k = max(0, run.count - kStages); k < run.count; ++k)
      mbar_wait(full + 8 * (k % kStages), (uint32_t)(k / kStages) & 1u, &go_on, p.status,
                kWaitLimitNs / 8);
  }
}

template <typename T, int DIM, int NT>
cudaError_t launch_tile(const Kv4AttnParams& p, cudaStream_t s) {
  const int smem = Ring<DIM>::kTotal + 8 * NT * (DIM + 4) * 4;
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
  kernel<<<p.ctas, kWarps * 32, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const Kv4AttnParams& p, cudaStream_t s) {
  if (p.cache.dim == 64)
    return p.tile_rows == 8 ? launch_tile<T, 64, 1>(p, s) : launch_tile<T, 64, 2>(p, s);
  return p.tile_rows == 8 ? launch_tile<T, 128, 1>(p, s) : launch_tile<T, 128, 2>(p, s);
}

}  // namespace

int kv4_rows_per_sm(int tile_rows) { return tile_rows == 8 ? 3 : 2; }

cudaError_t launch_kv4_rows(int dtype, const Kv4AttnParams& p, cudaStream_t s) {
  return dtype == LBGEMM_BF16 ? launch_typed<__nv_bfloat16>(p, s) : launch_typed<__half>(p, s);
}

}  // namespace lbg
