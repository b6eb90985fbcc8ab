// w4_rows.cu -- products with 4-bit weights for few tokens: the weights stream
// through warp MMAs once for 8 columns (tokens).
//
//   linear  Y[m][n] = row_scale[n] * sum_k X[m][k] * (code * scale)[n][k]
//   up      h[pick][i] = silu(gate) * up, for every pick (token, expert)
//   down    y[t] = sum over a token's picks, in order, of weight * (Down h[pick])
//
// Bound by the weights' stream from HBM (about 0.53 bytes a weight), and close
// behind it by issue slots: a word of eight codes takes twelve operations to
// become halves (w4_codes.cuh).  So the codes go to the MMA's 16-row side, which
// has no row to spare, and the tokens to its 8-column side.  Measured: 1 token x 128000 x
// 4096 in 64 us (4.2 TB/s), x 11008 x 4096 in 13.0 beyond L2 and 10.7 from it (4 of them
// launch, staging and the last sums); 24 tokens, 6 of 64 experts of 2048 / 1024, in 68 us (2.8
// TB/s; logic operations half of the time).
//
// A CTA an SM, 24 warps.  CTAs take equal runs of weight rows: of the rows of all
// experts with a pick one after the other (linear, up), or, so that a token's
// picks are joined within a CTA, the same rows of every such expert (down).  A run
// goes in tiles of up to 16 rows and steps of 256 elements, tile by tile, and every
// warp takes an equal piece of that row of steps: warps stay even whatever k is,
// and meet few tiles.  Lane (g, t) loads 32
// consecutive codes at 32 t of rows g and g + 8 of each half of a step: the MMA's k
// slots are any 16 elements as long as both sides agree, so a word of codes (8
// neighbours) and the 16 bytes of a token's same 8 elements feed two MMAs with no
// shuffle.  Codes are copied `depth` steps ahead into a ring in shared memory, in
// which every lane reads what it copied itself (so no barrier is in the loop);
// scales come a step ahead into registers.  Rows and columns that a tile does not
// have are computed from others' data and not stored.
//
// Tokens are laid out in shared memory first (STAGED), in the order in which lanes
// read them.  Where they do not fit, the experts read them through L1, at 2 conflicts a
// load; a linear layer goes to w4_tiles.cu.
//
// A tile's shares of the warps that met it are added in shared memory, in the
// order of the warps, at the end of the run (of a round of it, where it has more
// tiles than there is room for shares).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "attn_common.cuh"
#include "ffn.h"
#include "ptx.cuh"
#include "w4_codes.cuh"
#include "w4_kernels.h"

namespace lbg {
namespace {

constexpr int kStep = 256;
constexpr int kSlotBytes = 2048;  // a warp's codes of a step
constexpr int kMaxDepth = 6;
constexpr int kSmem = 227 * 1024;  // of an SM; kSmem / 2 - 512 of one of two CTAs

enum Mode { kLinear, kUp, kDown };

// What a CTA knows of the picks: experts with a pick ("segments", of up to 8
// picks each), and the picks in their order.
struct Picks {
  int segments;
  short expert[kRowsMaxPicks], first[kRowsMaxPicks], count[kRowsMaxPicks];
  short pick[kRowsMaxPicks];
};

struct NoPicks {
  static constexpr int segments = 1;
  static constexpr short expert[1] = {0}, first[1] = {0}, count[1] = {0}, pick[1] = {0};
};
template <int MODE>
using PicksOf = std::conditional_t<MODE == kLinear, NoPicks, Picks>;

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1,
                                                   uint32_t a2, uint32_t a3, uint32_t b0,
                                                   uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes into shared memory; or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_if(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint4 load_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ void copies_done(int behind) {  // all but the last `behind` steps'
  switch (behind) {
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
  }
}

// Sorts the picks by expert (all threads of the CTA; `counts`: kRowsMaxExperts + 1).
__device__ void sort_picks(const W4RowsParams& p, int columns, Picks& picks, int* counts) {
  const int total = p.picks;
  if (total <= 32) {  // a warp settles it in registers, in the order of first appearance
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      const int e = lane < total ? p.ids[lane] : -1;
      if (e >= p.experts) atomicOr(p.status, kStatusBadIndex);
      const bool live = e >= 0 && e < p.experts;
      const uint32_t same = __match_any_sync(0xffffffffu, live ? e : -1);
      const int leader = __ffs(same) - 1;
      const int n = live && leader == lane ? __popc(same) : 0;
      const int parts = (n + columns - 1) / columns;
      int a = n, b = parts;  // running sums: picks and segments
#pragma unroll
      for (int off = 1; off < 32; off *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, a, off), y = __shfl_up_sync(0xffffffffu, b, off);
        if (lane >= off) a += x, b += y;
      }
      const int first = a - n, at = __shfl_sync(0xffffffffu, first, leader);
      if (live) picks.pick[at + __popc(same & ((1u << lane) - 1))] = (short)lane;
      for (int q = 0; q < parts; ++q) {
        const int seg = b - parts + q;
        picks.expert[seg] = (short)e;
        picks.first[seg] = (short)(first + q * columns);
        picks.count[seg] = (short)min(n - q * columns, columns);
      }
      if (lane == 31) picks.segments = b;
    }
    __syncthreads();
    return;
  }
  for (int e = threadIdx.x; e <= p.experts; e += blockDim.x) counts[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += blockDim.x) {
    const int e = p.ids[i];
    if (e >= 0 && e < p.experts) atomicAdd(&counts[e], 1);
    if (e >= p.experts) atomicOr(p.status, kStatusBadIndex);
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // a warp's running sums: picks and segments before an expert
    int before = 0, segments = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int e = e0 + threadIdx.x;
      const int n = e < p.experts ? counts[e] : 0;
      int a = n, b = (n + columns - 1) / columns;
#pragma unroll
      for (int off = 1; off < 32; off *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, a, off), y = __shfl_up_sync(0xffffffffu, b, off);
        if (threadIdx.x >= off) a += x, b += y;
      }
      if (n > 0) {
        int at = before + a - n, seg = segments + b - (n + columns - 1) / columns;
        counts[e] = at;  // where its next pick goes
        for (int left = n; left > 0; left -= columns, at += columns, ++seg) {
          picks.expert[seg] = (short)e;
          picks.first[seg] = (short)at;
          picks.count[seg] = (short)min(left, columns);
        }
      }
      before += __shfl_sync(0xffffffffu, a, 31);
      segments += __shfl_sync(0xffffffffu, b, 31);
    }
    if (threadIdx.x == 0) picks.segments = segments;
  }
  __syncthreads();
  // In the order of the picks, so that every CTA has the same ones in a segment.
  if (threadIdx.x < 32) {
    for (int i0 = 0; i0 < total; i0 += 32) {
      const int i = i0 + threadIdx.x;
      const int e = i < total ? p.ids[i] : -1;
      const bool live = e >= 0 && e < p.experts;
      const uint32_t same = __match_any_sync(0xffffffffu, live ? e : -1);
      const int before = __popc(same & ((1u << threadIdx.x) - 1));
      const int at = live ? counts[e] + before : 0;
      __syncwarp();
      if (live) picks.pick[at] = (short)i;
      if (live && before == 0) counts[e] = at + __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
}

// The run of a CTA as tiles.
template <int MODE>
struct Run {
  int rows_per_segment;  // of the whole matrix (linear, up) or of this CTA (down)
  int first_segment, first_row, head_tiles, body_tiles, tiles;
  int end_row;           // of the run, counted from first_segment's row 0
  __device__ __forceinline__ void tile(int i, int& segment, int& row, int& rows) const {
    if (MODE == kDown) {
      segment = i / body_tiles;
      const int r = 16 * (i - segment * body_tiles);
      rows = min(16, rows_per_segment - r);
      row = first_row + r;
      return;
    }
    int s = 0, r = first_row + 16 * i;
    if (MODE == kUp && i >= head_tiles) {
      s = 1 + (i - head_tiles) / body_tiles;
      r = 16 * (i - head_tiles - (s - 1) * body_tiles);
    }
    segment = first_segment + s;
    row = r;
    rows = min(min(16, rows_per_segment - r), end_row - s * rows_per_segment - r);
  }
};

// kWarps: 24, as many as registers allow.  A mixture of few picks takes 12 and half of the
// shared memory, so that the CTAs of `down` stand beside those of `up`: they look up their
// picks and copy their first codes while `up` runs (1 token, 6 experts: 17.4 -> 14.9 us from L2).
constexpr int kAllWarps = 24, kFewWarps = 12, kFewPicks = 16;
// Tiles of 8 columns in a round (24 tokens to 64 experts, 49 and 58 tiles a CTA: 68.3 us,
// 69.7 with room for 48; no gain from 80).
constexpr int kShares = 64;

template <typename T, int MODE, bool STAGED, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps == kFewWarps ? 2 : 1)
    w4_rows_kernel(const W4RowsParams p) {
  constexpr int kThreads = 32 * kWarps;
  constexpr int COLS = 8, SHARE = 16 * COLS;  // columns; numbers of a tile
  extern __shared__ __align__(128) uint8_t smem[];
  float* shares = reinterpret_cast<float*>(smem + p.at_shares);  // [batch + kWarps][SHARE]
  // down: the picks' outputs [rows][picks]
  float* values = reinterpret_cast<float*>(smem + p.at_values);
  uint8_t* staged = smem + p.at_tokens;
  // (the linear layer's only segment is all rows and the tokens in their order)
  __shared__ PicksOf<MODE> picks;
  __shared__ int counts[MODE == kLinear ? 1 : kRowsMaxExperts + 1];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const int k = p.k;

  if (MODE != kDown) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (MODE != kLinear) sort_picks(p, COLS, picks, counts);
  auto columns_of = [&](int segment) { return MODE == kLinear ? p.picks : picks.count[segment]; };
  auto pick_of = [&](int segment, int column) {
    return MODE == kLinear ? column : picks.pick[picks.first[segment] + column];
  };
  auto first_row_of = [&](int segment) {
    return MODE == kLinear ? 0u : (uint32_t)picks.expert[segment] * (uint32_t)p.n;
  };

  // ---- the run ----
  Run<MODE> run;
  const int n = (int)p.n;
  const int cta = blockIdx.x;
  int own_rows = 0;
  if (MODE != kUp) {
    own_rows = p.rows_each + (cta < p.rows_more);
    run.first_row = cta * p.rows_each + min(cta, p.rows_more);
    run.first_segment = 0;
    run.rows_per_segment = MODE == kDown ? own_rows : n;
    run.end_row = run.first_row + own_rows;
    run.body_tiles = run.head_tiles = (own_rows + 15) / 16;
    run.tiles = MODE == kDown ? picks.segments * run.body_tiles : run.body_tiles;
  } else {
    // pairs of rows: a gate's row and its up row stay together
    const uint32_t units = (uint32_t)picks.segments * (uint32_t)(n / 2), ctas = gridDim.x;
    const uint32_t each = units / ctas, more = units - each * ctas;
    const uint32_t a = 2 * (cta * each + min((uint32_t)cta, more));
    const uint32_t b = a + 2 * (each + ((uint32_t)cta < more));
    run.rows_per_segment = n;
    run.first_segment = (int)(a / n);
    run.first_row = (int)(a - run.first_segment * n);
    run.end_row = (int)(b - run.first_segment * n);
    run.body_tiles = (n + 15) / 16;
    run.head_tiles = run.tiles = (min(run.end_row, n) - run.first_row + 15) / 16;
    if (run.end_row > n) {
      const int rest = run.end_row - n, whole = rest / n;
      run.tiles += whole * run.body_tiles + (rest - whole * n + 15) / 16;
    }
  }

  // ---- rounds ----
  const int steps = p.steps;  // of a tile
  // tiles of a round: as many in each, as few rounds as there is room for
  const int rounds = (run.tiles + p.batch - 1) / p.batch;
  const int TB = rounds > 1 ? (run.tiles + rounds - 1) / rounds : run.tiles;

  // A place in this warp's part of a round.
  struct Place {
    int round, tile, j, left;
  };
  auto begin = [&](Place& x) {
    const int total = min(TB, run.tiles - x.round * TB) * steps;
    const int each = total / kWarps, more = total - each * kWarps;
    const int first = warp * each + min(warp, more);
    x.left = each + (warp < more);
    x.tile = first / steps;
    x.j = first - x.tile * steps;
    x.tile += x.round * TB;
  };
  auto next_round = [&](Place& x) {
    if (++x.round < rounds) begin(x);
  };
  // On from a place without steps left to one that has some (or the end).
  auto settle = [&](Place& x) {
    while (x.left == 0 && x.round < rounds) next_round(x);
  };
  // A place's rows g and g + 8 (clamped: a row that the tile has not is another of it).
  auto rows_at = [&](const Place& x, uint32_t (&r)[2]) {
    int segment, row, rows;
    run.tile(x.tile, segment, row, rows);
    const uint32_t first = first_row_of(segment) + row;
    r[0] = first + min(g, rows - 1);
    r[1] = first + min(g + 8, rows - 1);
  };
  // Steps that lie within a row; of a later one, half h of this lane does where
  // what is left is more than 128 h.
  const int whole = k / kStep;
  auto left_of = [&](int step) { return k - step * kStep - 32 * t; };

  // ---- codes, `depth` steps ahead ----
  const uint32_t code_row = k / 2, scale_row = k / p.group;
  Place ahead = {0, 0, 0, 0};
  if (rounds > 0) begin(ahead);
  Place at = ahead;  // (every warp goes through every round)
  settle(ahead);
  Place scaled = ahead;
  const uint8_t *code_ptr[2], *scale_ptr[2];
  auto aim_codes = [&] {
    if (ahead.round >= rounds) return;
    uint32_t r[2];
    rows_at(ahead, r);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      code_ptr[i] = p.w.codes + (uint64_t)r[i] * code_row + 16 * t +
                    128 * ahead.j;
  };
  aim_codes();
  const uint32_t ring = smem_addr(smem) + warp * p.depth * kSlotBytes + lane * 16;
  uint32_t to = ring;  // the slot that is copied to next
  const uint32_t ring_end = ring + p.depth * kSlotBytes;
  auto copy_codes = [&] {
    if (ahead.left > 0) {
      const int step = ahead.j;
      if (step < whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) copy16(to + (2 * h + i) * 512, code_ptr[i] + 64 * h);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            copy16_if(to + (2 * h + i) * 512, code_ptr[i] + 64 * h, left_of(step) > 128 * h);
      }
      --ahead.left;
      ++ahead.j;
      if (ahead.left == 0 || ahead.j == steps) {
        if (ahead.j == steps) ahead.j = 0, ++ahead.tile;
        settle(ahead);
        aim_codes();
      } else {
        code_ptr[0] += 128;
        code_ptr[1] += 128;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    to += kSlotBytes;
    if (to == ring_end) to = ring;
  };
  // ---- scales, a step ahead ----
  const int shift = p.group == 32 ? 0 : p.group == 64 ? 1 : 2;  // of 32-element pieces
  uint32_t scale[2][2];  // [half of the step][row g, row g + 8]
  auto aim_scales = [&] {
    if (scaled.round >= rounds) return;
    uint32_t r[2];
    rows_at(scaled, r);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      scale_ptr[i] = p.w.scales + (uint64_t)r[i] * scale_row +
                     ((8 * scaled.j + t) >> shift);
      if (t == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.w.row_scales + r[i]));
    }
  };
  aim_scales();
  auto load_scales = [&] {
    if (scaled.left == 0) return;
    const int step = scaled.j;
    if (step < whole) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) scale[h][i] = __ldg(scale_ptr[i] + ((4 * h) >> shift));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i)  // (past the row: weights of 0)
          scale[h][i] = left_of(step) > 128 * h ? __ldg(scale_ptr[i] + ((4 * h) >> shift)) : 0;
    }
    --scaled.left;
    ++scaled.j;
    if (scaled.left == 0 || scaled.j == steps) {
      if (scaled.j == steps) scaled.j = 0, ++scaled.tile;
      settle(scaled);
      aim_scales();
    } else {
      scale_ptr[0] += 8 >> shift;
      scale_ptr[1] += 8 >> shift;
    }
  };
  for (int d = 0; d < p.depth; ++d) copy_codes();
  load_scales();
  // (weights and picks are older than the launch before this one; h is not)
  if (MODE == kDown) asm volatile("griddepcontrol.wait;" ::: "memory");

  float acc[4];
  // This lane's column: in memory, or staged: vector v of a piece at v * pitch, its
  // 16 bytes in the order that lanes read them, so that 8 lanes of neighbouring
  // vectors meet no conflict: [half step][word][t].
  const T* column = nullptr;
  const uint8_t* line = nullptr;
  const int pitch = steps * 512 + 64;
  uint32_t from = ring;

  while (at.round < rounds) {
    if (STAGED && at.round == 0) {
      const int pieces = steps * 32, vectors = MODE == kUp ? p.picks / p.top_k : p.picks;
      for (int v = warp; v < vectors; v += kWarps)
        for (int o = lane; o < pieces; o += 32) {
          const int at_k = 8 * o;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (at_k < k)
            x = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + v * p.x_stride + at_k);
          *reinterpret_cast<uint4*>(staged + v * pitch + (o >> 4) * 256 + (o & 3) * 64 +
                                    (o >> 2 & 3) * 16) = x;
        }
      __syncthreads();
    }
    while (at.left > 0) {
      // the steps of a tile
      int segment = 0, row, rows;
      if (MODE != kLinear) run.tile(at.tile, segment, row, rows);
      const int most = columns_of(segment) - 1;
      {
        const int pick = pick_of(segment, min(g, most));
        const int v = MODE == kUp ? pick / p.top_k : pick;
        if (STAGED)
          line = staged + v * pitch + 16 * t + at.j * 512;
        else
          column = static_cast<const T*>(p.x) + v * p.x_stride + 32 * t + at.j * kStep;
      }
      acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
      const int stop = min(steps, at.j + at.left);
      at.left -= stop - at.j;
      for (; at.j < stop; ++at.j) {
        W4Scale<T> lo[2], hi[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) w4_scales(scale[h][0], scale[h][1], lo[h], hi[h]);
        load_scales();
        copies_done(p.depth - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 cl = load_shared(from + 2 * h * 512);
          const uint4 ch = load_shared(from + (2 * h + 1) * 512);
          uint4 x[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if (STAGED)
              x[w] = *reinterpret_cast<const uint4*>(line + h * 256 + w * 64);
            else if (at.j < whole || left_of(at.j) > 128 * h)
              x[w] = *reinterpret_cast<const uint4*>(column + 128 * h + 8 * w);
            else
              x[w] = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a[4], c[4];
            w4_word(w == 0 ? cl.x : w == 1 ? cl.y : w == 2 ? cl.z : cl.w, lo[h], a);
            w4_word(w == 0 ? ch.x : w == 1 ? ch.y : w == 2 ? ch.z : ch.w, hi[h], c);
            mma<T>(acc, a[0], c[0], a[1], c[1], x[w].x, x[w].y);
            mma<T>(acc, a[2], c[2], a[3], c[3], x[w].z, x[w].w);
          }
        }
        // (each lane has read its own bytes of the slot: the next copy may land on it)
        copy_codes();
        from += kSlotBytes;
        if (from == ring_end) from = ring;
        if (STAGED)
          line += 512;
        else
          column += kStep;
      }
      // This warp's share of the tile: in place tile + warp, which no other share of the
      // round has (along the row of steps one of both grows).
      float* s = shares + (at.tile - at.round * TB + warp) * SHARE;
      *reinterpret_cast<float2*>(s + g * COLS + 2 * t) = make_float2(acc[0], acc[1]);
      *reinterpret_cast<float2*>(s + (g + 8) * COLS + 2 * t) = make_float2(acc[2], acc[3]);
      if (at.j == steps) at.j = 0, ++at.tile;
    }
    __syncthreads();

    // ---- the round's sums ----
    const int first_tile = at.round * TB, count = min(TB, run.tiles - first_tile);
    const int each = count * steps / kWarps, more = count * steps - each * kWarps;
    auto warp_of = [&](int q) {  // whose step q of the round is
      const int longer = more * (each + 1);
      return q < longer ? q / (each + 1) : more + (q - longer) / each;
    };
    // a warp a tile, its lanes along the rows (up: pairs of rows) of a column, then the next
    constexpr int log_rows = MODE == kUp ? 3 : 4;
    for (int which = warp; which < count; which += kWarps) {
      int segment, row, rows;
      run.tile(first_tile + which, segment, row, rows);
      const int cols = columns_of(segment);
      const int w0 = warp_of(which * steps), w1 = warp_of((which + 1) * steps - 1);
      const float* scales = p.w.row_scales + first_row_of(segment) + row;
      for (int i = lane; i < cols << log_rows; i += 32) {
        const int col = i >> log_rows;
        const int r = (i & ((1 << log_rows) - 1)) * (MODE == kUp ? 2 : 1);
        if (r >= rows) continue;
        const int pick = pick_of(segment, col);
        const float scale0 = __ldg(scales + r), scale1 = MODE == kUp ? __ldg(scales + r + 1) : 0.0f;
        const float* s = shares + (which + w0) * SHARE + r * COLS + col;
        float v = 0.0f, u = 0.0f;
        for (int w = w0; w <= w1; ++w, s += SHARE) {
          v += s[0];
          if (MODE == kUp) u += s[COLS];
        }
        if (MODE == kUp) {
          v *= scale0;
          u *= scale1;
          static_cast<T*>(p.y)[pick * p.y_stride + (row + r) / 2] =
              from_f32<T>(silu_times(v, u));
        } else if (MODE == kDown) {
          values[(row - run.first_row + r) * p.picks + pick] = v * scale0;
        } else {
          static_cast<T*>(p.y)[pick * p.y_stride + row + r] = from_f32<T>(v * scale0);
        }
      }
    }
    next_round(at);
    if (at.round < rounds) __syncthreads();  // (the shares' places are used again)
  }
  if (MODE == kDown) {
    __syncthreads();
    const int tokens = p.picks / p.top_k;
    for (int i = threadIdx.x; i < tokens * own_rows; i += kThreads) {
      const int token = i / own_rows, r = i - token * own_rows;
      float v = 0.0f;
      for (int j = 0; j < p.top_k; ++j) {
        const int pick = token * p.top_k + j, e = p.ids[pick];
        if (e >= 0 && e < p.experts) v += p.weights[pick] * values[r * p.picks + pick];
      }
      static_cast<T*>(p.y)[token * p.y_stride + run.first_row + r] = from_f32<T>(v);
    }
  }
}

// ---- how a launch lays out its shared memory -------------------------------------------
constexpr int kStatic = sizeof(Picks) + 4 * (kRowsMaxExperts + 1) + 256;
constexpr int kStaticLinear = 512;

int ctas_for(int64_t rows, int sm_count) {  // no CTA without a row
  return (int)std::min<int64_t>(sm_count, rows);
}

// Fills in the cut of a linear layer; false where its tokens do not fit.
bool cut_linear(W4RowsParams& p, int sm_count) {
  const int ctas = ctas_for(p.n, sm_count);
  p.rows_each = (int)(p.n / ctas);
  p.rows_more = (int)(p.n % ctas);
  const int rows = p.rows_each + (p.rows_more > 0), tiles = (rows + 15) / 16;
  p.batch = std::min(tiles, kShares);
  p.steps = (p.k + kStep - 1) / kStep;
  const int shares = (p.batch + kAllWarps) * 512;
  const int64_t tokens = (int64_t)p.picks * (p.steps * kStep * 2 + 64);
  const int64_t left = kSmem - kStaticLinear - shares - tokens;
  if (left < 2 * kAllWarps * kSlotBytes) return false;
  p.depth = (int)std::min<int64_t>(kMaxDepth, left / (kAllWarps * kSlotBytes));
  p.at_shares = p.depth * kAllWarps * kSlotBytes;
  p.at_tokens = p.at_shares + shares;
  p.bytes = p.at_tokens + (int)tokens;
  return true;
}

// ... and of a pass over the experts: staged where two slots of the ring are left.
bool cut_experts(W4RowsParams& p, int warps, int vectors, int values) {
  const int smem = warps == kFewWarps ? kSmem / 2 - 512 : kSmem;
  p.batch = warps == kFewWarps ? 24 : kShares;
  const int shares = (p.batch + warps) * 512;
  p.steps = (p.k + kStep - 1) / kStep;
  const int64_t tokens = (int64_t)vectors * (p.steps * kStep * 2 + 64);
  const int held = (values * 4 + 15) / 16 * 16;
  const int room = smem - kStatic - shares - held;
  const bool staged = tokens <= room - 2 * warps * kSlotBytes;
  p.depth = std::min<int>(kMaxDepth, (int)((room - (staged ? tokens : 0)) / (warps * kSlotBytes)));
  if (!staged) p.depth = 2;  // (L1 is what is left)
  p.at_shares = p.depth * warps * kSlotBytes;
  p.at_values = p.at_shares + shares;
  p.at_tokens = p.at_values + held;
  p.bytes = p.at_tokens + (staged ? (int)tokens : 0);
  return staged;
}

template <typename T, int MODE, bool STAGED, int WARPS = kAllWarps>
cudaError_t launch(const W4RowsParams& p, int ctas, cudaStream_t s) {
  auto kernel = w4_rows_kernel<T, MODE, STAGED, WARPS>;
  static std::atomic<uint64_t> set{0};  // devices on which the kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(set.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmem - (MODE == kLinear ? kStaticLinear : kStatic));
    if (e != cudaSuccess) return e;
    set |= uint64_t(1) << dev;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(32 * WARPS);
  cfg.dynamicSmemBytes = p.bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = MODE == kDown ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, int MODE>
cudaError_t launch_mode(const W4RowsParams& p, int warps, bool staged, int ctas, cudaStream_t s) {
  if constexpr (MODE == kLinear) {
    return launch<T, MODE, true>(p, ctas, s);
  } else {
    if (warps == kFewWarps)
      return staged ? launch<T, MODE, true, kFewWarps>(p, ctas, s)
                    : launch<T, MODE, false, kFewWarps>(p, ctas, s);
    return staged ? launch<T, MODE, true>(p, ctas, s) : launch<T, MODE, false>(p, ctas, s);
  }
}

template <int MODE>
cudaError_t launch_any(int dtype, const W4RowsParams& p, int warps, bool staged, int ctas,
                       cudaStream_t s) {
  return dtype == LBGEMM_BF16 ? launch_mode<__nv_bfloat16, MODE>(p, warps, staged, ctas, s)
                              : launch_mode<__half, MODE>(p, warps, staged, ctas, s);
}

}  // namespace

// Up to 8 tokens, where they fit shared memory beside the ring.  Rows of more than 8192 go to
// tiles where those cut k for themselves (with row tiles for at most half of the SMs: up to
// 9728 rows).  Measured, rows against tiles, in graphs over weights beyond L2:
//   tokens x rows x k       rows   tiles, us
//   1 x 4096 x 11008        13.8   13.1   (from L2 1, 4, 8 tokens: 13.3, 13.7, 15.0 and 11.9)
//   1, 4 x 4096 x 14336     16.2, 15.9   14.6
//   1 x 8192 x 28672        46.9   38.2
//   1, 4 x 9728 x 12288     21.9, 22.0   20.6, 20.4
//   1, 4 x 11008 x 12288    25.5, 25.0   30.2, 29.9
//   1 x 16384 x 16384       42.7   59.2
//   1 x 19456 x 28672       75.7   71.1
//   1, 4 x 32768 x 8320     40.5, 40.3   51.1, 46.6
//   1 x 128000 x 4096       66     94
// and from L2 1, 4 and 8 x 11008 x 4096 10.9, 11.2, 12.1 and 12.6; 1 x 1024 x 1024 4.5 and 6.3.
// Two blocks of 8 columns a pass: 12 x 4096 x 11008 16.5 us, tiles 12.2.
static bool linear_params(const W4LinearParams& l, int sm_count, W4RowsParams* p) {
  if (l.m > 8 || (l.k > 8192 && 2 * ((l.n + 127) / 128) <= sm_count)) return false;
  p->n = l.n;
  p->k = (int)l.k;
  p->group = l.group;
  p->x = l.x;
  p->x_stride = l.x_stride;
  p->w = l.w;
  p->y = l.y;
  p->y_stride = l.y_stride;
  p->picks = (int)l.m;
  p->status = l.status;
  return cut_linear(*p, sm_count);
}

bool w4_rows_take_linear(const W4LinearParams& l, int sm_count) {
  W4RowsParams p;
  return linear_params(l, sm_count, &p);
}

cudaError_t launch_w4_rows_linear(int dtype, const W4LinearParams& l, int sm_count, int* launches,
                                  cudaStream_t s) {
  W4RowsParams p;
  if (!linear_params(l, sm_count, &p)) return cudaErrorInvalidValue;
  const cudaError_t e =
      launch_any<kLinear>(dtype, p, kAllWarps, true, ctas_for(p.n, sm_count), s);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

// An expert's weights stream once for every 8 of its picks; 16 columns a pass were no
// faster (40 tokens, 6 of 64 experts of 2048 / 1024: 90 against 86 us).  Tiles cost more for
// few picks, but no more for many.  Measured, rows against tiles: 24, 32 and 64 tokens, 6 of
// 64 experts: 72, 80, 104 and 77 us; 16 and 32, 2 of 8 experts of 4096 / 2048: 43, 61 and
// 45; 32, 2 of 8 of 2048 / 1024: 24 and 23; 24 to one of those: 15 and 21.
bool w4_rows_take_moe(const MoeParams& m, int sm_count) {
  const int64_t picks = m.tokens * m.top_k;
  const int ctas = ctas_for(m.hidden, sm_count);
  // (runs are counted in 32 bits)
  return picks <= 2 * (int64_t)m.experts + 32 && picks <= kRowsMaxPicks &&
         (m.hidden + ctas - 1) / ctas * picks <= kRowsMaxValues &&
         picks * std::max<int64_t>(2 * (int64_t)m.inter, m.hidden) < INT32_MAX;
}

cudaError_t launch_w4_rows_moe(int dtype, const MoeParams& m, void* h, int sm_count,
                               int* launches, cudaStream_t s) {
  W4RowsParams p;
  p.n = 2 * (int64_t)m.inter;
  p.k = m.hidden;
  p.group = m.group;
  p.x = m.x;
  p.x_stride = m.x_stride;
  p.w = m.up;
  p.y = h;
  p.y_stride = m.inter;
  p.picks = (int)(m.tokens * m.top_k);
  p.top_k = m.top_k;
  p.experts = m.experts;
  p.ids = m.ids;
  p.weights = m.weights;
  p.status = m.status;
  const int warps = p.picks <= kFewPicks ? kFewWarps : kAllWarps;
  bool staged = cut_experts(p, warps, (int)m.tokens, 0);
  cudaError_t e = launch_any<kUp>(dtype, p, warps, staged, sm_count, s);
  if (e != cudaSuccess) return e;
  *launches += 1;
  p.n = m.hidden;
  p.k = m.inter;
  p.x = h;
  p.x_stride = m.inter;
  p.w = m.down;
  p.y = m.y;
  p.y_stride = m.y_stride;
  const int ctas = ctas_for(m.hidden, sm_count);
  p.rows_each = m.hidden / ctas;
  p.rows_more = m.hidden % ctas;
  staged = cut_experts(p, warps, p.picks, (p.rows_each + (p.rows_more > 0)) * p.picks);
  e = launch_any<kDown>(dtype, p, warps, staged, ctas, s);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

}  // namespace lbg
