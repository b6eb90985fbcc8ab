// w4_rows.cu -- products with 4-bit weights for few tokens: the weights stream
// through warp MMAs once for 8 or 16 columns (tokens).
//
//   linear  Y[m][n] = row_scale[n] * sum_k X[m][k] * (code * scale)[n][k]
//   up      h[pick][i] = silu(gate) * up, for every pick (token, expert)
//   down    y[t] = sum over a token's picks, in order, of weight * (Down h[pick])
//
// Bound by the weights' stream from HBM (about 0.53 bytes a weight), and close
// behind it by issue slots: a word of eight codes takes twelve operations to
// become halves (w4_codes.cuh).  So the codes go to the MMA's 16-row side, which
// has no row to spare, and the tokens to its 8-column side.
//
// A CTA an SM, 24 warps (16 for 16 columns).  CTAs take equal runs of weight rows: of the rows of all
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
// read them.  Where they do not fit, the linear layer gives parts of k to CTAs of their
// own (whose sums a second kernel adds), or takes k in pieces; the experts read them
// through L1 then, at 2 conflicts a column and load.
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

// What a CTA knows of the picks: experts with a pick ("segments", of up to 8 NB
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

// kWarps: 24, or the 16 that 16 columns leave registers for.  A mixture of few picks
// takes 12 and half of the shared memory, so that the CTAs of `down` stand beside those
// of `up`: they look up their picks and copy their first codes while `up` runs.
__host__ __device__ constexpr int warps_for(int nb) { return nb == 1 ? 24 : 16; }
constexpr int kFewWarps = 12, kFewPicks = 16;
// Tiles of 8 columns in a round (24 tokens to 64 experts, 49 and 58 tiles a CTA: 68.3 us,
// 69.7 with room for 48; no gain from 80).
constexpr int kShares = 64;

template <typename T, int MODE, int NB, bool STAGED, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps == kFewWarps ? 2 : 1)
    w4_rows_kernel(const W4RowsParams p) {
  constexpr int kThreads = 32 * kWarps;
  constexpr int COLS = 8 * NB, SHARE = 16 * COLS;  // columns; numbers of a tile
  extern __shared__ __align__(128) uint8_t smem[];
  float* shares = reinterpret_cast<float*>(smem + p.at_shares);  // [batch + kWarps][SHARE]
  // down: the picks' outputs [rows][picks]; linear: sums between pieces of k [rows][COLS]
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
  // (linear: CTAs by parts of k, then by rows)
  const int part = MODE == kLinear ? blockIdx.x / p.row_ctas : 0;
  const int cta = MODE == kLinear ? blockIdx.x - part * p.row_ctas : blockIdx.x;
  const int first_step = part * p.steps;  // (one piece of k where there are parts)
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

  // ---- rounds: pieces of k by batches of tiles ----
  const int steps = p.steps;  // of a tile in a piece
  // tiles of a round: as many in each, as few rounds as there is room for
  const int batches = (run.tiles + p.batch - 1) / p.batch;
  const int TB = batches > 1 ? (run.tiles + batches - 1) / batches : run.tiles;
  const int rounds = batches * p.chunks;

  // A place in this warp's part of a round.
  struct Place {
    int round, chunk, batch, tile, j, left;
  };
  auto begin = [&](Place& x) {
    const int total = min(TB, run.tiles - x.batch * TB) * steps;
    const int each = total / kWarps, more = total - each * kWarps;
    const int first = warp * each + min(warp, more);
    x.left = each + (warp < more);
    x.tile = first / steps;
    x.j = first - x.tile * steps;
    x.tile += x.batch * TB;
  };
  auto next_round = [&](Place& x) {
    ++x.round;
    if (++x.batch == batches) x.batch = 0, ++x.chunk;
    if (x.round < rounds) begin(x);
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
  Place ahead = {0, 0, 0, 0, 0, 0};
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
                    128 * (first_step + ahead.chunk * steps + ahead.j);
  };
  aim_codes();
  const uint32_t ring = smem_addr(smem) + warp * p.depth * kSlotBytes + lane * 16;
  uint32_t to = ring;  // the slot that is copied to next
  const uint32_t ring_end = ring + p.depth * kSlotBytes;
  auto copy_codes = [&] {
    if (ahead.left > 0) {
      const int step = first_step + ahead.chunk * steps + ahead.j;
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
                     ((8 * (first_step + scaled.chunk * steps + scaled.j) + t) >> shift);
      if (t == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.w.row_scales + r[i]));
    }
  };
  aim_scales();
  auto load_scales = [&] {
    if (scaled.left == 0) return;
    const int step = first_step + scaled.chunk * steps + scaled.j;
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

  float acc[NB][4];
  // This lane's columns: in memory, or staged: vector v of a piece at v * pitch, its
  // 16 bytes in the order that lanes read them, so that 8 lanes of neighbouring
  // vectors meet no conflict: [half step][word][t].
  const T* column[NB];
  const uint8_t* line[NB];
  const int pitch = steps * 512 + 64;
  uint32_t from = ring;

  while (at.round < rounds) {
    if (STAGED && at.batch == 0) {
      const int pieces = steps * 32, vectors = MODE == kUp ? p.picks / p.top_k : p.picks;
      for (int v = warp; v < vectors; v += kWarps)
        for (int o = lane; o < pieces; o += 32) {
          const int at_k = (first_step + at.chunk * steps) * kStep + 8 * o;
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
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int pick = pick_of(segment, min(8 * b + g, most));
        const int v = MODE == kUp ? pick / p.top_k : pick;
        if (STAGED)
          line[b] = staged + v * pitch + 16 * t + at.j * 512;
        else
          column[b] = static_cast<const T*>(p.x) + v * p.x_stride + 32 * t + at.j * kStep;
        acc[b][0] = acc[b][1] = acc[b][2] = acc[b][3] = 0.0f;
      }
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
          uint4 x[NB][4];
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              if (STAGED)
                x[b][w] = *reinterpret_cast<const uint4*>(line[b] + h * 256 + w * 64);
              else if (at.j < whole || left_of(at.j) > 128 * h)
                x[b][w] = *reinterpret_cast<const uint4*>(column[b] + 128 * h + 8 * w);
              else
                x[b][w] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a[4], c[4];
            w4_word(w == 0 ? cl.x : w == 1 ? cl.y : w == 2 ? cl.z : cl.w, lo[h], a);
            w4_word(w == 0 ? ch.x : w == 1 ? ch.y : w == 2 ? ch.z : ch.w, hi[h], c);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              mma<T>(acc[b], a[0], c[0], a[1], c[1], x[b][w].x, x[b][w].y);
              mma<T>(acc[b], a[2], c[2], a[3], c[3], x[b][w].z, x[b][w].w);
            }
          }
        }
        // (each lane has read its own bytes of the slot: the next copy may land on it)
        copy_codes();
        from += kSlotBytes;
        if (from == ring_end) from = ring;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (STAGED)
            line[b] += 512;
          else
            column[b] += kStep;
        }
      }
      // This warp's share of the tile: in place tile + warp, which no other share of the
      // round has (along the row of steps one of both grows).
      float* s = shares + (at.tile - at.batch * TB + warp) * SHARE;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        *reinterpret_cast<float2*>(s + g * COLS + 8 * b + 2 * t) =
            make_float2(acc[b][0], acc[b][1]);
        *reinterpret_cast<float2*>(s + (g + 8) * COLS + 8 * b + 2 * t) =
            make_float2(acc[b][2], acc[b][3]);
      }
      if (at.j == steps) at.j = 0, ++at.tile;
    }
    __syncthreads();

    // ---- the round's sums ----
    const int first_tile = at.batch * TB, count = min(TB, run.tiles - first_tile);
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
              from_f32<T>(v / (1.0f + expf(-v)) * u);
        } else if (MODE == kDown) {
          values[(row - run.first_row + r) * p.picks + pick] = v * scale0;
        } else {
          // (the same lane meets an output in every piece of k)
          float* sum = values + (row - run.first_row + r) * COLS + col;
          if (at.chunk > 0) v += *sum;
          if (at.chunk + 1 < p.chunks)
            *sum = v;
          else if (p.parts > 1)
            p.part_sums[((int64_t)part * p.picks + pick) * n + row + r] = v * scale0;
          else
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

// y[m][n] = the sum of the parts of k, in order.
template <typename T>
__global__ void __launch_bounds__(256) rows_join_kernel(const W4RowsParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t total = p.picks * p.n;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / p.n, c = i - m * p.n;
    float v = 0.0f;
    for (int q = 0; q < p.parts; ++q) v += p.part_sums[q * total + i];
    static_cast<T*>(p.y)[m * p.y_stride + c] = from_f32<T>(v);
  }
}

// ---- how a launch lays out its shared memory -------------------------------------------
constexpr int kStatic = sizeof(Picks) + 4 * (kRowsMaxExperts + 1) + 256;
constexpr int kStaticLinear = 512;

// Blocks of 8 columns for so many tokens.
int blocks_of(int tokens) { return tokens <= 8 ? 1 : 2; }

// Fills in the cut of a linear layer into parts of k, each of its own CTAs; false where
// it does not fit.  A part's tokens are staged at once; only one part may take several
// pieces (of 16 steps at least: fewer are too many rounds).
bool cut_linear(W4RowsParams& p, int parts, int sm_count) {
  const int nb = blocks_of(p.picks), warps = warps_for(nb);
  p.parts = parts;
  p.row_ctas = (int)std::min<int64_t>(sm_count / parts, p.n);
  p.rows_each = (int)(p.n / p.row_ctas);
  p.rows_more = (int)(p.n % p.row_ctas);
  const int rows = p.rows_each + (p.rows_more > 0), tiles = (rows + 15) / 16;
  p.batch = std::min(tiles, kShares / nb);
  const int shares = (p.batch + warps) * nb * 512;
  const int all_steps = (p.k + kStep - 1) / kStep, steps = (all_steps + parts - 1) / parts;
  if (parts > 1 && (steps < 4 || (parts - 1) * steps >= all_steps)) return false;
  const int64_t sums = (int64_t)rows * 8 * nb * 4;
  const int room = kSmem - kStaticLinear - 2 * warps * kSlotBytes - shares;
  int64_t most = (room / p.picks - 64) / (kStep * 2);
  if (most < steps) {
    if (parts > 1) return false;
    most = ((room - sums) / p.picks - 64) / (kStep * 2);
    if (most < 16) return false;
  }
  p.chunks = (int)((steps + most - 1) / most);
  p.steps = (steps + p.chunks - 1) / p.chunks;
  const int held = p.chunks > 1 ? (int)(sums + 15) / 16 * 16 : 0;
  const int tokens = p.picks * (p.steps * kStep * 2 + 64);
  const int left = kSmem - kStaticLinear - shares - held - tokens;
  p.depth = std::min(kMaxDepth, left / (warps * kSlotBytes));
  p.at_shares = p.depth * warps * kSlotBytes;
  p.at_values = p.at_shares + shares;
  p.at_tokens = p.at_values + held;
  p.bytes = p.at_tokens + tokens;
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

template <typename T, int MODE, int NB, bool STAGED, int WARPS = warps_for(NB)>
cudaError_t launch(const W4RowsParams& p, int ctas, cudaStream_t s) {
  auto kernel = w4_rows_kernel<T, MODE, NB, STAGED, WARPS>;
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
cudaError_t launch_mode(const W4RowsParams& p, int nb, int warps, bool staged, int ctas,
                        cudaStream_t s) {
  if constexpr (MODE != kLinear) {
    if (warps == kFewWarps)
      return staged ? launch<T, MODE, 1, true, kFewWarps>(p, ctas, s)
                    : launch<T, MODE, 1, false, kFewWarps>(p, ctas, s);
    return staged ? launch<T, MODE, 1, true>(p, ctas, s) : launch<T, MODE, 1, false>(p, ctas, s);
  } else {
    return nb == 1 ? launch<T, MODE, 1, true>(p, ctas, s) : launch<T, MODE, 2, true>(p, ctas, s);
  }
}

template <int MODE>
cudaError_t launch_any(int dtype, const W4RowsParams& p, int nb, int warps, bool staged, int ctas,
                       cudaStream_t s) {
  return dtype == LBGEMM_BF16
             ? launch_mode<__nv_bfloat16, MODE>(p, nb, warps, staged, ctas, s)
             : launch_mode<__half, MODE>(p, nb, warps, staged, ctas, s);
}

int ctas_for(int64_t rows, int sm_count) {  // no CTA without a row
  return (int)std::min<int64_t>(sm_count, rows);
}

// The cut of a linear layer of up to 16 tokens (32 columns measured 31 us where the tiles
// of w4_tiles.cu take 20: the parts of k come to too many): the fewest parts of k whose tokens fit
// shared memory at once, else one part in pieces.
bool linear_params(const W4LinearParams& l, int sm_count, W4RowsParams* p) {
  if (l.m > 16) return false;
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
  for (int parts = 1; parts <= 8; ++parts)
    if (cut_linear(*p, parts, sm_count) && p->chunks == 1) return true;
  return cut_linear(*p, 1, sm_count);
}

}  // namespace

bool w4_rows_take_linear(const W4LinearParams& l, int sm_count, size_t* scratch) {
  W4RowsParams p;
  if (!linear_params(l, sm_count, &p)) return false;
  *scratch = p.parts > 1 ? (size_t)p.parts * l.m * l.n * sizeof(float) : 0;
  return true;
}

cudaError_t launch_w4_rows_linear(int dtype, const W4LinearParams& l, void* scratch, int sm_count,
                                  int* launches, cudaStream_t s) {
  W4RowsParams p;
  if (!linear_params(l, sm_count, &p)) return cudaErrorInvalidValue;
  p.part_sums = static_cast<float*>(scratch);
  const int nb = blocks_of(p.picks);
  cudaError_t e = launch_any<kLinear>(dtype, p, nb, warps_for(nb), true, p.parts * p.row_ctas, s);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (p.parts == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>((l.m * l.n + 255) / 256, 8 * sm_count));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = dtype == LBGEMM_BF16 ? cudaLaunchKernelEx(&cfg, rows_join_kernel<__nv_bfloat16>, p)
                           : cudaLaunchKernelEx(&cfg, rows_join_kernel<__half>, p);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

// An expert's weights stream once for every 8 of its picks; 16 columns a pass were no
// faster (40 tokens, 6 of 64 experts of 2048 / 1024: 90 against 86 us).  Tiles cost some 20
// us more for few picks, but no more for many.  Measured, rows against tiles: 64 tokens, 6
// of 64 experts (384 picks): 104 and 113 us; 2 of 8 experts of 4096 / 2048, 64 and 96 picks:
// 61 and 67, 76 and 67; of 2048 / 1024, 64 and 128 picks: 25 and 29, 35 and 29; one expert
// of it, 24 picks: 15 and 27.
bool w4_rows_take_moe(const MoeParams& m, int sm_count) {
  const int64_t picks = m.tokens * m.top_k;
  const int ctas = ctas_for(m.hidden, sm_count);
  // (runs are counted in 32 bits)
  return picks <= 6 * (int64_t)m.experts + 40 && picks <= kRowsMaxPicks &&
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
  const int warps = p.picks <= kFewPicks ? kFewWarps : warps_for(1);
  bool staged = cut_experts(p, warps, (int)m.tokens, 0);
  cudaError_t e = launch_any<kUp>(dtype, p, 1, warps, staged, sm_count, s);
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
  e = launch_any<kDown>(dtype, p, 1, warps, staged, ctas, s);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

}  // namespace lbg
