// kv4_attention.cuh -- what the kernels of attention over the 4-bit cache
// share: the rows and tokens of a unit of work, and where results go.
#pragma once
#include "attn.h"
#include "attn_common.cuh"

namespace lbg {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

constexpr int kStepTokens = 128;

// A tile of query rows of one sequence, and the tokens [first, last) that any
// of its rows sees; `base` is `first` rounded down to a multiple of 128, where
// its steps start.  A tile with rows has at least one step.
struct RowTile {
  int b, q0, n, len;     // the sequence, its first query row, its queries, its tokens
  int r0, rows;          // the tile's first row and its rows (0: nothing to do)
  int first, last, base, steps;
};

__device__ __forceinline__ RowTile row_tile(const Kv4AttnParams& p, int seq_tile) {
  RowTile t;
  t.b = p.row_tiles == 1 ? seq_tile : seq_tile / p.row_tiles;
  t.q0 = __ldg(p.cu_q + t.b);
  t.n = __ldg(p.cu_q + t.b + 1) - t.q0;
  t.len = __ldg(p.kv_lens + t.b);
  if (t.q0 < 0 || t.n < 0 || t.q0 > p.total_q - t.n || t.n > p.max_q || t.len < 0 ||
      t.len > p.max_kv) {
    atomicOr(p.status, kStatusBadIndex);
    if (t.q0 < 0 || t.n < 0 || t.q0 > p.total_q - t.n || t.n > p.max_q) t.n = 0;
    t.len = min(max(t.len, 0), p.max_kv);
  }
  t.r0 = (seq_tile - t.b * p.row_tiles) * p.tile_rows;
  t.rows = max(0, min(p.tile_rows, t.n * p.group - t.r0));
  t.first = 0;
  t.last = t.len;
  if (p.causal) {
    const int before = t.len - t.n;  // position of the first query
    const int i0 = (int)p.by_group((uint32_t)t.r0);
    const int i1 = (int)p.by_group((uint32_t)(t.r0 + max(t.rows, 1) - 1));
    t.last = min(t.len, before + i1 + 1);
    if (p.window) t.first = max(0, before + i0 - p.window + 1);
  }
  if (t.last <= t.first) t.first = t.last = 0;
  t.base = t.first & ~(kStepTokens - 1);
  t.steps = t.rows == 0 ? 0 : max(1, (t.last - t.base + kStepTokens - 1) / kStepTokens);
  return t;
}

// The tile to look at after `seq_tile`: past the sequence when this one, and so
// all of the sequence that follow, has no rows.  (With one long prompt beside
// thousands of single tokens nearly all tiles are such.)
__device__ __forceinline__ int tile_after(const Kv4AttnParams& p, const RowTile& t, int seq_tile) {
  return t.rows > 0 ? seq_tile + 1 : (t.b + 1) * p.row_tiles;
}

// The next tile with rows (the caller knows that there is one).
__device__ __forceinline__ RowTile next_row_tile(const Kv4AttnParams& p, int* seq_tile) {
  ++*seq_tile;
  RowTile t = row_tile(p, *seq_tile);
  while (t.rows == 0) {
    *seq_tile = tile_after(p, t, *seq_tile);
    t = row_tile(p, *seq_tile);
  }
  return t;
}

// This CTA's run of steps: it begins `off` steps into head `head` of sequence
// tile `seq_tile` and has `count` steps (0: none).
//
// A tile costs time beside its steps (its queries, its results), which is
// counted as `tile_cost` steps in front of its own: the row of steps with
// these in it is cut into runs of `per`.  `pos` is the place in that row of the
// run's first step, so that step s of the run, in its n-th tile (from 0), stands
// at pos + s + n tile_cost.
struct Run {
  int seq_tile, head, off, count;
  int64_t pos, per;
};

// Threads take equal segments of the sequence tiles, sum their steps, and the
// one whose segment holds the run's begin looks it up.  THREADS: of the block.
template <int THREADS>
__device__ __forceinline__ Run find_run(const Kv4AttnParams& p, int min_steps, int tile_cost) {
  __shared__ int64_t warp_sum[THREADS / 32];
  __shared__ Run run;
  const int tiles = p.batch * p.row_tiles;  // (below 2^31)
  const int64_t seg = ((int64_t)tiles + THREADS - 1) / THREADS;
  const int from = (int)min((int64_t)tiles, threadIdx.x * seg);
  const int to = (int)min((int64_t)tiles, from + seg);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  auto places = [&](int steps) { return steps > 0 ? steps + tile_cost : 0; };
  int64_t mine = 0;
  for (int i = from; i < to;) {
    const RowTile t = row_tile(p, i);
    mine += places(t.steps);
    i = tile_after(p, t, i);
  }
  int64_t upto = mine;  // inclusive over the warp, then the block
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += v;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int64_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const int64_t heads = p.cache.heads;
  total *= heads;
  const int64_t per = max((int64_t)min_steps, (total + gridDim.x - 1) / (int64_t)gridDim.x);
  const int64_t begin = per * blockIdx.x;
  if (begin >= total) {
    Run none = {0, 0, 0, 0, begin, per};
    return none;
  }
  int64_t at = (before + upto - mine) * heads;  // places before this thread's segment
  if (begin >= at && begin < at + mine * heads) {
    int i = from;
    RowTile t = row_tile(p, i);
    int n = t.steps, wide = places(n);
    while (begin >= at + wide * heads) {
      at += wide * heads;
      i = tile_after(p, t, i);
      t = row_tile(p, i);
      n = t.steps;
      wide = places(n);
    }
    run.seq_tile = i;
    run.head = (int)((begin - at) / wide);
    at += (int64_t)run.head * wide;
    run.off = max(0, (int)(begin - at) - tile_cost);
    run.pos = at + tile_cost + run.off;
    run.per = per;
    // its steps: what is left of this tile, then whole heads and tiles, then a part
    const int64_t end = min(begin + per, total);
    int64_t count = max((int64_t)0, min((int64_t)(n - run.off), end - run.pos));
    at += wide;
    for (int64_t left = heads - run.head - 1; at < end;) {
      if (wide > 0) {
        const int64_t whole = min(left, (end - at) / wide);
        count += whole * n;
        at += whole * wide;
        if (whole < left) {
          count += max((int64_t)0, end - at - tile_cost);
          break;
        }
      }
      i = tile_after(p, t, i);
      if (i >= tiles) break;
      t = row_tile(p, i);
      n = t.steps;
      wide = places(n);
      left = heads;
    }
    run.count = (int)count;
  }
  __syncthreads();
  return run;
}

// One past the last token that a row at query i of the sequence sees (may be
// negative), and the first one.
__device__ __forceinline__ int last_seen(const Kv4AttnParams& p, const RowTile& t, int i) {
  return p.causal ? t.len - t.n + i + 1 : t.len;
}
__device__ __forceinline__ int first_seen(const Kv4AttnParams& p, int last) {
  return p.window ? last - p.window : 0;
}

// Offset into O (in rows of dim) of row r of a tile.
__device__ __forceinline__ int64_t out_row(const Kv4AttnParams& p, const RowTile& t, int head,
                                           int r) {
  const int i = (int)p.by_group((uint32_t)r);
  return (int64_t)(t.q0 + i) * p.heads_q + head * p.group + (r - i * p.group);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace lbg
