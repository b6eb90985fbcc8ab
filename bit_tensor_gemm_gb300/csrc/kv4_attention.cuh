// kv4_attention.cuh -- what the kernels of attention over the 4-bit cache
// share: the rows and tokens of a unit of work, and where results go.
#pragma once
#include "attn.h"
#include "attn_common.cuh"

namespace lbg {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A tile of query rows of one sequence, and the tokens [first, last) that any
// of its rows sees; `base` is `first` rounded down to a multiple of 32, where
// its chunks start.
struct RowTile {
  int q0, n, len;        // the sequence's first query row, its queries, its tokens
  int r0, rows;          // the tile's first row and its rows (0: nothing to do)
  int first, last, base, chunks;
};

__device__ __forceinline__ RowTile row_tile(const Kv4AttnParams& p, int b, int tile) {
  RowTile t;
  t.q0 = p.cu_q[b];
  t.n = p.cu_q[b + 1] - t.q0;
  t.len = p.kv_lens[b];
  if (t.q0 < 0 || t.n < 0 || t.q0 > p.total_q - t.n || t.n > p.max_q || t.len < 0 ||
      t.len > p.max_kv) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
    if (t.q0 < 0 || t.n < 0 || t.q0 > p.total_q - t.n || t.n > p.max_q) t.n = 0;
    t.len = min(max(t.len, 0), p.max_kv);
  }
  t.r0 = tile * p.tile_rows;
  t.rows = min(p.tile_rows, t.n * p.group - t.r0);
  if (t.rows <= 0) {
    t.rows = t.first = t.last = t.base = t.chunks = 0;
    return t;
  }
  t.first = 0;
  t.last = t.len;
  if (p.causal) {
    const int before = t.len - t.n;  // position of the first query
    const int i0 = (int)p.by_group((uint32_t)t.r0);
    const int i1 = (int)p.by_group((uint32_t)(t.r0 + t.rows - 1));
    t.last = min(t.len, before + i1 + 1);
    if (p.window) t.first = max(0, before + i0 - p.window + 1);
  }
  if (t.last <= t.first) t.first = t.last = 0;
  t.base = t.first & ~31;
  t.chunks = max(1, (t.last - t.base + p.chunk - 1) / p.chunk);
  return t;
}

// One past the last token that a row at query i of the sequence sees (may be
// negative), and the first one.
__device__ __forceinline__ int last_seen(const Kv4AttnParams& p, const RowTile& t, int i) {
  return p.causal ? t.len - t.n + i + 1 : t.len;
}
__device__ __forceinline__ int first_seen(const Kv4AttnParams& p, int last) {
  return p.window ? last - p.window : 0;
}

__device__ __forceinline__ int64_t unit_of(const Kv4AttnParams& p, int b, int head, int tile,
                                           int chunk) {
  return (((int64_t)b * p.cache.heads + head) * p.row_tiles + tile) * p.max_chunks + chunk;
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
