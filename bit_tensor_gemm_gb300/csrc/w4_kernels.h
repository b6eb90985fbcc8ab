// w4_kernels.h -- the kernels behind the 4-bit products (w4_rows.cu for few
// tokens) and how a call chooses among them (w4.cu).
#pragma once
#include <cuda.h>

#include "ffn.h"

namespace lbg {

// ---- few tokens -------------------------------------------------------------------------
constexpr int kRowsMaxPicks = 512, kRowsMaxExperts = 1024;
constexpr int kRowsMaxValues = 6 * 1024;  // floats that a CTA keeps of the picks' outputs
struct W4RowsParams {
  int64_t n = 0;  // rows of a matrix (of one expert)
  int k = 0, group = 0;
  const void* x = nullptr;
  int64_t x_stride = 0;
  W4 w;
  void* y = nullptr;
  int64_t y_stride = 0;
  int picks = 0;  // tokens times choices (linear: tokens)
  int top_k = 1, experts = 1;
  const int32_t* ids = nullptr;
  const float* weights = nullptr;
  int* status = nullptr;
  // How the launch cuts the call: rows a CTA (rows_more CTAs have one more), steps of a
  // row, tiles of a round at most, steps that codes are copied ahead; and where things lie
  // in shared memory.
  int rows_each = 0, rows_more = 0, steps = 1, batch = 1, depth = 2;
  int at_shares = 0, at_values = 0, at_tokens = 0, bytes = 0;
};
bool w4_rows_take_linear(const W4LinearParams& l, int sm_count);
cudaError_t launch_w4_rows_linear(int dtype, const W4LinearParams& l, int sm_count, int* launches,
                                  cudaStream_t s);
bool w4_rows_take_moe(const MoeParams& m, int sm_count);
// h: [tokens * top_k][inter] of dtype
cudaError_t launch_w4_rows_moe(int dtype, const MoeParams& m, void* h, int sm_count, int* launches,
                               cudaStream_t s);

// ---- many tokens --------------------------------------------------------------------------
constexpr int kTilesMaxExperts = 1024;
struct W4TilesParams {
  int64_t n = 0;  // rows of a matrix (of one expert)
  int k = 0, group = 0;
  const uint8_t* scales = nullptr;
  const float* row_scales = nullptr;
  void* out = nullptr;  // linear: Y; up: h; down: fp32 [pick][n]
  int64_t out_stride = 0;
  bool vector = false;  // (linear) Y's rows are 16-byte aligned
  int m = 0;  // tokens (linear) or picks
  int experts = 1;
  const int* offsets = nullptr;  // [experts + 1]
  // The cut: blocks of tokens (linear), tiles of rows, slices of k; tiles that are not cut
  // along k, parts of the others and a part's slices, and where their shares go.
  int blocks = 0, row_tiles = 0, slices = 0, whole = 0, parts = 1, part_slices = 0;
  float* shares = nullptr;  // fp32 [cut tile][part][token][row] of a tile's
  int* status = nullptr;
};
struct MoeSort {
  const int32_t* ids = nullptr;
  int picks = 0, top_k = 1, experts = 1, piece = 0, pieces = 0;
  int *counts = nullptr, *offsets = nullptr, *token_of = nullptr, *pos_of = nullptr;
  int* status = nullptr;
};
size_t w4_tiles_linear_scratch(const W4LinearParams& l, int sm_count);
cudaError_t launch_w4_tiles_linear(int dtype, const W4LinearParams& l, void* scratch, int sm_count,
                                   int* launches, cudaStream_t s);
size_t w4_tiles_moe_scratch(const MoeParams& m);
cudaError_t launch_w4_tiles_moe(int dtype, const MoeParams& m, void* scratch, int sm_count,
                                int* launches, cudaStream_t s);

// A 2D tensor map (api.cu): rows of `width` elements of a dtype (or bytes) `stride` bytes
// apart, boxes of box_width x box_rows, swizzled by 64 or 128 bytes.
constexpr int LBGEMM_MAP_U8 = -1;
bool encode_map(CUtensorMap* map, int dtype, const void* base, int64_t width, int64_t rows,
                int64_t stride, int box_width, int box_rows, int swizzle);

}  // namespace lbg
