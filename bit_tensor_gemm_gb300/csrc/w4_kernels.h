// w4_kernels.h -- the kernels behind the 4-bit products (w4_rows.cu for few
// tokens) and how a call chooses among them (w4.cu).
#pragma once
#include "ffn.h"

namespace lbg {

// ---- few tokens -------------------------------------------------------------------------
constexpr int kRowsMaxPicks = 512, kRowsMaxExperts = 1024;
constexpr int kRowsMaxValues = 12 * 1024;  // floats that a CTA keeps of the picks' outputs
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
  // How the launch cuts the call: rows a CTA (rows_more CTAs have one more), pieces of
  // k and their steps, tiles of a round, steps that codes are copied ahead; columns as
  // a power of two; and where things lie in shared memory.
  int rows_each = 0, rows_more = 0, chunks = 1, steps = 1, batch = 1, depth = 2;
  int log_columns = 0;
  int at_shares = 0, at_values = 0, at_tokens = 0, bytes = 0;
};
bool w4_rows_take_linear(const W4LinearParams& l, int sm_count);
cudaError_t launch_w4_rows_linear(int dtype, const W4LinearParams& l, int sm_count, cudaStream_t s);
bool w4_rows_take_moe(const MoeParams& m, int sm_count);
// h: [tokens * top_k][inter] of dtype
cudaError_t launch_w4_rows_moe(int dtype, const MoeParams& m, void* h, int sm_count, int* launches,
                               cudaStream_t s);

}  // namespace lbg
