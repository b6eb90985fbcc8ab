// w4.cu -- which kernel a call with 4-bit weights takes.
//
// Few tokens (up to 8 of a linear layer, two or three picks an expert: the rules stand in
// w4_rows.cu) stream the weights through warp MMAs; more run on tcgen05.
#include "ffn.h"
#include "w4_kernels.h"

namespace lbg {

size_t w4_linear_scratch(const W4LinearParams& p, int sm_count) {
  return w4_rows_take_linear(p, sm_count) ? 0 : w4_tiles_linear_scratch(p, sm_count);
}

cudaError_t launch_w4_linear(int dtype, const W4LinearParams& p, void* scratch, int sm_count,
                             int* launches, cudaStream_t s) {
  return w4_rows_take_linear(p, sm_count)
             ? launch_w4_rows_linear(dtype, p, sm_count, launches, s)
             : launch_w4_tiles_linear(dtype, p, scratch, sm_count, launches, s);
}

size_t moe_w4_scratch(const MoeParams& p, int sm_count) {
  return w4_rows_take_moe(p, sm_count) ? (size_t)p.tokens * p.top_k * p.inter * 2
                                       : w4_tiles_moe_scratch(p);
}

cudaError_t launch_moe_w4(int dtype, const MoeParams& p, void* scratch, int sm_count,
                          int* launches, cudaStream_t s) {
  return w4_rows_take_moe(p, sm_count)
             ? launch_w4_rows_moe(dtype, p, scratch, sm_count, launches, s)
             : launch_w4_tiles_moe(dtype, p, scratch, sm_count, launches, s);
}

}  // namespace lbg
