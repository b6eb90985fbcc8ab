// attn_api.cu -- the C ABI of the attention operators (include/lbgemm.h):
// argument checks, scratch and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "api_checks.h"
#include "attn.h"
#include "lbgemm.h"

namespace {

using namespace lbg;

std::mutex g_attn_mu;  // the attention operators' scratch

// A [tokens, heads, dim] tensor given by pointer and token stride.
lbgemm_status check_tensor(const char* name, const void* p, int64_t stride, int64_t tokens,
                           int64_t heads, int64_t dim, int dtype) {
  if (heads == 0 || tokens == 0) return LBGEMM_OK;
  if (!p) return bad(LBGEMM_ERR_INVALID_ARG, "%s is a null pointer", name);
  if (stride > kMaxStride || (tokens > 1 && stride < heads * dim))
    return bad(LBGEMM_ERR_INVALID_ARG, "%s: token stride %lld does not hold %lld heads of %lld",
               name, (long long)stride, (long long)heads, (long long)dim);
  if (!aligned(p, 16) || (tokens > 1 && stride * elem_size(dtype) % 16))
    return bad(LBGEMM_ERR_ALIGNMENT, "%s: pointer and token stride must be 16-byte aligned", name);
  return LBGEMM_OK;
}

lbgemm_status check_cache(int64_t heads, int64_t dim, const void* cache, int64_t pages,
                          int64_t page_size) {
  if (heads < 1 || heads > 65535)
    return bad(LBGEMM_ERR_INVALID_ARG, "%lld key-value heads", (long long)heads);
  if (dim != 64 && dim != 128)
    return bad(LBGEMM_ERR_INVALID_ARG, "the 4-bit cache has head_dim 64 or 128 (got %lld)",
               (long long)dim);
  if (page_size < 16 || page_size % 16 || page_size > (int64_t(1) << 24))
    return bad(LBGEMM_ERR_INVALID_ARG, "page_size must be a multiple of 16 up to 2^24 (got %lld)",
               (long long)page_size);
  if (pages < 1 || pages > INT32_MAX)
    return bad(LBGEMM_ERR_INVALID_ARG, "%lld pages", (long long)pages);
  if (!cache) return bad(LBGEMM_ERR_INVALID_ARG, "the cache is a null pointer");
  if (!aligned(cache, 16)) return bad(LBGEMM_ERR_ALIGNMENT, "the cache must be 16-byte aligned");
  return LBGEMM_OK;
}

lbgemm_status check_norm_rope(int dtype, int64_t tokens, int64_t heads_q, int64_t heads_k,
                              int64_t dim, float eps, const void* wq, const void* wk,
                              const float* cosines, const float* sines, int64_t table_rows,
                              const int64_t* positions, int64_t rot) {
  lbgemm_status st = check_dtype(dtype, true);
  if (st != LBGEMM_OK) return st;
  if (tokens < 0 || tokens > INT32_MAX)
    return bad(LBGEMM_ERR_INVALID_ARG, "%lld tokens", (long long)tokens);
  if (heads_q < 0 || heads_k < 0 || heads_q + heads_k < 1 || heads_q + heads_k > 65535)
    return bad(LBGEMM_ERR_INVALID_ARG, "%lld query and %lld key heads", (long long)heads_q,
               (long long)heads_k);
  if (dim < 8 || dim > 512 || dim % 8)
    return bad(LBGEMM_ERR_INVALID_ARG, "head_dim must be a multiple of 8 up to 512 (got %lld)",
               (long long)dim);
  if (rot < 0 || rot > dim || rot % 2)
    return bad(LBGEMM_ERR_INVALID_ARG, "rot_dim must be even and at most head_dim (got %lld)",
               (long long)rot);
  if (!(eps >= 0.0f) || std::isinf(eps)) return bad(LBGEMM_ERR_INVALID_ARG, "eps must be >= 0");
  if (!aligned(wq, 16) || !aligned(wk, 16))
    return bad(LBGEMM_ERR_ALIGNMENT, "norm weights must be 16-byte aligned");
  if (tokens > 0 && rot > 0) {
    if (!cosines || !sines || !positions)
      return bad(LBGEMM_ERR_INVALID_ARG, "rotation needs cosines, sines and positions");
    if (table_rows < 1) return bad(LBGEMM_ERR_INVALID_ARG, "table_rows must be >= 1");
    if (!aligned(cosines, 16) || !aligned(sines, 16) || !aligned(positions, 8))
      return bad(LBGEMM_ERR_ALIGNMENT, "the rotation tables must be 16-byte aligned");
  }
  return LBGEMM_OK;
}

}  // namespace

extern "C" {

lbgemm_status lbgemm_qk_norm_rope(int dtype, int64_t tokens, int64_t heads_q, int64_t heads_k,
                                  int64_t head_dim, const void* Q, int64_t q_stride, const void* K,
                                  int64_t k_stride, const void* wq, const void* wk, float eps,
                                  const float* cosines, const float* sines, int64_t table_rows,
                                  const int64_t* positions, int64_t rot_dim, int interleaved,
                                  void* Q_out, int64_t q_out_stride, void* K_out,
                                  int64_t k_out_stride, void* stream) {
  try {
    lbgemm_status st = check_norm_rope(dtype, tokens, heads_q, heads_k, head_dim, eps, wq, wk,
                                       cosines, sines, table_rows, positions, rot_dim);
    if (st == LBGEMM_OK) st = check_tensor("Q", Q, q_stride, tokens, heads_q, head_dim, dtype);
    if (st == LBGEMM_OK) st = check_tensor("K", K, k_stride, tokens, heads_k, head_dim, dtype);
    if (st == LBGEMM_OK)
      st = check_tensor("Q_out", Q_out, q_out_stride, tokens, heads_q, head_dim, dtype);
    if (st == LBGEMM_OK)
      st = check_tensor("K_out", K_out, k_out_stride, tokens, heads_k, head_dim, dtype);
    if (st != LBGEMM_OK || tokens == 0) return st;
    CallDevice dev;
    st = call_device(&dev);
    if (st != LBGEMM_OK) return st;
    NormRopeParams p;
    p.side[0] = {Q, wq, Q, Q_out, nullptr, q_stride, q_stride, q_out_stride};
    p.side[1] = {K, wk, K, K_out, nullptr, k_stride, k_stride, k_out_stride};
    p.heads[0] = (int)heads_q;
    p.heads[1] = (int)heads_k;
    p.tokens = tokens;
    p.dim = (int)head_dim;
    p.rot = (int)rot_dim;
    p.interleaved = interleaved != 0;
    p.eps = eps;
    p.cosines = cosines;
    p.sines = sines;
    p.table_rows = table_rows;
    p.positions = positions;
    p.status = dev.status;
    cudaError_t e = launch_norm_rope(dtype, p, dev.sm_count, as_stream(stream));
    if (e != cudaSuccess) return report_cuda_error(e, "norm and rotation launch");
    count_launches(1);
    return LBGEMM_OK;
  } catch (...) {
    return report_error(LBGEMM_ERR_CUDA, "internal error");
  }
}

lbgemm_status lbgemm_qk_norm_rope_backward(
    int dtype, int64_t tokens, int64_t heads_q, int64_t heads_k, int64_t head_dim,
    const void* dQ_out, int64_t dq_out_stride, const void* dK_out, int64_t dk_out_stride,
    const void* Q, int64_t q_stride, const void* K, int64_t k_stride, const void* wq,
    const void* wk, float eps, const float* cosines, const float* sines, int64_t table_rows,
    const int64_t* positions, int64_t rot_dim, int interleaved, void* dQ, int64_t dq_stride,
    void* dK, int64_t dk_stride, float* dwq, float* dwk, void* stream) {
  try {
    lbgemm_status st = check_norm_rope(dtype, tokens, heads_q, heads_k, head_dim, eps, wq, wk,
                                       cosines, sines, table_rows, positions, rot_dim);
    if (st == LBGEMM_OK)
      st = check_tensor("dQ_out", dQ_out, dq_out_stride, tokens, heads_q, head_dim, dtype);
    if (st == LBGEMM_OK)
      st = check_tensor("dK_out", dK_out, dk_out_stride, tokens, heads_k, head_dim, dtype);
    // the forward input is read for a norm only
    if (st == LBGEMM_OK && wq)
      st = check_tensor("Q", Q, q_stride, tokens, heads_q, head_dim, dtype);
    if (st == LBGEMM_OK && wk)
      st = check_tensor("K", K, k_stride, tokens, heads_k, head_dim, dtype);
    if (st == LBGEMM_OK) st = check_tensor("dQ", dQ, dq_stride, tokens, heads_q, head_dim, dtype);
    if (st == LBGEMM_OK) st = check_tensor("dK", dK, dk_stride, tokens, heads_k, head_dim, dtype);
    if (st != LBGEMM_OK) return st;
    if ((wq != nullptr) != (dwq != nullptr) || (wk != nullptr) != (dwk != nullptr))
      return bad(LBGEMM_ERR_INVALID_ARG, "dwq and dwk are given exactly where wq and wk are");
    if (!aligned(dwq, 16) || !aligned(dwk, 16))
      return bad(LBGEMM_ERR_ALIGNMENT, "dwq and dwk must be 16-byte aligned");
    if (tokens == 0 && !wq && !wk) return LBGEMM_OK;
    CallDevice dev;
    st = call_device(&dev);
    if (st != LBGEMM_OK) return st;
    NormRopeParams p;
    p.side[0] = {Q, wq, dQ_out, dQ, dwq, q_stride, dq_out_stride, dq_stride};
    p.side[1] = {K, wk, dK_out, dK, dwk, k_stride, dk_out_stride, dk_stride};
    p.heads[0] = (int)heads_q;
    p.heads[1] = (int)heads_k;
    p.tokens = tokens;
    p.dim = (int)head_dim;
    p.rot = (int)rot_dim;
    p.interleaved = interleaved != 0;
    p.eps = eps;
    p.cosines = cosines;
    p.sines = sines;
    p.table_rows = table_rows;
    p.positions = positions;
    p.status = dev.status;
    cudaStream_t s = as_stream(stream);
    int launches = 0;
    const size_t bytes = norm_rope_scratch(dtype, p, dev.sm_count);
    cudaError_t e;
    if (bytes == 0) {
      e = launch_norm_rope_backward(dtype, p, dev.sm_count, nullptr, &launches, s);
      if (e != cudaSuccess) return report_cuda_error(e, "norm and rotation backward launch");
    } else {
      std::lock_guard<std::mutex> lock(g_attn_mu);
      void* scratch = nullptr;
      st = attn_scratch_acquire(dev, bytes, s, &scratch);
      if (st != LBGEMM_OK) return st;
      e = launch_norm_rope_backward(dtype, p, dev.sm_count, static_cast<float*>(scratch),
                                    &launches, s);
      st = attn_scratch_release(dev, s, scratch);
      if (e != cudaSuccess) return report_cuda_error(e, "norm and rotation backward launch");
      if (st != LBGEMM_OK) return st;
    }
    count_launches(launches);
    return LBGEMM_OK;
  } catch (...) {
    return report_error(LBGEMM_ERR_CUDA, "internal error");
  }
}

size_t lbgemm_kv4_page_bytes(int64_t heads, int64_t head_dim, int64_t page_size) {
  if (heads < 1 || heads > 65535 || (head_dim != 64 && head_dim != 128) || page_size < 16 ||
      page_size % 16 || page_size > (int64_t(1) << 24))
    return 0;
  return (size_t)(heads * kv4_block_bytes(head_dim, page_size));
}

static lbgemm_status kv4_copy(bool write, int dtype, int64_t tokens, int64_t heads,
                              int64_t head_dim, void* K, int64_t k_stride, void* V,
                              int64_t v_stride, const int64_t* slots, void* cache, int64_t pages,
                              int64_t page_size, void* stream) {
  lbgemm_status st = check_dtype(dtype, true);
  if (st != LBGEMM_OK) return st;
  if (tokens < 0 || tokens > INT32_MAX)
    return bad(LBGEMM_ERR_INVALID_ARG, "%lld tokens", (long long)tokens);
  st = check_cache(heads, head_dim, cache, pages, page_size);
  if (st == LBGEMM_OK) st = check_tensor("K", K, k_stride, tokens, heads, head_dim, dtype);
  if (st == LBGEMM_OK) st = check_tensor("V", V, v_stride, tokens, heads, head_dim, dtype);
  if (st != LBGEMM_OK || tokens == 0) return st;
  if (!slots) return bad(LBGEMM_ERR_INVALID_ARG, "slots is a null pointer");
  if (!aligned(slots, 8)) return bad(LBGEMM_ERR_ALIGNMENT, "slots must be 8-byte aligned");
  CallDevice dev;
  st = call_device(&dev);
  if (st != LBGEMM_OK) return st;
  Kv4CopyParams p;
  p.cache = {static_cast<uint8_t*>(cache), pages, page_size, (int)heads, (int)head_dim};
  p.tokens = tokens;
  p.k = K;
  p.v = V;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = slots;
  p.status = dev.status;
  cudaError_t e = write ? launch_kv4_write(dtype, p, as_stream(stream))
                        : launch_kv4_read(dtype, p, as_stream(stream));
  if (e != cudaSuccess) return report_cuda_error(e, write ? "cache write launch" : "cache read launch");
  count_launches(1);
  return LBGEMM_OK;
}

lbgemm_status lbgemm_kv4_write(int dtype, int64_t tokens, int64_t heads, int64_t head_dim,
                               const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                               const int64_t* slots, void* cache, int64_t pages,
                               int64_t page_size, void* stream) {
  try {
    return kv4_copy(true, dtype, tokens, heads, head_dim, const_cast<void*>(K), k_stride,
                    const_cast<void*>(V), v_stride, slots, cache, pages, page_size, stream);
  } catch (...) {
    return report_error(LBGEMM_ERR_CUDA, "internal error");
  }
}

lbgemm_status lbgemm_kv4_read(int dtype, int64_t tokens, int64_t heads, int64_t head_dim,
                              const int64_t* slots, const void* cache, int64_t pages,
                              int64_t page_size, void* K, int64_t k_stride, void* V,
                              int64_t v_stride, void* stream) {
  try {
    return kv4_copy(false, dtype, tokens, heads, head_dim, K, k_stride, V, v_stride, slots,
                    const_cast<void*>(cache), pages, page_size, stream);
  } catch (...) {
    return report_error(LBGEMM_ERR_CUDA, "internal error");
  }
}

lbgemm_status lbgemm_kv4_attention(int dtype, int64_t batch, int64_t total_q, int64_t max_q,
                                   int64_t heads_q, int64_t heads_kv, int64_t head_dim,
                                   const void* Q, int64_t q_stride, const int32_t* cu_q,
                                   const void* cache, int64_t pages, int64_t page_size,
                                   const int32_t* page_table, int64_t table_width,
                                   const int32_t* kv_lens, int64_t max_kv, float scale, int causal,
                                   int64_t window, void* O, float* lse, void* stream) {
  try {
    lbgemm_status st = check_dtype(dtype, false);
    if (st != LBGEMM_OK) return st;
    if (batch < 0 || batch > 65535 || total_q < 0 || total_q > INT32_MAX || max_q < 0 ||
        max_q > total_q)
      return bad(LBGEMM_ERR_INVALID_ARG, "batch %lld, total_q %lld, max_q %lld", (long long)batch,
                 (long long)total_q, (long long)max_q);
    st = check_cache(heads_kv, head_dim, cache, pages, page_size);
    if (st != LBGEMM_OK) return st;
    if (heads_q < heads_kv || heads_q % heads_kv || heads_q > 65535)
      return bad(LBGEMM_ERR_INVALID_ARG, "%lld query heads do not share %lld key-value heads",
                 (long long)heads_q, (long long)heads_kv);
    if (max_q * heads_q / heads_kv > INT32_MAX)
      return bad(LBGEMM_ERR_INVALID_ARG, "max_q times the heads of a group must be below 2^31");
    // (the kernels count tiles in 32 bits)
    if (kv4_attention_tiles(batch, max_q, heads_q / heads_kv) > INT32_MAX)
      return bad(LBGEMM_ERR_INVALID_ARG, "%lld sequences of up to %lld rows are too many tiles",
                 (long long)batch, (long long)max_q);
    if (max_kv < 0 || max_kv > (int64_t(1) << 30) || table_width < 0 || table_width > INT32_MAX)
      return bad(LBGEMM_ERR_INVALID_ARG, "max_kv %lld (at most 2^30), table_width %lld",
                 (long long)max_kv, (long long)table_width);
    if (max_kv > table_width * page_size)
      return bad(LBGEMM_ERR_INVALID_ARG, "max_kv %lld exceeds the %lld tokens of a page-table row",
                 (long long)max_kv, (long long)(table_width * page_size));
    if (window < 0 || (window > 0 && !causal))
      return bad(LBGEMM_ERR_INVALID_ARG, "a window is >= 0 and needs the causal mask");
    if (!std::isfinite(scale)) return bad(LBGEMM_ERR_INVALID_ARG, "scale must be finite");
    st = check_tensor("Q", Q, q_stride, total_q, heads_q, head_dim, dtype);
    if (st == LBGEMM_OK)
      st = check_tensor("O", O, heads_q * head_dim, total_q, heads_q, head_dim, dtype);
    if (st != LBGEMM_OK || total_q == 0) return st;
    if (batch == 0 || max_q == 0)
      return bad(LBGEMM_ERR_INVALID_ARG, "batch and max_q must be >= 1 when there are queries");
    if (!cu_q || !kv_lens || (!page_table && max_kv > 0))
      return bad(LBGEMM_ERR_INVALID_ARG, "cu_q, kv_lens or page_table is a null pointer");
    if (!aligned(cu_q, 4) || !aligned(kv_lens, 4) || !aligned(page_table, 4) || !aligned(lse, 4))
      return bad(LBGEMM_ERR_ALIGNMENT, "cu_q, kv_lens, page_table and lse must be 4-byte aligned");
    CallDevice dev;
    st = call_device(&dev);
    if (st != LBGEMM_OK) return st;
    Kv4AttnParams p;
    p.cache = {const_cast<uint8_t*>(static_cast<const uint8_t*>(cache)), pages, page_size,
               (int)heads_kv, (int)head_dim};
    p.batch = (int)batch;
    p.total_q = (int)total_q;
    p.max_q = (int)max_q;
    p.heads_q = (int)heads_q;
    p.group = (int)(heads_q / heads_kv);
    p.q = Q;
    p.q_stride = q_stride;
    p.cu_q = cu_q;
    p.page_table = page_table;
    p.kv_lens = kv_lens;
    p.table_width = table_width;
    p.max_kv = (int)max_kv;
    p.causal = causal != 0;
    p.window = (int)(window < (int64_t(1) << 30) ? window : (int64_t(1) << 30));
    p.scale = scale;
    p.o = O;
    p.lse = lse;
    p.status = dev.status;
    int launches = 0;
    cudaStream_t s = as_stream(stream);
    cudaError_t e;
    const size_t bytes = kv4_attention_plan(&p, dev.sm_count);
    if (bytes == 0) {
      e = launch_kv4_attention(dtype, p, &launches, s);
      if (e != cudaSuccess) return report_cuda_error(e, "attention launch");
    } else {
      std::lock_guard<std::mutex> lock(g_attn_mu);
      void* scratch = nullptr;
      st = attn_scratch_acquire(dev, bytes, s, &scratch);
      if (st != LBGEMM_OK) return st;
      kv4_attention_scratch(&p, scratch);
      e = launch_kv4_attention(dtype, p, &launches, s);
      st = attn_scratch_release(dev, s, scratch);
      if (e != cudaSuccess) return report_cuda_error(e, "attention launch");
      if (st != LBGEMM_OK) return st;
    }
    count_launches(launches);
    return LBGEMM_OK;
  } catch (...) {
    return report_error(LBGEMM_ERR_CUDA, "internal error");
  }
}

}  // extern "C"
