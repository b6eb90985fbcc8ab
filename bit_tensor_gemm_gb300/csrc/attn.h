// attn.h -- parameters and launchers of the attention operators: per-head
// norm with rotation (norm_rope.cu), the 4-bit paged cache (kv4_cache.cu) and
// attention over it (kv4_attention.cu); their C ABI is in attn_api.cu.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "lbgemm.h"

namespace lbg {

// Device status word: a kernel met an index out of range (beside the time-out
// bit of ptx.cuh).
constexpr int kStatusBadIndex = 2;

// ---- what api.cu keeps for every entry point ------------------------------------
struct CallDevice {
  int sm_count = 0;
  int* status = nullptr;
  void* state = nullptr;  // api.cu's record of the device
};
lbgemm_status report_error(lbgemm_status st, const char* message);
lbgemm_status report_cuda_error(cudaError_t e, const char* what);
lbgemm_status call_device(CallDevice* out);
// The attention operators' scratch on this device; the caller holds one lock
// from acquire to release.
lbgemm_status attn_scratch_acquire(const CallDevice& dev, size_t bytes, cudaStream_t s, void** ptr);
lbgemm_status attn_scratch_release(const CallDevice& dev, cudaStream_t s, void* ptr);
void count_launches(int n);

// ---- norm and rotation ------------------------------------------------------------
// One side (queries or keys) of a call.  x, w: the forward input; in: what the
// pass turns (x, or dy for the backward pass); out: y, or dx.
struct NormRopeSide {
  const void* x = nullptr;
  const void* w = nullptr;
  const void* in = nullptr;
  void* out = nullptr;
  float* dw = nullptr;
  int64_t x_stride = 0, in_stride = 0, out_stride = 0;
};
struct NormRopeParams {
  NormRopeSide side[2];  // queries, keys
  int heads[2] = {0, 0};
  int64_t tokens = 0;
  int dim = 0, rot = 0, interleaved = 0;
  float eps = 0.0f;
  const float *cosines = nullptr, *sines = nullptr;
  int64_t table_rows = 0;
  const int64_t* positions = nullptr;
  int* status = nullptr;
};
cudaError_t launch_norm_rope(int dtype, const NormRopeParams& p, int sm_count, cudaStream_t s);
// partial: scratch of norm_rope_scratch() bytes (unused when no weight is given).
size_t norm_rope_scratch(int dtype, const NormRopeParams& p, int sm_count);
cudaError_t launch_norm_rope_backward(int dtype, const NormRopeParams& p, int sm_count,
                                      float* partial, int* launches, cudaStream_t s);

// Division of non-negative 32-bit numbers by a number known at launch, as a
// multiplication: x / d = (x * mul) >> 32 >> shift, exact for x < 2^31.
struct FastDiv {
  uint32_t mul = 0, shift = 0, d = 1;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    if (div == 1) return;  // (mul 0: the number itself)
    while ((uint64_t(1) << shift) < div) ++shift;
    shift -= 1;
    mul = (uint32_t)(((uint64_t(1) << (32 + shift)) + div - 1) / div);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t operator()(uint32_t x) const {
    return mul ? __umulhi(x, mul) >> shift : x;
  }
#endif
};

// ---- the cache ----------------------------------------------------------------------
struct Kv4Cache {
  uint8_t* base = nullptr;
  int64_t pages = 0, page_size = 0;
  int heads = 0, dim = 0;
};
// Byte offsets inside a head's block of a page.
__host__ __device__ inline int64_t kv4_block_bytes(int64_t dim, int64_t page_size) {
  return page_size * (dim + 4);
}

struct Kv4CopyParams {  // write: K, V -> cache; read: cache -> K, V
  Kv4Cache cache;
  int64_t tokens = 0;
  void *k = nullptr, *v = nullptr;
  int64_t k_stride = 0, v_stride = 0;
  const int64_t* slots = nullptr;
  int* status = nullptr;
  // how the launch cuts the vectors
  int per_block = 1;
  FastDiv by_chunks, by_page;
};
cudaError_t launch_kv4_write(int dtype, const Kv4CopyParams& p, cudaStream_t s);
cudaError_t launch_kv4_read(int dtype, const Kv4CopyParams& p, cudaStream_t s);

// ---- attention ------------------------------------------------------------------------
// A call's work is a row of steps: for each sequence, each tile of its query
// rows and each key-value head, the steps of 128 tokens that the tile sees.
// A row is a (token, head of the group) pair, token-major.  Every CTA takes an
// equal run of steps.  A tile that lies within one run is written to O; of one
// that is cut, every CTA writes its share (o normalised by its own sum, and
// the log2 of that sum), and a second kernel joins the shares in CTA order.
// A CTA has at most two shares: the rest of a tile begun before its run (0)
// and the begin of one that goes on after it (1).
// The record of a cut tile, written by the CTA that begins it; kept by tile
// where the call has no more tiles than CTAs, else by CTA.
struct Kv4Join {
  int seq_tile, head, first_cta, last_cta;  // last_cta < 0: not cut
};
struct Kv4AttnParams {
  Kv4Cache cache;  // heads = heads_kv
  int batch = 0, total_q = 0, max_q = 0, heads_q = 0, group = 0;
  const void* q = nullptr;
  int64_t q_stride = 0;
  const int32_t *cu_q = nullptr, *page_table = nullptr, *kv_lens = nullptr;
  int64_t table_width = 0;
  int max_kv = 0, causal = 0, window = 0;
  float scale = 0.0f;
  void* o = nullptr;
  float* lse = nullptr;
  int* status = nullptr;
  // the cut, and the shares' scratch
  FastDiv by_group, by_page16;  // rows by group, groups of 16 tokens by pages
  int tile_rows = 0, row_tiles = 0, ctas = 0;
  int joins = 0, by_tile = 0;   // records (0: no tile can be cut)
  Kv4Join* join = nullptr;      // [joins]
  float* share_o = nullptr;     // [cta][2][tile_rows][dim]
  float* share_lse = nullptr;   // [cta][2][tile_rows]
};
// Tiles of rows of a call, those that a shorter sequence leaves empty among them.
int64_t kv4_attention_tiles(int64_t batch, int64_t max_q, int64_t group);
// Fills in the cut for this device; the scratch that it needs.
size_t kv4_attention_plan(Kv4AttnParams* p, int sm_count);
void kv4_attention_scratch(Kv4AttnParams* p, void* scratch);
cudaError_t launch_kv4_attention(int dtype, const Kv4AttnParams& p, int* launches, cudaStream_t s);

// The kernel for few rows (kv4_rows.cu): tiles of 8 or 16 rows.
int kv4_rows_per_sm(int tile_rows);  // CTAs that an SM holds
cudaError_t launch_kv4_rows(int dtype, const Kv4AttnParams& p, cudaStream_t s);

// The kernel for more (kv4_tiles.cu): tiles of 256 rows, one CTA an SM.
cudaError_t launch_kv4_tiles(int dtype, const Kv4AttnParams& p, cudaStream_t s);

}  // namespace lbg
