// kv4_attention.cu -- attention of new tokens over the 4-bit paged cache: how
// a call is cut into units, and the kernel that joins the chunks of a tile.
//
//   t_ij = scale * ks_j * (q_i . kc_j)       kc, vc codes; ks, vs their scales
//   o_i  = sum_j softmax_j(t_ij) vs_j vc_j,  lse_i = log sum_j exp(t_ij)
//
// Both products run on the codes, which 16-bit floats hold exactly: the key
// scale multiplies a column of scores, the value scale a column of weights.
#include <cuda_runtime.h>

#include <algorithm>

#include "attn.h"
#include "attn_common.cuh"
#include "kv4_attention.cuh"

namespace lbg {
namespace {

// Joins the chunks of a tile's row: with share c's o_c and lse_c (log2),
//   o = sum_c 2^(lse_c - lse) o_c,  lse = log2 sum_c 2^lse_c.
// A block per (tile, row); GROUPS thread groups take every GROUPS-th chunk
// and are added in order.
constexpr int kJoinThreads = 256;

template <typename T, int DIM>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const Kv4AttnParams p) {
  constexpr int LANES = DIM / 4, GROUPS = kJoinThreads / LANES;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int row = blockIdx.y;
  int tile = blockIdx.x;
  const int b = tile / (p.cache.heads * p.row_tiles);
  tile -= b * p.cache.heads * p.row_tiles;
  const int head = tile / p.row_tiles;
  tile -= head * p.row_tiles;
  const RowTile t = row_tile(p, b, tile);
  if (row >= t.rows || t.chunks <= 1) return;
  const int64_t unit = unit_of(p, b, head, tile, 0);
  const float* lse = p.share_lse + unit * p.tile_rows + row;
  const float* o = p.share_o + (unit * p.tile_rows + row) * DIM;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  __shared__ float4 sh[GROUPS][LANES];
  __shared__ float top_sh[kJoinThreads / 32], sum_sh[GROUPS];
  // the maximum, with a NaN kept: every thread over its own chunks
  float top = -INFINITY;
  bool nan = false;
  for (int c = threadIdx.x; c < t.chunks; c += kJoinThreads) {
    const float v = lse[(int64_t)c * p.tile_rows];
    nan |= v != v;
    top = fmaxf(top, v);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (threadIdx.x % 32 == 0) top_sh[threadIdx.x / 32] = top;
  nan = __syncthreads_or(nan);
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) top = fmaxf(top, top_sh[w]);
  const float ref = top == -INFINITY ? 0.0f : top;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float sum = 0.0f;
#pragma unroll 4
  for (int c = group; c < t.chunks; c += GROUPS) {
    const float w = ex2(lse[(int64_t)c * p.tile_rows] - ref);
    const float4 v =
        reinterpret_cast<const float4*>(o + (int64_t)c * p.tile_rows * DIM)[lane];
    // a chunk that a row sees nothing of has o = 0 and weight 0
    sum += w;
    acc.x += w * v.x;
    acc.y += w * v.y;
    acc.z += w * v.z;
    acc.w += w * v.w;
  }
  sh[group][lane] = acc;
  if (lane == 0) sum_sh[group] = sum;
  __syncthreads();
  if (group != 0) return;
#pragma unroll
  for (int g = 1; g < GROUPS; ++g) {
    const float4 v = sh[g][lane];
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
    sum += sum_sh[g];
  }
  const float inv = nan ? NAN : sum > 0.0f ? 1.0f / sum : 0.0f;
  const int64_t at = out_row(p, t, head, t.r0 + row);
  T h[4] = {from_f32<T>(acc.x * inv), from_f32<T>(acc.y * inv), from_f32<T>(acc.z * inv),
            from_f32<T>(acc.w * inv)};
  reinterpret_cast<uint2*>(static_cast<T*>(p.o) + at * DIM)[lane] =
      *reinterpret_cast<const uint2*>(h);
  if (p.lse && lane == 0)
    p.lse[at] = nan ? NAN : sum > 0.0f ? (ref + log2f(sum)) * kLn2 : -INFINITY;
}

template <typename T>
cudaError_t launch_join(const Kv4AttnParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * p.cache.heads * p.row_tiles), (unsigned)p.tile_rows);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  // may be scheduled while the last chunks run; it waits for them itself
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.cache.dim == 64 ? cudaLaunchKernelEx(&cfg, kv4_join_kernel<T, 64>, p)
                           : cudaLaunchKernelEx(&cfg, kv4_join_kernel<T, 128>, p);
}

}  // namespace

size_t kv4_attention_plan(Kv4AttnParams* p, int sm_count) {
  const int64_t rows = (int64_t)p->max_q * p->group;
  p->by_group = FastDiv((uint32_t)p->group);
  p->by_page16 = FastDiv((uint32_t)(p->cache.page_size / 16));
  p->tile_rows = rows <= 8 ? 8 : 16;
  p->row_tiles = (int)((rows + p->tile_rows - 1) / p->tile_rows);
  // Tokens that a tile can see at most, and the chunks they are cut into:
  // about three waves of CTAs (four a SM), so that sequences of unequal
  // lengths even out, chunks of 512 tokens or more.
  int64_t span = p->max_kv;
  if (p->window)
    span = std::min<int64_t>(span, (int64_t)p->window + (p->tile_rows + p->group - 1) / p->group + 32);
  const int64_t tiles = (int64_t)p->batch * p->cache.heads * p->row_tiles;
  const int64_t want = std::max<int64_t>(1, (int64_t)sm_count * 12 / tiles);
  int64_t chunk = (span + want - 1) / want;
  chunk = std::max<int64_t>(512, (chunk + 127) / 128 * 128);
  p->chunk = (int)std::min<int64_t>(chunk, int64_t(1) << 30);
  p->max_chunks = (int)std::max<int64_t>(1, (span + p->chunk - 1) / p->chunk);
  if (p->max_chunks == 1) return 0;
  return (size_t)(tiles * p->max_chunks * p->tile_rows) * (p->cache.dim + 1) * sizeof(float);
}

cudaError_t launch_kv4_attention(int dtype, const Kv4AttnParams& p, int* launches, cudaStream_t s) {
  cudaError_t e = launch_kv4_rows(dtype, p, s);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (p.max_chunks > 1) {
    e = dtype == LBGEMM_BF16 ? launch_join<__nv_bfloat16>(p, s) : launch_join<__half>(p, s);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  return cudaSuccess;
}

}  // namespace lbg
