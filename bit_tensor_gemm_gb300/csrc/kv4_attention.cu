// kv4_attention.cu -- attention of new tokens over the 4-bit paged cache: how
// a call is cut, and the kernel that joins the shares of a tile.
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

// Rows of a sequence (query tokens x heads of a group) up to which the kernel
// for few rows runs: it streams the cache once for every 16 of them (from L2, but
// for the first), the other works for 256 rows whatever there are.  16 sequences
// of up to 8192 tokens: 64 rows 82 us with the one, 92 with the other, 96 rows
// 162 and 100; one sequence of 4096: 64 rows 17.9 and 29.1, 96 rows 23.8 and 30.0
// (a single sequence would do better with the first up to 128 rows: the threshold is
// one that a batch does not lose by).
constexpr int64_t kFewRows = 64;

// Joins the shares of a tile's row: with share c's o_c and lse_c (log2),
//   o = sum_c 2^(lse_c - lse) o_c,  lse = log2 sum_c 2^lse_c.
// TEAMS teams of DIM / 4 threads a block.  PER_ROW teams take every PER_ROW-th
// share of a row and are added in order: all of them where a tile has few rows
// (it may have many shares), one for tiles of 256 (few shares).  Many small blocks:
// 8 of them an SM, 32 registers a thread (44: 24 drafts of 5 tokens 20.5 us, 18.4 so).
constexpr int kJoinThreads = 256;

template <typename T, int DIM, bool MANY_ROWS>
__global__ void __launch_bounds__(kJoinThreads, MANY_ROWS ? 6 : 8)
    kv4_join_kernel(const Kv4AttnParams p) {
  constexpr int LANES = DIM / 4, TEAMS = kJoinThreads / LANES, PER_ROW = MANY_ROWS ? 1 : TEAMS;
  const int lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
  const int row = MANY_ROWS ? blockIdx.y * TEAMS + team : blockIdx.y;
  // (what comes from the call's inputs is looked up before the shares are there;
  // by tile, one without rows has no record)
  RowTile t = {};
  if (p.by_tile) {
    t = row_tile(p, blockIdx.x / p.cache.heads);
    if ((MANY_ROWS ? blockIdx.y * TEAMS : row) >= t.rows) return;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Kv4Join j = p.join[blockIdx.x];
  if (j.last_cta < 0) return;
  if (!p.by_tile) t = row_tile(p, j.seq_tile);
  const bool live = row < t.rows;
  // share 0 of the tile is its first CTA's share 1, the others' share 0 follow
  const int shares = live ? j.last_cta - j.first_cta + 1 : 0;
  auto index = [&](int c) -> int64_t {
    return (int64_t)((j.first_cta + c) * 2 + (c == 0)) * p.tile_rows + row;
  };
  // the first shares, on their way while the largest lse is found
  constexpr int AHEAD = 2;
  float4 v_ahead[AHEAD];
  float lse_ahead[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    const int c = (MANY_ROWS ? 0 : team) + k * PER_ROW;
    v_ahead[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    lse_ahead[k] = -INFINITY;
    if (c < shares) {
      v_ahead[k] = reinterpret_cast<const float4*>(p.share_o + index(c) * DIM)[lane];
      lse_ahead[k] = p.share_lse[index(c)];
    }
  }
  // the largest lse, and whether one is a NaN
  float top = -INFINITY;
  int nan = 0;
  for (int c = lane; c < shares; c += LANES) {
    const float v = p.share_lse[index(c)];
    nan |= v != v;
    top = fmaxf(top, v);
  }
#pragma unroll
  for (int x = LANES / 2; x >= 1; x >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    nan |= __shfl_xor_sync(0xffffffffu, nan, x);
  }
  // (weights are at most 1 over the shares, rounded up to a power of two: their sum
  // with values near fp32's largest stays in range)
  const float ref = top == -INFINITY ? 0.0f : top + (float)(32 - __clz(shares));
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float sum = 0.0f;
  // (a share that the row sees nothing of has o = 0 and weight 0; a weight is split in
  // two, as the exponential gives 0 below 2^-126: beside a largest share of tiny
  // values such a one still counts)
  auto add = [&](float share_lse, const float4& v) {
    const float w = ex2(fmaxf(share_lse - ref, -120.0f));
    const float x = ex2(fminf(share_lse - ref + 120.0f, 0.0f));
    sum += w * x;
    acc.x += w * v.x * x;
    acc.y += w * v.y * x;
    acc.z += w * v.z * x;
    acc.w += w * v.w * x;
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) add(lse_ahead[k], v_ahead[k]);
#pragma unroll 4
  for (int c = (MANY_ROWS ? 0 : team) + AHEAD * PER_ROW; c < shares; c += PER_ROW)
    add(p.share_lse[index(c)], reinterpret_cast<const float4*>(p.share_o + index(c) * DIM)[lane]);
  if constexpr (!MANY_ROWS) {
    __shared__ float4 sh[TEAMS][LANES];
    __shared__ float sum_sh[TEAMS];
    sh[team][lane] = acc;
    if (lane == 0) sum_sh[team] = sum;
    __syncthreads();
    if (team != 0) return;
#pragma unroll
    for (int g = 1; g < TEAMS; ++g) {
      const float4 v = sh[g][lane];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
      sum += sum_sh[g];
    }
  }
  if (!live) return;
  const float inv = nan ? NAN : sum > 0.0f ? 1.0f / sum : 0.0f;
  const int64_t at = out_row(p, t, j.head, t.r0 + row);
  T h[4] = {from_f32<T>(acc.x * inv), from_f32<T>(acc.y * inv), from_f32<T>(acc.z * inv),
            from_f32<T>(acc.w * inv)};
  reinterpret_cast<uint2*>(static_cast<T*>(p.o) + at * DIM)[lane] =
      *reinterpret_cast<const uint2*>(h);
  if (p.lse && lane == 0)
    p.lse[at] = nan ? NAN : sum > 0.0f ? (ref + log2f(sum)) * kLn2 : -INFINITY;
}

template <typename T, int DIM>
cudaError_t launch_join_dim(const Kv4AttnParams& p, cudaStream_t s) {
  const bool many = p.tile_rows == 256;
  const int rows = (int)std::min<int64_t>(p.tile_rows, (int64_t)p.max_q * p.group);
  const int per_block = many ? kJoinThreads / (DIM / 4) : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.joins, (unsigned)((rows + per_block - 1) / per_block));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  // may be scheduled while the last shares are computed; it waits for them itself
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, kv4_join_kernel<T, DIM, true>, p)
              : cudaLaunchKernelEx(&cfg, kv4_join_kernel<T, DIM, false>, p);
}

template <typename T>
cudaError_t launch_join(const Kv4AttnParams& p, cudaStream_t s) {
  return p.cache.dim == 64 ? launch_join_dim<T, 64>(p, s) : launch_join_dim<T, 128>(p, s);
}

// (8 rows of those 16 sequences 32 us; 9 to 16, which need twice the MMAs, 50)
int tile_rows_of(int64_t rows) { return rows <= 8 ? 8 : rows <= kFewRows ? 16 : 256; }

}  // namespace

int64_t kv4_attention_tiles(int64_t batch, int64_t max_q, int64_t group) {
  const int64_t rows = max_q * group, tile = tile_rows_of(rows);
  return batch * ((rows + tile - 1) / tile);
}

size_t kv4_attention_plan(Kv4AttnParams* p, int sm_count) {
  const int64_t rows = (int64_t)p->max_q * p->group;
  p->by_group = FastDiv((uint32_t)p->group);
  p->by_page16 = FastDiv((uint32_t)(p->cache.page_size / 16));
  p->tile_rows = tile_rows_of(rows);
  p->row_tiles = (int)kv4_attention_tiles(1, p->max_q, p->group);
  // one wave of CTAs, or fewer where the longest lengths would not fill it
  const int64_t tiles = kv4_attention_tiles(p->batch, p->max_q, p->group) * p->cache.heads;
  const int64_t steps = tiles * (p->max_kv / kStepTokens + 2);
  const int per_sm = p->tile_rows == 256 ? 1 : kv4_rows_per_sm(p->tile_rows);
  p->ctas = (int)std::min<int64_t>((int64_t)sm_count * per_sm, steps);
  // (tiles of one step each cannot be cut)
  p->by_tile = tiles <= p->ctas;
  p->joins = p->max_kv <= kStepTokens ? 0 : p->by_tile ? (int)tiles : p->ctas;
  if (p->joins == 0) return 0;
  return (size_t)p->joins * sizeof(Kv4Join) +
         (size_t)p->ctas * 2 * p->tile_rows * (p->cache.dim + 1) * sizeof(float);
}

void kv4_attention_scratch(Kv4AttnParams* p, void* scratch) {
  p->join = static_cast<Kv4Join*>(scratch);
  p->share_o = reinterpret_cast<float*>(p->join + p->joins);
  p->share_lse = p->share_o + (int64_t)p->ctas * 2 * p->tile_rows * p->cache.dim;
}

cudaError_t launch_kv4_attention(int dtype, const Kv4AttnParams& p, int* launches, cudaStream_t s) {
  cudaError_t e = p.tile_rows == 256 ? launch_kv4_tiles(dtype, p, s) : launch_kv4_rows(dtype, p, s);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (p.joins > 0) {
    e = dtype == LBGEMM_BF16 ? launch_join<__nv_bfloat16>(p, s) : launch_join<__half>(p, s);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  return cudaSuccess;
}

}  // namespace lbg
