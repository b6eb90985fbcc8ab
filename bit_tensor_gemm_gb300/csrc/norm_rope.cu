// norm_rope.cu -- RMS norm of each query and key head with the position
// rotation in the same pass, and its backward pass.
//
//   forward   y  = R(p) (w . xhat),  xhat = x * rstd,  rstd = (mean(x^2) + eps)^-1/2
//   backward  g  = R(-p) dy          (R turns pairs by an angle: its transpose turns back)
//             dw = sum over tokens and heads of g . xhat
//             dx = rstd * (w . g - xhat * mean(w . g . xhat))
//
// A few operations per element against 4 bytes moved (8 for the backward
// pass): bound by HBM.  One pass: a head's vector lives in the registers of a
// few lanes from its load to its store, its sum of squares is a shuffle
// reduction, and the rotation's partner channel comes by shuffle.
#include <cuda_runtime.h>

#include <algorithm>

#include "attn.h"
#include "attn_common.cuh"

namespace lbg {
namespace {

constexpr int kThreads = 256;
constexpr int kFwdHeads = 4;  // heads of one token that a lane group holds at once
constexpr int kBwdHeads = 2;  // (the backward pass holds two vectors a head)

// The table row of a token, clamped into the table (and reported) when the
// position is out of range.
__device__ __forceinline__ int64_t table_row(const NormRopeParams& p, int64_t token) {
  int64_t row = p.positions[token];
  if (row < 0 || row >= p.table_rows) {
    atomicOr(p.status, kStatusBadIndex);
    row = row < 0 ? 0 : p.table_rows - 1;
  }
  return row;
}

// ---- heads of 64, 128 or 256 channels ---------------------------------------------
// LPH = dim / 8 lanes hold a head, 8 consecutive channels each.  Channel pairs
// (j, j + rot / 2) with rot % 16 == 0 sit in the same register of lanes
// rot / 16 apart; interleaved pairs in neighbouring registers of one lane.
template <int LPH, bool INTER>
struct Rotation {
  float c[INTER ? 4 : 8], s[INTER ? 4 : 8];
  int partner;
  bool on;

  __device__ __forceinline__ void load(const NormRopeParams& p, int64_t token, int lane, bool back) {
    on = lane * 8 < p.rot;
    partner = lane;
    if (!on) return;
    const int rl = p.rot / 16;  // lanes of the first half
    const int64_t at = table_row(p, token) * (p.rot / 2) + (INTER ? lane * 4 : lane % rl * 8);
    const float4* cp = reinterpret_cast<const float4*>(p.cosines + at);
    const float4* sp = reinterpret_cast<const float4*>(p.sines + at);
#pragma unroll
    for (int i = 0; i < (INTER ? 1 : 2); ++i) {
      reinterpret_cast<float4*>(c)[i] = __ldg(cp + i);
      reinterpret_cast<float4*>(s)[i] = __ldg(sp + i);
    }
    // y = own * cos + partner * (-sin for the first of a pair, sin for the second)
    const bool minus = (!INTER && lane < rl) != back;
    if (!INTER) partner = lane < rl ? lane + rl : lane - rl;
    if (INTER ? back : minus) {
#pragma unroll
      for (int i = 0; i < (INTER ? 4 : 8); ++i) s[i] = -s[i];
    }
  }

  __device__ __forceinline__ void turn(float (&x)[8]) const {
    if (INTER) {
      if (on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[2 * i], b = x[2 * i + 1];
          x[2 * i] = a * c[i] - b * s[i];
          x[2 * i + 1] = a * s[i] + b * c[i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = __shfl_sync(0xffffffffu, x[i], partner, LPH);
        if (on) x[i] = x[i] * c[i] + other * s[i];
      }
    }
  }
};

template <int LPH>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = LPH / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// One item is `HEADS` heads of one side of one token; item index = token *
// (chunks_q + chunks_k) + chunk, the queries' chunks first.
struct Item {
  int64_t token;
  int side, head, count;
};
template <int HEADS>
__device__ __forceinline__ Item item_of(const NormRopeParams& p, int64_t item, int chunks_q,
                                        int chunks) {
  Item it;
  it.token = item / chunks;
  int c = (int)(item - it.token * chunks);
  it.side = c >= chunks_q;
  if (it.side) c -= chunks_q;
  it.head = c * HEADS;
  it.count = min(HEADS, p.heads[it.side] - it.head);
  return it;
}

template <typename T, int LPH, bool INTER>
__global__ void __launch_bounds__(kThreads)
    norm_rope_kernel(const NormRopeParams p, int64_t items, int chunks_q, int chunks) {
  constexpr int DIM = LPH * 8;
  const int lane = threadIdx.x % LPH;
  const int64_t index = (int64_t)blockIdx.x * (kThreads / LPH) + threadIdx.x / LPH;
  // (the lanes of a warp shuffle together: a group without an item computes
  // the last one again and stores nothing)
  const Item it = item_of<kFwdHeads>(p, index < items ? index : items - 1, chunks_q, chunks);
  const int count = index < items ? it.count : 0;
  const NormRopeSide& sd = p.side[it.side];
  const T* in = static_cast<const T*>(sd.in) + it.token * sd.in_stride + (int64_t)it.head * DIM +
                lane * 8;
  Raw8<T> raw[kFwdHeads];
#pragma unroll
  for (int h = 0; h < kFwdHeads; ++h)
    if (h < count) raw[h] = load8_raw(in + h * DIM);
  Rotation<LPH, INTER> rot;
  rot.load(p, it.token, lane, false);
  float w[8];
  if (sd.w) load8(static_cast<const T*>(sd.w) + lane * 8, w);
  T* out = static_cast<T*>(sd.out) + it.token * sd.out_stride + (int64_t)it.head * DIM + lane * 8;
#pragma unroll
  for (int h = 0; h < kFwdHeads; ++h) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    if (h < count) unpack8(raw[h], x);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
    sum = group_sum<LPH>(sum);
    if (sd.w) {
      const float r = rsqrtf(sum * (1.0f / DIM) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
    }
    rot.turn(x);
    if (h < count) store8(out + h * DIM, x);
  }
}

// The backward pass: blocks stride over the items, each lane summing its
// channels' weight gradients in registers; a block's lane groups are then
// added in order into partial[block][side][channel].
template <typename T, int LPH, bool INTER>
__global__ void __launch_bounds__(kThreads)
    norm_rope_backward_kernel(const NormRopeParams p, int64_t items, int chunks_q, int chunks,
                              float* __restrict__ partial) {
  constexpr int DIM = LPH * 8, GROUPS = kThreads / LPH;
  const int lane = threadIdx.x % LPH, group = threadIdx.x / LPH;
  float dw[2][8] = {};
  for (int64_t first = (int64_t)blockIdx.x * GROUPS; first < items;
       first += (int64_t)gridDim.x * GROUPS) {
    const int64_t index = first + group;
    const Item it = item_of<kBwdHeads>(p, index < items ? index : items - 1, chunks_q, chunks);
    const int count = index < items ? it.count : 0;
    const NormRopeSide& sd = p.side[it.side];
    const int64_t at = (int64_t)it.head * DIM + lane * 8;
    const T* in = static_cast<const T*>(sd.in) + it.token * sd.in_stride + at;
    const T* xp = static_cast<const T*>(sd.x) + it.token * sd.x_stride + at;
    Raw8<T> rg[kBwdHeads], rx[kBwdHeads];
#pragma unroll
    for (int h = 0; h < kBwdHeads; ++h)
      if (h < count) {
        rg[h] = load8_raw(in + h * DIM);
        if (sd.w) rx[h] = load8_raw(xp + h * DIM);
      }
    Rotation<LPH, INTER> rot;
    rot.load(p, it.token, lane, true);
    float w[8];
    if (sd.w) load8(static_cast<const T*>(sd.w) + lane * 8, w);
    T* out = static_cast<T*>(sd.out) + it.token * sd.out_stride + at;
#pragma unroll
    for (int h = 0; h < kBwdHeads; ++h) {
      float g[8], x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = x[i] = 0.0f;
      if (h < count) {
        unpack8(rg[h], g);
        if (sd.w) unpack8(rx[h], x);
      }
      rot.turn(g);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
      sum = group_sum<LPH>(sum);
      const float r = rsqrtf(sum * (1.0f / DIM) + p.eps);
      if (sd.w) {
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= r;
          const float t = g[i] * x[i];
          if (it.side) dw[1][i] += h < count ? t : 0.0f;
          else dw[0][i] += h < count ? t : 0.0f;
          dot += t * w[i];
        }
        sum = dot;
      }
      sum = group_sum<LPH>(sum) * (1.0f / DIM);
      if (sd.w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = r * (w[i] * g[i] - x[i] * sum);
      }
      if (h < count) store8(out + h * DIM, g);
    }
  }
  if (partial == nullptr) return;
  __shared__ float sh[GROUPS][2][DIM + 4];
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int i = 0; i < 8; ++i) sh[group][side][lane * 8 + i] = dw[side][i];
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * DIM; c += kThreads) {
    float v = 0.0f;
    for (int g = 0; g < GROUPS; ++g) v += sh[g][c / DIM][c % DIM];
    partial[(int64_t)blockIdx.x * 2 * DIM + c] = v;
  }
}

// ---- any head of up to 512 channels, any even rotation --------------------------------
// One warp a head, its vectors in shared memory as fp32, channels strided over
// the lanes: for head sizes and rotations that do not fit the layout above.
constexpr int kMaxDim = 512, kAnyWarps = 4;

__device__ __forceinline__ void pair_of(const NormRopeParams& p, int c, int* a, int* b, int* j) {
  if (p.interleaved) {
    *j = c >> 1;
    *a = c & ~1;
    *b = c | 1;
  } else {
    *j = c < p.rot / 2 ? c : c - p.rot / 2;
    *a = *j;
    *b = *j + p.rot / 2;
  }
}

// Channel c of R(p) x (back: of R(-p) x), x in shared memory.
__device__ __forceinline__ float turned(const NormRopeParams& p, const float* x, int c,
                                        int64_t row, bool back) {
  if (c >= p.rot) return x[c];
  int a, b, j;
  pair_of(p, c, &a, &b, &j);
  const float co = __ldg(p.cosines + row * (p.rot / 2) + j);
  float si = __ldg(p.sines + row * (p.rot / 2) + j);
  if (back) si = -si;
  return c == a ? x[a] * co - x[b] * si : x[a] * si + x[b] * co;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <typename T, bool BACK>
__global__ void __launch_bounds__(kAnyWarps * 32)
    norm_rope_any_kernel(const NormRopeParams p, float* __restrict__ partial) {
  extern __shared__ float sh[];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, dim = p.dim;
  float* v = sh + warp * (BACK ? 4 : 1) * dim;  // x (BACK: dy), then x and the two dw sums
  float* x = BACK ? v + dim : v;
  float* dw = v + 2 * dim;
  if (BACK)
    for (int c = lane; c < 2 * dim; c += 32) dw[c] = 0.0f;
  const int heads = p.heads[0] + p.heads[1];
  const int64_t items = p.tokens * heads;
  for (int64_t item = (int64_t)blockIdx.x * kAnyWarps + warp; item < items;
       item += (int64_t)gridDim.x * kAnyWarps) {
    const int64_t token = item / heads;
    int head = (int)(item - token * heads);
    const int side = head >= p.heads[0];
    if (side) head -= p.heads[0];
    const NormRopeSide& sd = p.side[side];
    const T* in = static_cast<const T*>(sd.in) + token * sd.in_stride + (int64_t)head * dim;
    const T* xp = static_cast<const T*>(sd.x) + token * sd.x_stride + (int64_t)head * dim;
    T* out = static_cast<T*>(sd.out) + token * sd.out_stride + (int64_t)head * dim;
    const T* w = static_cast<const T*>(sd.w);
    int64_t row = 0;
    if (p.rot > 0) row = table_row(p, token);
    float sum = 0.0f;
    __syncwarp();
    for (int c = lane; c < dim; c += 32) {
      v[c] = to_f32(in[c]);
      if (BACK && w) x[c] = to_f32(xp[c]);
      if (w) sum += x[c] * x[c];
    }
    const float r = rsqrtf(warp_sum(sum) / (float)dim + p.eps);
    if (!BACK) {
      if (w)
        for (int c = lane; c < dim; c += 32) v[c] = v[c] * r * to_f32(w[c]);
      __syncwarp();
      for (int c = lane; c < dim; c += 32) out[c] = from_f32<T>(turned(p, v, c, row, false));
    } else {
      __syncwarp();
      float dot = 0.0f;
      if (w)
        for (int c = lane; c < dim; c += 32) {
          const float t = turned(p, v, c, row, true) * x[c] * r;
          dw[side * dim + c] += t;
          dot += t * to_f32(w[c]);
        }
      dot = warp_sum(dot) / (float)dim;
      for (int c = lane; c < dim; c += 32) {
        float g = turned(p, v, c, row, true);
        if (w) g = r * (g * to_f32(w[c]) - x[c] * r * dot);
        out[c] = from_f32<T>(g);
      }
    }
  }
  if (!BACK || partial == nullptr) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * dim; c += kAnyWarps * 32) {
    float s = 0.0f;
    for (int g = 0; g < kAnyWarps; ++g) s += sh[g * 4 * dim + 2 * dim + c];
    partial[(int64_t)blockIdx.x * 2 * dim + c] = s;
  }
}

// dw[side][c] = sum over blocks of partial[block][side][c], in block order
// within each of 8 strided sums and those in order: the same bits every time.
__global__ void __launch_bounds__(256)
    norm_weight_grad_kernel(const float* __restrict__ partial, int blocks, int dim,
                            float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float sh[8][33];
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + x;
  float v = 0.0f;
  if (c < 2 * dim)
    for (int b = y; b < blocks; b += 8) v += partial[(int64_t)b * 2 * dim + c];
  sh[y][x] = v;
  __syncthreads();
  if (y == 0 && c < 2 * dim) {
#pragma unroll
    for (int g = 1; g < 8; ++g) v += sh[g][x];
    float* dw = c < dim ? dwq : dwk;
    if (dw) dw[c < dim ? c : c - dim] = v;
  }
}

// Heads of 64, 128 or 256 channels whose pairs fit the register layout.
bool in_registers(const NormRopeParams& p) {
  return (p.dim == 64 || p.dim == 128 || p.dim == 256) && p.rot % 16 == 0;
}

struct Plan {
  int64_t items = 0;
  int chunks_q = 0, chunks = 0, blocks = 0;
};
Plan plan_of(const NormRopeParams& p, int heads, bool back, int sm_count) {
  Plan pl;
  if (in_registers(p)) {
    pl.chunks_q = (p.heads[0] + heads - 1) / heads;
    pl.chunks = pl.chunks_q + (p.heads[1] + heads - 1) / heads;
    pl.items = p.tokens * pl.chunks;
    const int64_t per = kThreads / (p.dim / 8);
    const int64_t blocks = (pl.items + per - 1) / per;
    pl.blocks = (int)(back ? std::min<int64_t>(blocks, (int64_t)sm_count * 4) : blocks);
  } else {
    pl.items = p.tokens * (p.heads[0] + p.heads[1]);
    pl.blocks = (int)std::min<int64_t>((pl.items + kAnyWarps - 1) / kAnyWarps,
                                       (int64_t)sm_count * (back ? 4 : 16));
  }
  return pl;
}

template <typename T, int LPH>
void launch_in_registers(const NormRopeParams& p, const Plan& pl, bool back, float* partial,
                         cudaStream_t s) {
  if (back) {
    if (p.interleaved)
      norm_rope_backward_kernel<T, LPH, true>
          <<<pl.blocks, kThreads, 0, s>>>(p, pl.items, pl.chunks_q, pl.chunks, partial);
    else
      norm_rope_backward_kernel<T, LPH, false>
          <<<pl.blocks, kThreads, 0, s>>>(p, pl.items, pl.chunks_q, pl.chunks, partial);
  } else {
    if (p.interleaved)
      norm_rope_kernel<T, LPH, true>
          <<<pl.blocks, kThreads, 0, s>>>(p, pl.items, pl.chunks_q, pl.chunks);
    else
      norm_rope_kernel<T, LPH, false>
          <<<pl.blocks, kThreads, 0, s>>>(p, pl.items, pl.chunks_q, pl.chunks);
  }
}

template <typename T>
void launch_typed(const NormRopeParams& p, const Plan& pl, bool back, float* partial,
                  cudaStream_t s) {
  if (in_registers(p)) {
    if (p.dim == 64) launch_in_registers<T, 8>(p, pl, back, partial, s);
    else if (p.dim == 128) launch_in_registers<T, 16>(p, pl, back, partial, s);
    else launch_in_registers<T, 32>(p, pl, back, partial, s);
  } else if (back) {
    norm_rope_any_kernel<T, true>
        <<<pl.blocks, kAnyWarps * 32, kAnyWarps * 4 * p.dim * sizeof(float), s>>>(p, partial);
  } else {
    norm_rope_any_kernel<T, false>
        <<<pl.blocks, kAnyWarps * 32, kAnyWarps * p.dim * sizeof(float), s>>>(p, nullptr);
  }
}

void launch_any_type(int dtype, const NormRopeParams& p, const Plan& pl, bool back, float* partial,
                     cudaStream_t s) {
  if (dtype == LBGEMM_BF16) launch_typed<__nv_bfloat16>(p, pl, back, partial, s);
  else if (dtype == LBGEMM_F16) launch_typed<__half>(p, pl, back, partial, s);
  else launch_typed<float>(p, pl, back, partial, s);
}

}  // namespace

cudaError_t launch_norm_rope(int dtype, const NormRopeParams& p, int sm_count, cudaStream_t s) {
  const Plan pl = plan_of(p, kFwdHeads, false, sm_count);
  launch_any_type(dtype, p, pl, false, nullptr, s);
  return cudaGetLastError();
}

size_t norm_rope_scratch(const NormRopeParams& p, int sm_count) {
  if (!p.side[0].w && !p.side[1].w) return 0;
  const Plan pl = plan_of(p, kBwdHeads, true, sm_count);
  return (size_t)std::max(1, pl.blocks) * 2 * p.dim * sizeof(float);
}

cudaError_t launch_norm_rope_backward(int dtype, const NormRopeParams& p, int sm_count,
                                      float* partial, int* launches, cudaStream_t s) {
  const Plan pl = plan_of(p, kBwdHeads, true, sm_count);
  if (pl.blocks > 0) {
    launch_any_type(dtype, p, pl, true, partial, s);
    *launches += 1;
  }
  if (partial) {
    norm_weight_grad_kernel<<<(2 * p.dim + 31) / 32, 256, 0, s>>>(partial, pl.blocks, p.dim,
                                                                 p.side[0].dw, p.side[1].dw);
    *launches += 1;
  }
  return cudaGetLastError();
}

}  // namespace lbg
