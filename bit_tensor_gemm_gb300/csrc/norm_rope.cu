// norm_rope.cu -- RMS norm of each query and key head with the position
// rotation in the same pass, and its backward pass.
//
//   forward   y  = R(p) (w . xhat),  xhat = x * rstd,  rstd = (mean(x^2) + eps)^-1/2
//   backward  g  = R(-p) dy          (R turns pairs by an angle: its transpose turns back)
//             dw = sum over tokens and heads of g . xhat
//             dx = rstd * (w . g - xhat * mean(w . g . xhat))
//
// A few operations per element against 4 bytes moved (6 for the backward
// pass): bound by HBM.  One pass: a head's vector lives in the registers of a
// few lanes from its load to its store, its sum of squares is a shuffle
// reduction, and the rotation's partner channel is in the same lane.
// Measured, bf16, 40 heads of 128 channels: 16384 tokens 60.2 us (5.7 TB/s; a
// block a few rows, loads into registers: 70.6); 8192 tokens with the backward
// pass 84.8 us (123), of which the backward pass 52 (252 MB: 4.9 TB/s).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "attn.h"
#include "attn_common.cuh"
#include "ptx.cuh"

namespace lbg {
namespace {

constexpr int kWarps = 8;  // that compute; one more copies
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxStages = 8;
// Blocks an SM is to hold, and the ring that each may have for it (the backward
// pass keeps its sums in shared memory as well).
constexpr int kFwdBlocks = 4, kBwdBlocks = 3;
constexpr int kFwdRing = 54 * 1024, kBwdRing = 64 * 1024;
// Runs to a block's place on the SM: blocks do not all proceed at one rate, and
// a second, shorter run evens that out in the forward pass (16384 tokens of 40
// heads: 68.3 us with one, 64.3 with two, 65.6 with three); the backward pass,
// which ends every block with its sums, lost by it (85.1, 90.8, 89.9).
constexpr int kFwdRuns = 2, kBwdRuns = 1;

// How a call is cut: blocks for the queries, then for the keys, and the stages
// that a block of either makes.  (The kernel for any size uses `blocks` only.)
struct NormRopeCut {
  int blocks = 0, q_blocks = 0;
  int64_t per[2] = {0, 0};
  FastDiv by_heads[2];
  int stages = 0, stage_bytes = 0;  // of the ring
};

// The table row of a position, clamped into the table (and reported) when it is
// out of range.
__device__ __forceinline__ int64_t table_row(const NormRopeParams& p, int64_t row) {
  if (row < 0 || row >= p.table_rows) {
    atomicOr(p.status, kStatusBadIndex);
    row = row < 0 ? 0 : p.table_rows - 1;
  }
  return row;
}

// ---- heads of 64, 128 or 256 channels ---------------------------------------------
// LPH = dim / 8 lanes hold a head, 8 channels each, so placed that both
// channels of a pair sit in one lane: pairs (j, j + rot / 2) as 4 channels from
// each half of the turned part, interleaved pairs as 8 in a row, like the
// channels that are not turned.  The lane's pairs are (a[i], b[i]), i < 4, kept
// two to a 64-bit register for the paired fp32 operations.
//
// Blocks belong to the queries or to the keys, in proportion to the heads, and
// take equal runs of the side's rows (the heads of every token, token-major).
// One warp copies ahead of the others, kRows rows a stage with the table rows of
// their tokens, by bulk copies into a ring in shared memory: it takes some 60 KB
// in flight on every SM to keep HBM busy, more than the registers can hold.
struct Lane {
  float2x a[2], b[2];
};

template <typename T, int LPH, bool INTER>
struct Layout {
  int first, second;  // channels of the two loads of four
  bool on;            // turned at all

  __device__ __forceinline__ Layout(int lane, int rot) {
    on = lane * 8 < rot;
    first = lane * 8;
    second = first + 4;
    if (!INTER && on) {
      first = lane * 4;
      second = first + rot / 2;
    }
  }
  __device__ __forceinline__ Lane load(const T* head) const {
    float u[4], v[4];
    load4(head + first, u);
    load4(head + second, v);
    if (INTER) return {{pair(u[0], u[2]), pair(v[0], v[2])}, {pair(u[1], u[3]), pair(v[1], v[3])}};
    return {{pair(u[0], u[1]), pair(u[2], u[3])}, {pair(v[0], v[1]), pair(v[2], v[3])}};
  }
  __device__ __forceinline__ void store(T* head, const Lane& x) const {
    float u[4], v[4];
    if (INTER) {
      unpair(x.a[0], u[0], u[2]);
      unpair(x.a[1], v[0], v[2]);
      unpair(x.b[0], u[1], u[3]);
      unpair(x.b[1], v[1], v[3]);
    } else {
      unpair(x.a[0], u[0], u[1]);
      unpair(x.a[1], u[2], u[3]);
      unpair(x.b[0], v[0], v[1]);
      unpair(x.b[1], v[2], v[3]);
    }
    store4(head + first, u);
    store4(head + second, v);
  }
};

template <int LPH>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = LPH / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

__device__ __forceinline__ float halves(float2x v) {
  float lo, hi;
  unpair(v, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ float2x twice(float v) { return pair(v, v); }
__device__ __forceinline__ float2x minus(float2x v) { return v ^ 0x8000000080000000ull; }

// Sum of x * y over the lane's channels.
__device__ __forceinline__ float lane_dot(const Lane& x, const Lane& y) {
  float2x s = mul2(x.a[0], y.a[0]);
  s = fma2(x.a[1], y.a[1], s);
  s = fma2(x.b[0], y.b[0], s);
  return halves(fma2(x.b[1], y.b[1], s));
}

// y_a = x_a cos - x_b sin, y_b = x_a sin + x_b cos
__device__ __forceinline__ void turn(Lane& x, const float2x (&c)[2], const float2x (&s)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2x a = x.a[i];
    x.a[i] = fma2(x.b[i], minus(s[i]), mul2(a, c[i]));
    x.b[i] = fma2(a, s[i], mul2(x.b[i], c[i]));
  }
}

// Rows of a stage: two a lane group, as far as one warp can look up their tokens.
template <int LPH>
constexpr int kRows = 2 * (kThreads / LPH) < 32 ? 2 * (kThreads / LPH) : 32;
// ... and the most tokens among them.
constexpr int most_tokens(int rows, int heads) {
  return heads < 1 ? 0 : (rows - 2) / heads + 2 < rows ? (rows - 2) / heads + 2 : rows;
}

// BACK: the backward pass.  Each lane sums its channels' weight gradients in
// registers; a block's lane groups are then added in order into
// partial[block][channel].  Both of a head's sums (x^2 and w . g . x) are taken
// before either is needed, so that their shuffles overlap.
template <typename T, int LPH, bool INTER, bool BACK>
__global__ void __launch_bounds__(kThreads + 32, BACK ? kBwdBlocks : kFwdBlocks)
    norm_rope_kernel(const NormRopeParams p, const NormRopeCut cut, float* __restrict__ partial) {
  constexpr int DIM = LPH * 8, GROUPS = kThreads / LPH, ROWS = kRows<LPH>;
  constexpr int kData = ROWS * DIM * (int)sizeof(T);
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t bars[2 * kMaxStages];
  __shared__ int abort_flag;
  const int warp = threadIdx.x / 32;
  const int side = blockIdx.x >= cut.q_blocks;
  const NormRopeSide sd = side ? p.side[1] : p.side[0];
  const FastDiv by_heads = side ? cut.by_heads[1] : cut.by_heads[0];
  const int heads = side ? p.heads[1] : p.heads[0];
  const bool norm = sd.w != nullptr;
  const int table = p.rot / 2;  // entries of a table's row

  // the run: rows first .. first + count, counted from the begin of their first token
  const int64_t per = side ? cut.per[1] : cut.per[0];
  const int64_t begin = (int64_t)(blockIdx.x - (side ? cut.q_blocks : 0)) * per * ROWS;
  const int64_t token0 = begin >> 31 ? begin / heads : by_heads((uint32_t)begin);
  const uint32_t first = (uint32_t)(begin - token0 * heads);
  const uint32_t end = first + (uint32_t)max((int64_t)0, min(per * ROWS, p.tokens * heads - begin));
  const int steps = (int)((end - first + ROWS - 1) / ROWS);

  const uint32_t full = smem_addr(bars), empty = full + 8 * kMaxStages;
  if (threadIdx.x < cut.stages) {
    mbar_init(full + 8 * threadIdx.x, 1);
    mbar_init(empty + 8 * threadIdx.x, kWarps);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();

  if (warp == kWarps) {
    // ---- the copies: a lane a token ----
    const int lane = threadIdx.x % 32;
    const uint32_t base = smem_addr(ring);
    int slot = 0, parity = 1;
    int64_t position = 0;  // of this lane's token of the next stage, looked up ahead
    uint32_t at = first;
    auto look_up = [&] {
      const uint32_t token = by_heads(at) + lane;
      if (p.rot > 0 && token * heads < min(at + ROWS, end)) position = p.positions[token0 + token];
    };
    look_up();
    bool dead = false;
    int step = 0;
    for (; step < steps; ++step) {
      if (step >= cut.stages)
        dead = !__all_sync(0xffffffffu, mbar_wait(empty + 8 * slot, parity, &abort_flag, p.status));
      if (dead) break;
      const uint32_t stop = min(at + ROWS, end), bar = full + 8 * slot;
      const uint32_t token_a = by_heads(at), token = token_a + lane;
      const uint32_t lo = max(at, token * heads), hi = min(stop, (token + 1) * heads);
      const uint32_t dst = base + slot * cut.stage_bytes;
      if (lane == 0)
        mbar_arrive_expect_tx(bar, (stop - at) * DIM * sizeof(T) * (BACK && norm ? 2 : 1) +
                                       (by_heads(stop - 1) - token_a + 1) * table * 8);
      __syncwarp();
      if (lo < hi) {
        const int64_t head = (int64_t)(lo - token * heads) * DIM;
        const uint32_t to = dst + (lo - at) * DIM * sizeof(T);
        const uint32_t bytes = (hi - lo) * DIM * sizeof(T);
        bulk_load(to, static_cast<const T*>(sd.in) + (token0 + token) * sd.in_stride + head, bytes,
                  bar);
        if (BACK && norm)
          bulk_load(to + kData, static_cast<const T*>(sd.x) + (token0 + token) * sd.x_stride + head,
                    bytes, bar);
        if (table > 0) {
          const int64_t row = table_row(p, position);
          const uint32_t tab = dst + kData * (BACK ? 2 : 1) + lane * table * 8;
          bulk_load(tab, p.cosines + row * table, table * 4, bar);
          bulk_load(tab + table * 4, p.sines + row * table, table * 4, bar);
        }
      }
      at = stop;
      if (++slot == cut.stages) slot = 0, parity ^= 1;
      if (step + 1 < steps) look_up();
    }
    if (dead) {  // let the copies in flight land (again with a limit)
      volatile int go_on = 0;
      for (int k = max(0, step - cut.stages); k < step; ++k)
        mbar_wait(full + 8 * (k % cut.stages), (uint32_t)(k / cut.stages) & 1u, &go_on, p.status,
                  kWaitLimitNs / 8);
    }
    return;
  }

  // ---- the rows ----
  const int lane = threadIdx.x % LPH, group = threadIdx.x / LPH;
  const Layout<T, LPH, INTER> layout(lane, p.rot);
  Lane w, dw;
  w.a[0] = w.a[1] = w.b[0] = w.b[1] = twice(1.0f);
  dw.a[0] = dw.a[1] = dw.b[0] = dw.b[1] = 0;
  if (norm) w = layout.load(static_cast<const T*>(sd.w));
  T* const out = static_cast<T*>(sd.out) + token0 * sd.out_stride;
  int slot = 0, parity = 0;
  uint32_t at = first;
  for (int step = 0; step < steps; ++step) {
    if (!__all_sync(0xffffffffu, mbar_wait(full + 8 * slot, parity, &abort_flag, p.status))) break;
    const uint8_t* stage = ring + slot * cut.stage_bytes;
    const uint32_t token_a = by_heads(at);
#pragma unroll
    for (int j = 0; j < ROWS / GROUPS; ++j) {
      // (the lanes of a warp shuffle together: past the end a group computes
      // the last row again and stores nothing)
      const uint32_t mine = at + group + j * GROUPS, r = min(mine, end - 1);
      const uint32_t token = by_heads(r);
      const T* row = reinterpret_cast<const T*>(stage) + (r - at) * DIM;
      T* to = out + token * sd.out_stride + (int64_t)(r - token * heads) * DIM;
      Lane g = layout.load(row);
      float2x c[2], s[2];
      if (layout.on) {
        const float* tab = reinterpret_cast<const float*>(stage + kData * (BACK ? 2 : 1)) +
                           (token - token_a) * (2 * table) + lane * 4;
        const float4 co = *reinterpret_cast<const float4*>(tab);
        const float4 si = *reinterpret_cast<const float4*>(tab + table);
        c[0] = pair(co.x, co.y);
        c[1] = pair(co.z, co.w);
        s[0] = pair(si.x, si.y);
        s[1] = pair(si.z, si.w);
      }
      if (!BACK) {
        if (norm) {
          const float sum = group_sum<LPH>(lane_dot(g, g));
          const float2x rs = twice(rsqrtf(sum * (1.0f / DIM) + p.eps));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            g.a[i] = mul2(mul2(g.a[i], rs), w.a[i]);
            g.b[i] = mul2(mul2(g.b[i], rs), w.b[i]);
          }
        }
        if (layout.on) turn(g, c, s);
      } else {
        if (layout.on) {
          s[0] = minus(s[0]);
          s[1] = minus(s[1]);
          turn(g, c, s);
        }
        if (norm) {
          Lane x = layout.load(row + ROWS * DIM), wg;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            wg.a[i] = mul2(w.a[i], g.a[i]);
            wg.b[i] = mul2(w.b[i], g.b[i]);
          }
          const float sum = group_sum<LPH>(lane_dot(x, x));
          const float dot = group_sum<LPH>(lane_dot(x, wg));
          const float rs = rsqrtf(sum * (1.0f / DIM) + p.eps);
          const float2x r2 = twice(rs), mean = twice(-(rs * dot * (1.0f / DIM)));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            x.a[i] = mul2(x.a[i], r2);
            x.b[i] = mul2(x.b[i], r2);
            if (mine < end) {
              dw.a[i] = fma2(g.a[i], x.a[i], dw.a[i]);
              dw.b[i] = fma2(g.b[i], x.b[i], dw.b[i]);
            }
            g.a[i] = mul2(r2, fma2(x.a[i], mean, wg.a[i]));
            g.b[i] = mul2(r2, fma2(x.b[i], mean, wg.b[i]));
          }
        }
      }
      if (mine < end) layout.store(to, g);
    }
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(empty + 8 * slot);
    at += ROWS;
    if (++slot == cut.stages) slot = 0, parity ^= 1;
  }
  if (!BACK || !norm) return;
  // (only the computing warps are left)
  __shared__ __align__(16) float sums[BACK ? GROUPS : 1][BACK ? DIM : 1];
  const Layout<float, LPH, INTER> order(lane, p.rot);
  order.store(sums[BACK ? group : 0], dw);
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
  for (int ch = threadIdx.x; ch < DIM; ch += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) v += sums[i][ch];
    partial[(int64_t)blockIdx.x * DIM + ch] = v;
  }
}

// ---- any head of up to 512 channels, any even rotation --------------------------------
// One warp a head, its vectors in shared memory as fp32, channels strided over
// the lanes: for head sizes and rotations that do not fit the layout above.
constexpr int kAnyWarps = 4;

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
    if (p.rot > 0) row = table_row(p, p.positions[token]);
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

// dw[side][c] = the sum of column c of the side's rows of partial, as 32 strided
// sums and those by halves: the same bits every time.
struct GradRows {
  const float* first;
  int rows, stride;
  float* dw;
};
struct GradRowsOf {
  GradRows side[2];
};
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const GradRowsOf of, int dim) {
  __shared__ float sh[32][33];
  const GradRows& r = of.side[blockIdx.y];
  if (r.dw == nullptr) return;
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + x;
  float v = 0.0f;
  for (int b = y; b < r.rows; b += 8 * 32) {
    float part[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      part[i] = c < dim && b + 32 * i < r.rows ? r.first[(int64_t)(b + 32 * i) * r.stride + c] : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += part[i];
  }
  sh[y][x] = v;
  __syncthreads();
  v = warp_sum(sh[x][y]);
  const int mine = blockIdx.x * 32 + y;
  if (x == 0 && mine < dim) r.dw[mine] = v;
}

// Heads of 64, 128 or 256 channels whose pairs fit the register layout (16384
// tokens of 40 heads of 128: 60 us so, 355 with the kernel for any size).
bool in_registers(const NormRopeParams& p) {
  return (p.dim == 64 || p.dim == 128 || p.dim == 256) && p.rot % 8 == 0;
}

NormRopeCut cut_of(int dtype, const NormRopeParams& p, bool back, int sm_count) {
  NormRopeCut cut;
  if (in_registers(p)) {
    const int rows = p.dim == 64 ? kRows<8> : p.dim == 128 ? kRows<16> : kRows<32>;
    const int per_sm = back ? kBwdBlocks * kBwdRuns : kFwdBlocks * kFwdRuns;
    int64_t blocks[2];
    for (int side = 0; side < 2; ++side) {
      const int64_t steps = (p.tokens * p.heads[side] + rows - 1) / rows;
      const int64_t share = (int64_t)sm_count * per_sm * p.heads[side] / (p.heads[0] + p.heads[1]);
      blocks[side] = 0;
      if (steps > 0) {
        const int64_t most = std::max<int64_t>(1, share);
        cut.per[side] = (steps + most - 1) / most;
        blocks[side] = (steps + cut.per[side] - 1) / cut.per[side];
        cut.by_heads[side] = FastDiv(p.heads[side]);
      }
    }
    cut.q_blocks = (int)blocks[0];
    cut.blocks = (int)(blocks[0] + blocks[1]);
    const int tokens = std::max(most_tokens(rows, p.heads[0]), most_tokens(rows, p.heads[1]));
    const int size = dtype == LBGEMM_F32 ? 4 : 2;
    cut.stage_bytes = rows * p.dim * size * (back ? 2 : 1) + tokens * p.rot * 4;
    // two stages at least (at most 96 KB), but none without use
    cut.stages = std::max(2, std::min(kMaxStages, (back ? kBwdRing : kFwdRing) / cut.stage_bytes));
    cut.stages = (int)std::min<int64_t>(cut.stages, std::max(cut.per[0], cut.per[1]));
  } else {
    const int64_t items = p.tokens * (p.heads[0] + p.heads[1]);
    cut.blocks = (int)std::min<int64_t>((items + kAnyWarps - 1) / kAnyWarps,
                                        (int64_t)sm_count * (back ? 4 : 16));
  }
  return cut;
}

template <typename T, int LPH, bool INTER, bool BACK>
cudaError_t launch_in_registers(const NormRopeParams& p, const NormRopeCut& cut, float* partial,
                                cudaStream_t s) {
  auto kernel = norm_rope_kernel<T, LPH, INTER, BACK>;
  static std::atomic<uint64_t> set{0};  // devices on which the kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(set.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
    if (e != cudaSuccess) return e;
    set |= uint64_t(1) << dev;
  }
  kernel<<<cut.blocks, kThreads + 32, cut.stages * cut.stage_bytes, s>>>(p, cut, partial);
  return cudaGetLastError();
}

template <typename T, int LPH>
cudaError_t launch_in_registers(const NormRopeParams& p, const NormRopeCut& cut, bool back,
                                float* partial, cudaStream_t s) {
  if (back)
    return p.interleaved ? launch_in_registers<T, LPH, true, true>(p, cut, partial, s)
                         : launch_in_registers<T, LPH, false, true>(p, cut, partial, s);
  return p.interleaved ? launch_in_registers<T, LPH, true, false>(p, cut, partial, s)
                       : launch_in_registers<T, LPH, false, false>(p, cut, partial, s);
}

template <typename T>
cudaError_t launch_typed(const NormRopeParams& p, const NormRopeCut& cut, bool back,
                         float* partial, cudaStream_t s) {
  if (in_registers(p)) {
    if (p.dim == 64) return launch_in_registers<T, 8>(p, cut, back, partial, s);
    if (p.dim == 128) return launch_in_registers<T, 16>(p, cut, back, partial, s);
    return launch_in_registers<T, 32>(p, cut, back, partial, s);
  }
  if (back)
    norm_rope_any_kernel<T, true>
        <<<cut.blocks, kAnyWarps * 32, kAnyWarps * 4 * p.dim * sizeof(float), s>>>(p, partial);
  else
    norm_rope_any_kernel<T, false>
        <<<cut.blocks, kAnyWarps * 32, kAnyWarps * p.dim * sizeof(float), s>>>(p, nullptr);
  return cudaGetLastError();
}

cudaError_t launch_any_type(int dtype, const NormRopeParams& p, const NormRopeCut& cut, bool back,
                            float* partial, cudaStream_t s) {
  if (dtype == LBGEMM_BF16) return launch_typed<__nv_bfloat16>(p, cut, back, partial, s);
  if (dtype == LBGEMM_F16) return launch_typed<__half>(p, cut, back, partial, s);
  return launch_typed<float>(p, cut, back, partial, s);
}

}  // namespace

cudaError_t launch_norm_rope(int dtype, const NormRopeParams& p, int sm_count, cudaStream_t s) {
  return launch_any_type(dtype, p, cut_of(dtype, p, false, sm_count), false, nullptr, s);
}

size_t norm_rope_scratch(int dtype, const NormRopeParams& p, int sm_count) {
  if (!p.side[0].w && !p.side[1].w) return 0;
  return (size_t)std::max(1, cut_of(dtype, p, true, sm_count).blocks) * 2 * p.dim * sizeof(float);
}

cudaError_t launch_norm_rope_backward(int dtype, const NormRopeParams& p, int sm_count,
                                      float* partial, int* launches, cudaStream_t s) {
  const NormRopeCut cut = cut_of(dtype, p, true, sm_count);
  if (cut.blocks > 0) {
    const cudaError_t e = launch_any_type(dtype, p, cut, true, partial, s);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  if (!partial) return cudaSuccess;
  GradRowsOf of;
  for (int side = 0; side < 2; ++side) {
    GradRows& r = of.side[side];
    r.dw = p.side[side].w ? p.side[side].dw : nullptr;
    if (in_registers(p)) {  // a row a block, the queries' blocks first
      r.first = partial + (side ? (int64_t)cut.q_blocks * p.dim : 0);
      r.rows = side ? cut.blocks - cut.q_blocks : cut.q_blocks;
      r.stride = p.dim;
    } else {  // every block a row for both sides
      r.first = partial + side * p.dim;
      r.rows = cut.blocks;
      r.stride = 2 * p.dim;
    }
  }
  norm_weight_grad_kernel<<<dim3((p.dim + 31) / 32, 2), 1024, 0, s>>>(of, p.dim);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace lbg
