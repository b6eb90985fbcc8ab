// residual_norm.cu -- the norms after and before a block with its gate and the
// residual stream, and the backward pass.
//
//   z  = y r1 post (or y),      r1 = (mean(y^2) + eps)^-1/2
//   x' = a x + b gate z
//   n  = x' r2 next,            r2 = (mean(x'^2) + eps)^-1/2
// backward, with xhat = x' r2, yhat = y r1:
//   d  = dx' + r2 (next dn - xhat mean(next dn xhat))        dnext = sum dn xhat
//   dx = a d,  dz = b gate d,  dgate = b z d                 dpost = sum dz yhat
//   dy = r1 (post dz - yhat mean(post dz yhat))  (or dz)
//
// Some ten operations an element against 8 bytes moved (12 backward): bound by
// HBM.  One pass over the rows: they come by bulk copies into a ring of stages in
// shared memory, a few rows ahead, so that the bytes in flight do not depend on
// registers; x' is computed anew from x and y in the backward pass, in fp32, so
// nothing but the inputs is kept for it.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "attn_common.cuh"
#include "ffn.h"
#include "ptx.cuh"

namespace lbg {
namespace {

constexpr int kMaxStages = 4;
// Blocks an SM is to hold and the shared memory each may take for its ring.
constexpr int kFwdBlocks = 3, kBwdBlocks = 2;
constexpr int kFwdRing = 70 * 1024, kBwdRing = 108 * 1024;
constexpr int kMostRing = 220 * 1024;  // where one stage alone is more than that

struct NormCut {
  int blocks = 0, stages = 0, stage_bytes = 0;
  int groups = 0;  // rows of a stage
};

template <typename T>
struct Vec {
  float2x v[4];
};
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* p) {
  float f[8];
  unpack8(load8_raw(p), f);
  return {{pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7])}};
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const Vec<T>& x) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpair(x.v[i], f[2 * i], f[2 * i + 1]);
  store8(p, f);
}
template <typename T>
__device__ __forceinline__ Vec<T> ones() {
  const float2x o = pair(1.0f, 1.0f);
  return {{o, o, o, o}};
}
__device__ __forceinline__ float halves(float2x v) {
  float lo, hi;
  unpair(v, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ float2x twice(float v) { return pair(v, v); }

// Sums of one or two numbers over a row's WPR warps; every thread of the row gets
// them, in the same order.  `slots`: [2][16] floats of the row, another half for
// consecutive calls (so one barrier is enough).
template <int WPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* slots, int warp) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
  if constexpr (WPR > 1) {
    if (threadIdx.x % 32 == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) slots[i * 16 + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = slots[i * 16];
#pragma unroll
      for (int w = 1; w < WPR; ++w) s += slots[i * 16 + w];
      v[i] = s;
    }
  }
}

// WPR warps a row, VPT vectors of 8 elements a thread.  The tensors of a stage:
// x (if any), y, one row of gates each, dx', dn; each [groups][width].
template <typename T, int WPR, int VPT, bool BACK>
__global__ void __launch_bounds__(WPR <= 8 ? 256 : 512)
    residual_norm_kernel(const ResidualNormParams p, const NormCut cut,
                         float* __restrict__ partial) {
  constexpr int THREADS = WPR <= 8 ? 256 : 512;
  constexpr int LANES = 32 * WPR, GROUPS = THREADS / LANES;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t bars[kMaxStages];
  __shared__ int abort_flag;
  __shared__ float slots[3][GROUPS][32];
  const int group = threadIdx.x / LANES, at = threadIdx.x % LANES, warp = at / 32;
  const int width = p.width, vectors = width / 8;
  const int row_bytes = width * (int)sizeof(T);
  const bool own_gate = p.gate && p.gate_stride != 0;
  const float inv = 1.0f / (float)width;

  // which tensors a stage holds, and where
  const void* src[5];
  int64_t stride[5];
  int held = 0, at_x = -1, at_y = -1, at_gate = -1, at_dx = -1, at_dn = -1;
  auto hold = [&](const void* q, int64_t s, int& where) {
    if (!q) return;
    src[held] = q;
    stride[held] = s;
    where = held++;
  };
  hold(p.x, p.x_stride, at_x);
  hold(p.y, p.y_stride, at_y);
  if (own_gate) hold(p.gate, p.gate_stride, at_gate);
  if (BACK) hold(p.dx_out, p.dx_out_stride, at_dx);
  if (BACK) hold(p.dn, p.dn_stride, at_dn);

  const int64_t steps_all = (p.tokens + GROUPS - 1) / GROUPS;
  const int64_t step0 = blockIdx.x, stride_steps = gridDim.x;
  if (threadIdx.x < cut.stages) {
    mbar_init(smem_addr(bars) + 8 * threadIdx.x, 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  auto issue = [&](int64_t step, int slot) {  // by the first warp
    const int rows = (int)min((int64_t)GROUPS, p.tokens - step * GROUPS);
    const uint32_t bar = smem_addr(bars) + 8 * slot;
    const uint32_t dst = smem_addr(ring) + slot * cut.stage_bytes;
    if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, (uint32_t)(rows * held * row_bytes));
    __syncwarp();
    for (int i = threadIdx.x; i < rows * held; i += 32) {
      const int t = i / rows, r = i - t * rows;
      const void* base = src[0];
      int64_t st = stride[0];
#pragma unroll
      for (int k = 1; k < 5; ++k)
        if (k < held && t == k) base = src[k], st = stride[k];
      bulk_load(dst + (t * GROUPS + r) * row_bytes,
                static_cast<const T*>(base) + (step * GROUPS + r) * st, row_bytes, bar);
    }
  };
  if (threadIdx.x < 32)
    for (int s = 0; s < cut.stages; ++s)
      if (step0 + s * stride_steps < steps_all) issue(step0 + s * stride_steps, s);

  Vec<T> sum_post[BACK ? VPT : 1], sum_next[BACK ? VPT : 1], sum_gate[BACK ? VPT : 1];
  if (BACK) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) sum_post[j] = sum_next[j] = sum_gate[j] = {{0, 0, 0, 0}};
  }
  const T* post = static_cast<const T*>(p.post);
  const T* next = static_cast<const T*>(p.next);
  const float2x a2 = twice(p.a), b2 = twice(p.b);

  int slot = 0, parity = 0;
  for (int64_t step = step0; step < steps_all; step += stride_steps) {
    // every warp leaves together where the copies do not come
    const bool ok = mbar_wait(smem_addr(bars) + 8 * slot, parity, &abort_flag, p.status);
    if (!__syncthreads_and(ok)) break;
    const int64_t row = step * GROUPS + group;
    const bool live = row < p.tokens;  // (a row past the end computes what is there, stores nothing)
    const uint8_t* stage = ring + slot * cut.stage_bytes + group * row_bytes;
    auto part = [&](int which, int v) {
      return load_vec(reinterpret_cast<const T*>(stage + which * GROUPS * row_bytes) + v * 8);
    };
    auto gates = [&](int v) {
      return own_gate ? part(at_gate, v)
                      : p.gate ? load_vec(static_cast<const T*>(p.gate) + v * 8) : ones<T>();
    };
    float r1 = 1.0f;
    if (post) {
      float2x s = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = at + j * LANES;
        if (v < vectors) {
          const Vec<T> y = part(at_y, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) s = fma2(y.v[i], y.v[i], s);
        }
      }
      float t[1] = {halves(s)};
      row_sums<WPR>(t, slots[0][group], warp);
      r1 = rsqrtf(t[0] * inv + p.eps);
    }
    const float2x r1x = twice(r1);
    // x' of a vector; yhat and what the gate multiplies on the way
    auto stream = [&](int v, Vec<T>& yhat, Vec<T>& z, Vec<T>& g) {
      Vec<T> x = at_x >= 0 ? part(at_x, v) : Vec<T>{{0, 0, 0, 0}};
#pragma unroll
      for (int i = 0; i < 4; ++i) x.v[i] = mul2(x.v[i], a2);
      if (at_y < 0) return x;
      yhat = part(at_y, v);
      z = yhat;
      if (post) {
        const Vec<T> w = load_vec(post + v * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          yhat.v[i] = mul2(yhat.v[i], r1x);
          z.v[i] = mul2(yhat.v[i], w.v[i]);
        }
      }
      g = gates(v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g.v[i] = mul2(g.v[i], b2);
        x.v[i] = fma2(g.v[i], z.v[i], x.v[i]);
      }
      return x;
    };
    float2x s = 0, dot = 0;
    Vec<T> yhat, z, g;
    Vec<T> kept[VPT];  // x'
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = at + j * LANES;
      if (v >= vectors) continue;
      kept[j] = stream(v, yhat, z, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) s = fma2(kept[j].v[i], kept[j].v[i], s);
      if (BACK && next) {
        const Vec<T> w = load_vec(next + v * 8), dn = part(at_dn, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) dot = fma2(mul2(w.v[i], dn.v[i]), kept[j].v[i], dot);
      }
      if (!BACK && p.x_out && live)
        store_vec(static_cast<T*>(p.x_out) + row * p.x_out_stride + v * 8, kept[j]);
    }
    float r2 = 0.0f, mean2 = 0.0f;
    if (next) {
      float t[2] = {halves(s), halves(dot)};
      row_sums<WPR>(t, slots[1][group], warp);
      r2 = rsqrtf(t[0] * inv + p.eps);
      mean2 = r2 * (t[1] * inv);  // mean(next dn xhat)
    }
    const float2x r2x = twice(r2);
    if (!BACK) {
      if (next) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const int v = at + j * LANES;
          if (v >= vectors) continue;
          const Vec<T> w = load_vec(next + v * 8);
#pragma unroll
          for (int i = 0; i < 4; ++i) kept[j].v[i] = mul2(mul2(kept[j].v[i], r2x), w.v[i]);
          if (live) store_vec(static_cast<T*>(p.n_out) + row * p.n_out_stride + v * 8, kept[j]);
        }
      }
    } else {
      const float2x m2 = twice(-mean2);
      float2x dot1 = 0;
      Vec<T> wdz[VPT];  // post dz
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = at + j * LANES;
        if (v >= vectors) continue;
        stream(v, yhat, z, g);
        Vec<T> d = at_dx >= 0 ? part(at_dx, v) : Vec<T>{{0, 0, 0, 0}};
        if (next) {
          const Vec<T> w = load_vec(next + v * 8), dn = part(at_dn, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2x xhat = mul2(kept[j].v[i], r2x);
            if (live) sum_next[j].v[i] = fma2(dn.v[i], xhat, sum_next[j].v[i]);
            d.v[i] = fma2(r2x, fma2(xhat, m2, mul2(w.v[i], dn.v[i])), d.v[i]);
          }
        }
        if (p.dx && live) {
          Vec<T> dx;
#pragma unroll
          for (int i = 0; i < 4; ++i) dx.v[i] = mul2(d.v[i], a2);
          store_vec(static_cast<T*>(p.dx) + row * p.dx_stride + v * 8, dx);
        }
        if (at_y < 0) continue;
        if (p.dgate) {
          Vec<T> dg;
#pragma unroll
          for (int i = 0; i < 4; ++i) dg.v[i] = mul2(mul2(d.v[i], b2), z.v[i]);
          if (own_gate) {
            if (live) store_vec(static_cast<T*>(p.dgate) + row * p.dgate_stride + v * 8, dg);
          } else if (live) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sum_gate[j].v[i] = add2(sum_gate[j].v[i], dg.v[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) d.v[i] = mul2(d.v[i], g.v[i]);  // (the gate times b)
        if (post) {
          const Vec<T> w = load_vec(post + v * 8);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (live) sum_post[j].v[i] = fma2(d.v[i], yhat.v[i], sum_post[j].v[i]);
            wdz[j].v[i] = mul2(w.v[i], d.v[i]);
            dot1 = fma2(wdz[j].v[i], yhat.v[i], dot1);
          }
        } else if (live) {
          store_vec(static_cast<T*>(p.dy) + row * p.dy_stride + v * 8, d);
        }
      }
      if (post) {
        float t[1] = {halves(dot1)};
        row_sums<WPR>(t, slots[2][group], warp);
        const float2x m1 = twice(-t[0] * inv);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const int v = at + j * LANES;
          if (v >= vectors) continue;
          Vec<T> y = part(at_y, v);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y.v[i] = mul2(r1x, fma2(mul2(y.v[i], r1x), m1, wdz[j].v[i]));
          if (live) store_vec(static_cast<T*>(p.dy) + row * p.dy_stride + v * 8, y);
        }
      }
    }
    // the stage is read: copy the row that comes `stages` steps later over it
    __syncthreads();
    const int64_t later = step + cut.stages * stride_steps;
    if (threadIdx.x < 32 && later < steps_all) issue(later, slot);
    if (++slot == cut.stages) slot = 0, parity ^= 1;
  }
  if (abort_flag) {  // let the copies in flight land (again with a limit)
    volatile int go_on = 0;
    if (threadIdx.x == 0)
      for (int i = 0; i < cut.stages; ++i) {
        mbar_wait(smem_addr(bars) + 8 * slot, parity, &go_on, p.status, kWaitLimitNs / 8);
        if (++slot == cut.stages) slot = 0, parity ^= 1;
      }
    return;
  }
  if constexpr (BACK) {
    if (!partial) return;
    // the row of sums of this block and group: post, next, gate
    float* mine = partial + ((int64_t)blockIdx.x * GROUPS + group) * 3 * width;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = at + j * LANES;
      if (v >= vectors) continue;
      auto put = [&](int which, const Vec<T>& x) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) unpair(x.v[i], f[2 * i], f[2 * i + 1]);
        store8<float>(mine + (int64_t)which * width + v * 8, f);
      };
      if (p.dpost) put(0, sum_post[j]);
      if (p.dnext) put(1, sum_next[j]);
      if (p.dgate && !own_gate) put(2, sum_gate[j]);
    }
  }
}

// out[i][c] = the sum over rows of partial[row][i][c]: 32 strided sums and those by
// halves, the same bits every time.
struct SumOut {
  float* out[3];
};
__global__ void __launch_bounds__(1024)
    residual_norm_sums_kernel(const float* __restrict__ partial, int rows, int width,
                              const SumOut to) {
  __shared__ float sh[32][33];
  float* out = blockIdx.y == 0 ? to.out[0] : blockIdx.y == 1 ? to.out[1] : to.out[2];
  if (!out) return;
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + x;
  float v = 0.0f;
  for (int b = y; b < rows; b += 8 * 32) {
    float part[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      part[i] = c < width && b + 32 * i < rows
                    ? partial[((int64_t)(b + 32 * i) * 3 + blockIdx.y) * width + c]
                    : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += part[i];
  }
  sh[y][x] = v;
  __syncthreads();
  v = sh[x][y];
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  const int mine = blockIdx.x * 32 + y;
  if (x == 0 && mine < width) out[mine] = v;
}

int warps_per_row(int width) {
  const int vectors = width / 8;
  for (int w = 1; w < 16; w *= 2)
    if (vectors <= 32 * w) return w;
  return 16;
}

NormCut cut_of(int dtype, const ResidualNormParams& p, bool back, int sm_count) {
  NormCut cut;
  const int wpr = warps_per_row(p.width);
  cut.groups = wpr <= 8 ? 8 / wpr : 1;
  const int held = (p.x != nullptr) + (p.y != nullptr) + (p.gate && p.gate_stride != 0) +
                   (back && p.dx_out) + (back && p.dn);
  const int64_t steps = (p.tokens + cut.groups - 1) / cut.groups;
  cut.stage_bytes = cut.groups * p.width * (dtype == LBGEMM_F32 ? 4 : 2) * std::max(held, 1);
  const int per_sm = back ? kBwdBlocks : kFwdBlocks;
  cut.blocks = (int)std::min<int64_t>(steps, (int64_t)sm_count * per_sm);
  cut.stages = std::min(kMaxStages, (back ? kBwdRing : kFwdRing) / cut.stage_bytes);
  if (cut.stages < 2) cut.stages = std::max(1, std::min(2, kMostRing / cut.stage_bytes));
  if (cut.blocks > 0)
    cut.stages = (int)std::min<int64_t>(cut.stages, (steps + cut.blocks - 1) / cut.blocks);
  return cut;
}

template <typename T, int WPR, int VPT, bool BACK>
cudaError_t launch(const ResidualNormParams& p, const NormCut& cut, float* partial,
                   cudaStream_t s) {
  auto kernel = residual_norm_kernel<T, WPR, VPT, BACK>;
  static std::atomic<uint64_t> set{0};  // devices on which the kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(set.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostRing);
    if (e != cudaSuccess) return e;
    set |= uint64_t(1) << dev;
  }
  kernel<<<cut.blocks, WPR <= 8 ? 256 : 512, cut.stages * cut.stage_bytes, s>>>(p, cut, partial);
  return cudaGetLastError();
}

template <typename T, bool BACK>
cudaError_t launch_typed(const ResidualNormParams& p, const NormCut& cut, float* partial,
                         cudaStream_t s) {
  switch (warps_per_row(p.width)) {
    case 1: return launch<T, 1, 1, BACK>(p, cut, partial, s);
    case 2: return launch<T, 2, 1, BACK>(p, cut, partial, s);
    case 4: return launch<T, 4, 1, BACK>(p, cut, partial, s);
    case 8: return launch<T, 8, 1, BACK>(p, cut, partial, s);
    default: break;
  }
  if (p.width <= 4096) return launch<T, 16, 1, BACK>(p, cut, partial, s);
  if (p.width <= 8192) return launch<T, 16, 2, BACK>(p, cut, partial, s);
  if constexpr (sizeof(T) == 2) return launch<T, 16, 4, BACK>(p, cut, partial, s);
  return cudaErrorInvalidValue;
}

template <bool BACK>
cudaError_t launch_any(int dtype, const ResidualNormParams& p, const NormCut& cut, float* partial,
                       cudaStream_t s) {
  if (dtype == LBGEMM_BF16) return launch_typed<__nv_bfloat16, BACK>(p, cut, partial, s);
  if (dtype == LBGEMM_F16) return launch_typed<__half, BACK>(p, cut, partial, s);
  return launch_typed<float, BACK>(p, cut, partial, s);
}

bool sums(const ResidualNormParams& p) {
  return p.dpost || p.dnext || (p.dgate && p.gate_stride == 0);
}

}  // namespace

cudaError_t launch_residual_norm(int dtype, const ResidualNormParams& p, int sm_count,
                                 cudaStream_t s) {
  return launch_any<false>(dtype, p, cut_of(dtype, p, false, sm_count), nullptr, s);
}

size_t residual_norm_scratch(int dtype, const ResidualNormParams& p, int sm_count) {
  if (!sums(p)) return 0;
  const NormCut cut = cut_of(dtype, p, true, sm_count);
  return (size_t)std::max(1, cut.blocks * cut.groups) * 3 * p.width * sizeof(float);
}

cudaError_t launch_residual_norm_backward(int dtype, const ResidualNormParams& p, int sm_count,
                                          float* partial, int* launches, cudaStream_t s) {
  const NormCut cut = cut_of(dtype, p, true, sm_count);
  if (cut.blocks > 0) {
    const cudaError_t e = launch_any<true>(dtype, p, cut, partial, s);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  if (!sums(p)) return cudaSuccess;
  SumOut to = {{p.dpost, p.dnext, p.gate_stride == 0 ? static_cast<float*>(p.dgate) : nullptr}};
  residual_norm_sums_kernel<<<dim3((p.width + 31) / 32, 3), 1024, 0, s>>>(
      partial, cut.blocks * cut.groups, p.width, to);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace lbg
