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
//
// Measured, bf16, every output: 8192 rows of 4096 in 55 us forward (4.9 TB/s; issue slots
// three quarters full, as a word of two numbers takes some ten instructions an operand) and
// 124 backward (3.3 TB/s, at 126 registers a thread); of 8192 in 104 and 238; 8192 x 4096 of
// fp32 in 97 and 160 (5.5 and 5.0 TB/s).
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
constexpr int kRing = 216 * 1024;
// ... where one stage alone is more than that (seven rows of 32 KB: up to five tensors in
// a stage and the weights that are not among them)
__host__ __device__ constexpr int most_ring(int vpt) { return (vpt > 1 ? 224 : 220) * 1024; }
__host__ __device__ constexpr int blocks_for(int wpr, int vpt, bool back) {
  return back ? (wpr <= 8 ? 2 : 1) : vpt > 1 ? (wpr == 12 ? 2 : 1) : wpr <= 8 ? 4 : 2;
}
__host__ __device__ constexpr int threads_for(int wpr) { return wpr <= 8 ? 256 : 32 * wpr; }

// Warps and vectors a thread of a row, and rows that are taken at once.
struct Shape {
  int wpr, vpt, rows;
};
// A backward pass with several vectors a thread keeps the weights in shared memory: its
// sums take the registers (8192 x 8192: 416 us with spills, 238 without).
__host__ __device__ constexpr bool weights_aside(int vpt, bool back) { return back && vpt > 1; }
struct NormCut {
  Shape shape = {};
  int blocks = 0, stages = 0, stage_bytes = 0, aside_bytes = 0;
};

// Two numbers; as plain fp32 operations, since the paired ones of this file's other
// kind cost more in moves here than they save (8192 rows of 4096: 75 against 65 us).
struct Two {
  float a, b;
};
__device__ __forceinline__ Two two(float a, float b) { return {a, b}; }
__device__ __forceinline__ Two fma2(Two x, Two y, Two z) {
  return {fmaf(x.a, y.a, z.a), fmaf(x.b, y.b, z.b)};
}
__device__ __forceinline__ Two mul2(Two x, Two y) { return {x.a * y.a, x.b * y.b}; }
__device__ __forceinline__ Two add2(Two x, Two y) { return {x.a + y.a, x.b + y.b}; }
template <typename T>
struct Vec {
  Two v[4];
};
template <typename T>
__device__ __forceinline__ Vec<T> vec_of(const Raw8<T>& r) {
  float f[8];
  unpack8(r, f);
  return {{two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7])}};
}
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* p) {
  return vec_of(load8_raw(p));
}
template <typename T>
__device__ __forceinline__ void store8_raw(T* p, const Raw8<T>& r) {
  reinterpret_cast<uint4*>(p)[0] = r.v[0];
  if constexpr (sizeof(T) == 4) reinterpret_cast<uint4*>(p)[1] = r.v[1];
}
__device__ __forceinline__ uint32_t round2(float lo, float hi, __nv_bfloat16) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t round2(float lo, float hi, __half) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const Vec<T>& x) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = x.v[i].a, f[2 * i + 1] = x.v[i].b;
  if constexpr (sizeof(T) == 4) {
    store8(p, f);
  } else {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(round2(f[0], f[1], T()), round2(f[2], f[3], T()), round2(f[4], f[5], T()),
                   round2(f[6], f[7], T()));
  }
}
__device__ __forceinline__ float halves(Two v) { return v.a + v.b; }
__device__ __forceinline__ Two twice(float v) { return two(v, v); }

// The WPR warps of a row meet; true where any of them asks to stop.
template <int WPR>
__device__ __forceinline__ bool row_meet(int group, bool stop) {
  if constexpr (WPR == 1) {
    return __any_sync(0xffffffffu, stop);
  } else {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %3, 0;\n\t"
        "barrier.cta.red.or.aligned.pred q, %1, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(group + 1), "n"(32 * WPR), "r"((int)stop)
        : "memory");
    return r != 0;
  }
}

// Sums of one or two numbers over a row's warps; every thread of the row gets them, in
// the same order.  `slots`: [2][16] floats of the row, others for consecutive calls (so
// one meeting is enough).
template <int WPR, int N>
__device__ __forceinline__ bool row_sums(float (&v)[N], float* slots, int group, int warp,
                                         bool stop = false) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
  if constexpr (WPR > 1) {
    if (threadIdx.x % 32 == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) slots[i * 16 + warp] = v[i];
  }
  stop = row_meet<WPR>(group, stop);
  if constexpr (WPR > 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      constexpr int PLACES = WPR == 12 ? 16 : WPR;
      const int place = threadIdx.x % PLACES;
      v[i] = place < WPR ? slots[i * 16 + place] : 0.0f;
#pragma unroll
      for (int off = PLACES / 2; off >= 1; off >>= 1)
        v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    }
  }
  return stop;
}

// WPR warps a row, VPT vectors of 8 elements a thread, ROWS rows at once (a meeting of
// the warps costs the same for one and two); the first warp issues the
// copies (a warp of its own would leave fewer registers to the others).  The tensors of
// a stage: x, y, a gate for each row, dx', dn, those that are given; each [rows][width].
template <typename T, int WPR, int VPT, int ROWS, bool BACK>
__global__ void __launch_bounds__(threads_for(WPR), blocks_for(WPR, VPT, BACK))
    residual_norm_kernel(const ResidualNormParams p, const NormCut cut,
                         float* __restrict__ partial) {
  constexpr int THREADS = threads_for(WPR);
  constexpr int LANES = 32 * WPR, GROUPS = THREADS / LANES, HELD = GROUPS * ROWS;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t bars[2 * kMaxStages];
  __shared__ int abort_flag;
  __shared__ float slots[4][GROUPS][ROWS * 32];
  const int group = threadIdx.x / LANES, at = threadIdx.x % LANES, warp = at / 32;
  const int width = p.width, vectors = width / 8;
  const int row_bytes = width * (int)sizeof(T);
  const bool own_gate = p.gate && p.gate_stride != 0;
  const float inv = 1.0f / (float)width;

  // the tensors of a stage, in order
  const int at_x = 0, at_y = p.y ? 1 : -1;
  int held = p.y ? 2 : 1;
  const int at_gate = own_gate ? held++ : -1;
  const int at_dx = BACK && p.dx_out ? held++ : -1;
  const int at_dn = BACK && p.dn ? held++ : -1;

  const int64_t steps_all = (p.tokens + HELD - 1) / HELD;
  const int64_t step0 = blockIdx.x, stride_steps = gridDim.x;
  const uint32_t full = smem_addr(bars), empty = full + 8 * kMaxStages;
  if (threadIdx.x < cut.stages) {
    mbar_init(full + 8 * threadIdx.x, 1);
    mbar_init(empty + 8 * threadIdx.x, THREADS / 32);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();

  auto issue = [&](int64_t step, int slot) {  // by the first warp
    const int rows = (int)min((int64_t)HELD, p.tokens - step * HELD);
    const uint32_t bar = full + 8 * slot, dst = smem_addr(ring) + slot * cut.stage_bytes;
    if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, (uint32_t)(rows * held * row_bytes));
    __syncwarp();
    for (int i = threadIdx.x; i < held * HELD; i += 32) {
      const int t = i / HELD, r = i % HELD;
      const void* from = p.x;
      int64_t stride = p.x_stride;
      if (t == at_y) from = p.y, stride = p.y_stride;
      if (t == at_gate) from = p.gate, stride = p.gate_stride;
      if (t == at_dx) from = p.dx_out, stride = p.dx_out_stride;
      if (t == at_dn) from = p.dn, stride = p.dn_stride;
      if (r < rows)
        bulk_load(dst + i * row_bytes, static_cast<const T*>(from) + (step * HELD + r) * stride,
                  row_bytes, bar);
    }
  };
  // The copy into a slot that all warps are to have read by now; `use`: how often the
  // slot has been filled before.
  auto refill = [&](int64_t step, int slot, int use) {
    if (threadIdx.x >= 32 || step >= steps_all) return;
    if (__all_sync(0xffffffffu, mbar_wait(empty + 8 * slot, (use - 1) & 1, &abort_flag, p.status)))
      issue(step, slot);
  };
  if (threadIdx.x < 32)
    for (int s = 0; s < cut.stages; ++s)
      if (step0 + s * stride_steps < steps_all) issue(step0 + s * stride_steps, s);

  // weights of this thread's columns, as they are in memory
  constexpr bool ASIDE = weights_aside(VPT, BACK);
  constexpr int W = ASIDE ? 1 : VPT;
  Raw8<T> w_post[W], w_next[W], w_gate[W];
  const bool one_gate = p.gate && !own_gate, next = p.next != nullptr, post = p.post != nullptr;
  // [post, next, gate][width], those that are given; a thread reads what it has written
  T* const aside = reinterpret_cast<T*>(ring + cut.stages * cut.stage_bytes);
  const int aside_next = post ? width : 0, aside_gate = aside_next + (next ? width : 0);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = min(at + j * LANES, vectors - 1);
    Raw8<T> raw[3];
    if (post) raw[0] = load8_raw(static_cast<const T*>(p.post) + v * 8);
    if (next) raw[1] = load8_raw(static_cast<const T*>(p.next) + v * 8);
    if (one_gate) raw[2] = load8_raw(static_cast<const T*>(p.gate) + v * 8);
    if constexpr (ASIDE) {
      if (at + j * LANES >= vectors) continue;
      if (post) store8_raw(aside + v * 8, raw[0]);
      if (next) store8_raw(aside + aside_next + v * 8, raw[1]);
      if (one_gate) store8_raw(aside + aside_gate + v * 8, raw[2]);
    } else {
      w_post[j] = raw[0], w_next[j] = raw[1], w_gate[j] = raw[2];
    }
  }
  auto weight = [&](const Raw8<T>* raw, int offset, int j) -> Vec<T> {
    if constexpr (ASIDE)
      return load_vec(aside + offset + (at + j * LANES) * 8);
    else
      return vec_of(raw[j]);
  };
  auto post_of = [&](int j) { return weight(w_post, 0, j); };
  auto next_of = [&](int j) { return weight(w_next, aside_next, j); };
  Vec<T> sum_post[BACK ? VPT : 1], sum_next[BACK ? VPT : 1], sum_gate[BACK ? VPT : 1];
  if (BACK) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) sum_post[j] = sum_next[j] = sum_gate[j] = {};
  }
  const Two a2 = twice(p.a), b2 = twice(p.b);
  // Vector q is vector q % VPT of row q / VPT.  With one a thread, what a row's later
  // passes need stays in registers; with more it is taken from the stage again.
  constexpr int Q = ROWS * VPT;
  constexpr bool KEEP = Q == 1;

  int slot = 0, use = 0;  // the slot of a row, and how often it has been used before
  bool odd = false;
  for (int64_t step = step0; step < steps_all; step += stride_steps) {
    // (where the copies do not come, the warps of a row leave together below)
    bool stop = !mbar_wait(full + 8 * slot, use & 1, &abort_flag, p.status);
    const int64_t row = step * HELD + group * ROWS;
    // (a row past the end computes what is there, stores nothing)
    auto live = [&](int q) { return HELD == 1 || row + q / VPT < p.tokens; };
    const T* stage =
        reinterpret_cast<const T*>(ring + slot * cut.stage_bytes + group * ROWS * row_bytes);
    auto column = [&](int q) { return (at + q % VPT * LANES) * 8; };
    auto part = [&](int which, int q) {
      return load_vec(stage + ((which * HELD + q / VPT) * width + column(q)));
    };
    auto on = [&](int q) { return at + q % VPT * LANES < vectors; };

    // ---- rstd(Y) ----
    Vec<T> y[Q];  // KEEP: Y, then Y rstd(Y)
    float r1[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) r1[r] = 1.0f;
    if (at_y >= 0) {
      Two s[ROWS] = {};
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if (!on(q)) continue;
        y[q] = part(at_y, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[q / VPT] = fma2(y[q].v[i], y[q].v[i], s[q / VPT]);
      }
      if (post) {
        float t[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) t[r] = halves(s[r]);
        // (a forward pass without a second norm meets once a row: places in turn)
        stop = row_sums<WPR>(t, slots[odd ? 3 : 0][group], group, warp, stop);
        odd = !odd;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) r1[r] = rsqrtf(t[r] * inv + p.eps);
      }
    }
    if (!post) stop = row_meet<WPR>(group, stop);
    if (stop) break;
    // the slot of the rows before, for those `stages` steps after them
    if (cut.stages > 1 && step > step0)
      refill(step + (cut.stages - 1) * stride_steps, slot == 0 ? cut.stages - 1 : slot - 1,
             slot == 0 ? use : use + 1);

    // ---- x', its rstd, mean(next dn xhat) ----
    Vec<T> z[Q], g[Q], kept[Q], dn[Q];  // z; b gate; x'; dn
    // y = Y rstd(Y), z and b gate of a vector; Y again where it was not kept
    auto block = [&](int q) {
      if (!KEEP) y[q] = part(at_y, q);
      z[q] = y[q];
      if (post) {
        const Two r = twice(r1[q / VPT]);
        const Vec<T> w = post_of(q % VPT);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[q].v[i] = mul2(y[q].v[i], r);
          z[q].v[i] = mul2(y[q].v[i], w.v[i]);
        }
      }
      if (p.gate) {
        g[q] = own_gate ? part(at_gate, q) : weight(w_gate, aside_gate, q % VPT);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[q].v[i] = mul2(g[q].v[i], b2);
      } else {
        g[q] = {{b2, b2, b2, b2}};
      }
    };
    Two s[ROWS] = {}, dot[ROWS] = {};
    T* const to_x = !BACK && p.x_out ? static_cast<T*>(p.x_out) + row * p.x_out_stride : nullptr;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (!on(q)) continue;
      kept[q] = part(at_x, q);
#pragma unroll
      for (int i = 0; i < 4; ++i) kept[q].v[i] = mul2(kept[q].v[i], a2);
      if (at_y >= 0) {
        block(q);
#pragma unroll
        for (int i = 0; i < 4; ++i) kept[q].v[i] = fma2(g[q].v[i], z[q].v[i], kept[q].v[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[q / VPT] = fma2(kept[q].v[i], kept[q].v[i], s[q / VPT]);
      if (BACK && next) {
        const Vec<T> w = next_of(q % VPT);
        dn[q] = part(at_dn, q);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dot[q / VPT] = fma2(mul2(w.v[i], dn[q].v[i]), kept[q].v[i], dot[q / VPT]);
      }
      if (to_x && live(q)) store_vec(to_x + q / VPT * p.x_out_stride + column(q), kept[q]);
    }
    float r2[ROWS], mean2[ROWS];  // mean2: mean(next dn xhat)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) r2[r] = mean2[r] = 0.0f;
    if (next) {
      constexpr int N = BACK ? 2 * ROWS : ROWS;
      float t[N];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        t[r] = halves(s[r]);
        if (BACK) t[N - ROWS + r] = halves(dot[r]);
      }
      row_sums<WPR>(t, slots[1][group], group, warp);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        r2[r] = rsqrtf(t[r] * inv + p.eps);
        mean2[r] = r2[r] * (t[N - ROWS + r] * inv);
      }
    }

    if constexpr (!BACK) {
      // ---- n ----
      if (next) {
        T* const to = static_cast<T*>(p.n_out) + row * p.n_out_stride;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          if (!on(q)) continue;
          const Two r = twice(r2[q / VPT]);
          const Vec<T> w = next_of(q % VPT);
#pragma unroll
          for (int i = 0; i < 4; ++i) kept[q].v[i] = mul2(mul2(kept[q].v[i], r), w.v[i]);
          if (live(q)) store_vec(to + q / VPT * p.n_out_stride + column(q), kept[q]);
        }
      }
    } else {
      // ---- d, dx, dgate, dz ----
      Two dot1[ROWS] = {};
      T* const to_dx = static_cast<T*>(p.dx) + row * p.dx_stride;
      T* const to_dy = static_cast<T*>(p.dy) + row * p.dy_stride;
      T* const to_gate = static_cast<T*>(p.dgate) + (own_gate ? row * p.dgate_stride : 0);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if (!on(q)) continue;
        const int j = q % VPT;
        Vec<T> d = at_dx >= 0 ? part(at_dx, q) : Vec<T>{};
        if (next) {
          const Two r = twice(r2[q / VPT]), m = twice(-mean2[q / VPT]);
          const Vec<T> w = next_of(j);
          if (!KEEP) dn[q] = part(at_dn, q);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const Two xhat = mul2(kept[q].v[i], r);
            if (live(q)) sum_next[j].v[i] = fma2(dn[q].v[i], xhat, sum_next[j].v[i]);
            d.v[i] = fma2(r, fma2(xhat, m, mul2(w.v[i], dn[q].v[i])), d.v[i]);
          }
        }
        if (live(q)) {
          Vec<T> dx;
#pragma unroll
          for (int i = 0; i < 4; ++i) dx.v[i] = mul2(d.v[i], a2);
          store_vec(to_dx + q / VPT * p.dx_stride + column(q), dx);
        }
        if (at_y < 0) continue;
        if (!KEEP) block(q);
        if (p.gate) {
          Vec<T> dg;
#pragma unroll
          for (int i = 0; i < 4; ++i) dg.v[i] = mul2(mul2(d.v[i], b2), z[q].v[i]);
          if (own_gate) {
            if (live(q)) store_vec(to_gate + q / VPT * p.dgate_stride + column(q), dg);
          } else if (live(q)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sum_gate[j].v[i] = add2(sum_gate[j].v[i], dg.v[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) d.v[i] = mul2(d.v[i], g[q].v[i]);  // dz
        if (post) {
          const Vec<T> w = post_of(j);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (live(q)) sum_post[j].v[i] = fma2(d.v[i], y[q].v[i], sum_post[j].v[i]);
            kept[q].v[i] = mul2(w.v[i], d.v[i]);  // (x' has done its part)
            dot1[q / VPT] = fma2(kept[q].v[i], y[q].v[i], dot1[q / VPT]);
          }
        } else if (live(q)) {
          store_vec(to_dy + q / VPT * p.dy_stride + column(q), d);
        }
      }
      // ---- dy ----
      if (post) {
        float t[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) t[r] = halves(dot1[r]);
        row_sums<WPR>(t, slots[2][group], group, warp);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          if (!on(q)) continue;
          const Two r = twice(r1[q / VPT]), m = twice(-t[q / VPT] * inv);
          if (!KEEP) {
            y[q] = part(at_y, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[q].v[i] = mul2(y[q].v[i], r);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) y[q].v[i] = mul2(r, fma2(y[q].v[i], m, kept[q].v[i]));
          if (live(q)) store_vec(to_dy + q / VPT * p.dy_stride + column(q), y[q]);
        }
      }
    }
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(empty + 8 * slot);
    if (cut.stages == 1) refill(step + stride_steps, 0, use + 1);
    if (++slot == cut.stages) slot = 0, ++use;
  }
  if (__syncthreads_or(abort_flag)) {
    // Let the copies in flight land (again with a limit): those of the slots from this
    // row's on.
    volatile int go_on = 0;
    if (threadIdx.x == 0)
      for (int i = 0; i < cut.stages; ++i) {
        mbar_wait(full + 8 * slot, use & 1, &go_on, p.status, kWaitLimitNs / 8);
        if (++slot == cut.stages) slot = 0, ++use;
      }
    return;
  }
  if constexpr (BACK) {
    if (!partial) return;
    // the row of sums of this block: post, next, gate.  Several groups add theirs in shared
    // memory, in order (the ring is theirs now: a stage holds two rows a group at least, so
    // its bytes are a row of fp32 sums for each).
    float* mine = partial + (int64_t)blockIdx.x * 3 * width;
    float* const joined = reinterpret_cast<float*>(ring);
    auto put = [&](int which, const Vec<T>* sum) {
      if constexpr (GROUPS > 1) __syncthreads();
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = at + j * LANES;
        if (v >= vectors) continue;
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = sum[j].v[i].a, f[2 * i + 1] = sum[j].v[i].b;
        store8<float>((GROUPS > 1 ? joined + group * width : mine + which * width) + v * 8, f);
      }
      if constexpr (GROUPS > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < width; c += THREADS) {
          float f = joined[c];
#pragma unroll
          for (int g = 1; g < GROUPS; ++g) f += joined[g * width + c];
          mine[which * width + c] = f;
        }
      }
    };
    if (p.dpost) put(0, sum_post);
    if (p.dnext) put(1, sum_next);
    if (p.dgate && !own_gate) put(2, sum_gate);
  }
}

// out[i][c] = the sum over rows of partial[row][i][c]: 32 strided sums and those by
// halves, the same bits every time.
struct SumOut {
  float* out[3];
};
__global__ void __launch_bounds__(256)
    residual_norm_sums_kernel(const float* __restrict__ partial, int rows, int width,
                              const SumOut to) {
  __shared__ float4 sh[32][8];
  float* out = blockIdx.y == 0 ? to.out[0] : blockIdx.y == 1 ? to.out[1] : to.out[2];
  if (!out) return;
  const int x = threadIdx.x % 8, y = threadIdx.x / 8;
  const int c = blockIdx.x * 32 + 4 * x;
  float4 v = make_float4(0, 0, 0, 0);
  if (c < width) {
    const float* from = partial + (int64_t)blockIdx.y * width + c;
#pragma unroll 5
    for (int b = y; b < rows; b += 32) {
      const float4 q = *reinterpret_cast<const float4*>(from + (int64_t)b * 3 * width);
      v.x += q.x;
      v.y += q.y;
      v.z += q.z;
      v.w += q.w;
    }
  }
  sh[y][x] = v;
  for (int half = 16; half >= 1; half /= 2) {
    __syncthreads();
    if (y < half) {
      const float4 q = sh[y + half][x];
      v.x += q.x;
      v.y += q.y;
      v.z += q.z;
      v.w += q.w;
      sh[y][x] = v;
    }
  }
  if (y == 0 && c < width) *reinterpret_cast<float4*>(out + c) = v;
}

int groups_of(int wpr) { return wpr <= 8 ? 8 / wpr : 1; }

// How a call is cut with a shape; `roomy` tells whether two stages fit a block's share of
// an SM.
NormCut cut_with(const Shape& shape, int dtype, const ResidualNormParams& p, bool back,
                 int sm_count, bool* roomy) {
  NormCut cut;
  cut.shape = shape;
  const int row_bytes = p.width * (dtype == LBGEMM_F32 ? 4 : 2);
  const int rows = groups_of(shape.wpr) * shape.rows;
  const int held = (p.x != nullptr) + (p.y != nullptr) + (p.gate && p.gate_stride != 0) +
                   (back && p.dx_out) + (back && p.dn);
  const int64_t steps = (p.tokens + rows - 1) / rows;
  cut.stage_bytes = rows * row_bytes * std::max(held, 1);
  if (weights_aside(shape.vpt, back))
    cut.aside_bytes = ((p.post != nullptr) + (p.next != nullptr) +
                       (p.gate && p.gate_stride == 0)) * row_bytes;
  const int per_sm = blocks_for(shape.wpr, shape.vpt, back);
  cut.blocks = (int)std::min<int64_t>(steps, (int64_t)sm_count * per_sm);
  cut.stages = std::min(kMaxStages, (kRing / per_sm - cut.aside_bytes) / cut.stage_bytes);
  *roomy = cut.stages >= 2;
  if (cut.stages < 2)
    cut.stages = std::max(
        1, std::min(2, (most_ring(shape.vpt) - cut.aside_bytes) / cut.stage_bytes));
  if (cut.blocks > 0)
    cut.stages = (int)std::min<int64_t>(cut.stages, (steps + cut.blocks - 1) / cut.blocks);
  return cut;
}

NormCut cut_of(int dtype, const ResidualNormParams& p, bool back, int sm_count) {
  const int vectors = p.width / 8;
  int wpr = 1;
  while (wpr < 16 && vectors > 32 * wpr) wpr *= 2;
  bool roomy = false;
  // Where every group has several rows and two stages of them fit: two rows at once, or
  // (backward, wide rows) two vectors a thread and two blocks an SM.  8192 x 4096 backward:
  // 124 us, two rows at once 131, one 145; 65536 x 512: 55 and 142 us with two rows, 71 and
  // 159 with one; with a single stage 2048 x 1000 of fp32 takes 33 us backward, not 17.
  if (vectors <= 512 && p.tokens >= 8 * (int64_t)groups_of(wpr) * sm_count) {
    const Shape shape = back && wpr == 16 ? Shape{8, 2, 1} : Shape{wpr, 1, 2};
    const NormCut cut = cut_with(shape, dtype, p, back, sm_count, &roomy);
    if (roomy) return cut;
  }
  Shape shape = {wpr, 1, 1};
  // (8192 x 5120: forward 84 us, with 16 warps 93, backward 181 against 205; forward of
  // fp32 spills so, 4096 x 6144: 75 against 69)
  if (vectors > 512)
    shape = vectors <= 768 && (back || dtype != LBGEMM_F32)
                ? Shape{12, 2, 1}
                : Shape{16, vectors <= 1024 ? 2 : 4, 1};
  return cut_with(shape, dtype, p, back, sm_count, &roomy);
}

template <typename T, int WPR, int VPT, int ROWS, bool BACK>
cudaError_t launch(const ResidualNormParams& p, const NormCut& cut, float* partial,
                   cudaStream_t s) {
  auto kernel = residual_norm_kernel<T, WPR, VPT, ROWS, BACK>;
  static std::atomic<uint64_t> set{0};  // devices on which the kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(set.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             most_ring(VPT));
    if (e != cudaSuccess) return e;
    set |= uint64_t(1) << dev;
  }
  kernel<<<cut.blocks, threads_for(WPR), cut.stages * cut.stage_bytes + cut.aside_bytes, s>>>(
      p, cut, partial);
  return cudaGetLastError();
}

template <typename T, bool BACK>
cudaError_t launch_typed(const ResidualNormParams& p, const NormCut& cut, float* partial,
                         cudaStream_t s) {
  const Shape& shape = cut.shape;
  if (shape.rows == 2) {
    switch (shape.wpr) {
      case 1: return launch<T, 1, 1, 2, BACK>(p, cut, partial, s);
      case 2: return launch<T, 2, 1, 2, BACK>(p, cut, partial, s);
      case 4: return launch<T, 4, 1, 2, BACK>(p, cut, partial, s);
      case 8: return launch<T, 8, 1, 2, BACK>(p, cut, partial, s);
      default: break;
    }
    if constexpr (!BACK) return launch<T, 16, 1, 2, BACK>(p, cut, partial, s);
    return cudaErrorInvalidValue;
  }
  switch (shape.wpr) {
    case 1: return launch<T, 1, 1, 1, BACK>(p, cut, partial, s);
    case 2: return launch<T, 2, 1, 1, BACK>(p, cut, partial, s);
    case 4: return launch<T, 4, 1, 1, BACK>(p, cut, partial, s);
    case 8:
      if constexpr (BACK)
        if (shape.vpt == 2) return launch<T, 8, 2, 1, BACK>(p, cut, partial, s);
      return launch<T, 8, 1, 1, BACK>(p, cut, partial, s);
    case 12:
      if constexpr (BACK || sizeof(T) == 2) return launch<T, 12, 2, 1, BACK>(p, cut, partial, s);
      return cudaErrorInvalidValue;
    default: break;
  }
  if (shape.vpt == 1) return launch<T, 16, 1, 1, BACK>(p, cut, partial, s);
  if (shape.vpt == 2) return launch<T, 16, 2, 1, BACK>(p, cut, partial, s);
  if constexpr (sizeof(T) == 2) return launch<T, 16, 4, 1, BACK>(p, cut, partial, s);
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
  return (size_t)std::max(1, cut.blocks) * 3 * p.width * sizeof(float);
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
  residual_norm_sums_kernel<<<dim3((p.width + 31) / 32, 3), 256, 0, s>>>(
      partial, cut.blocks, p.width, to);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace lbg
