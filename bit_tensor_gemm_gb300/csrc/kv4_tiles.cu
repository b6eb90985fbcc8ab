// kv4_tiles.cu -- attention over the 4-bit cache for many query rows (prompts,
// chunks of prompts): tiles of 256 rows on the tensor cores, tcgen05.mma with
// scores, weights and sums in tensor memory.
//
// A CTA (one an SM) holds the queries of two 128-row tiles X = 0, 1 in shared
// memory and walks over the cached tokens in steps of 128:
//
//   converters (4 warps)   codes of a step -> fp16 in shared memory, keys for
//                          S = Q K^T and values for O += P V, each once for
//                          both tiles; codes as subnormal halves code 2^-24
//                          (every second one 16 times that), as in kv4_rows.cu
//   one thread             the MMAs: O_X += P_X V of step j - 1, then S_X = Q_X
//                          K^T of step j, for X = 0, then 1
//   softmax (4 warps an X) a thread a row: weights 2^(t - ref) from S_X, times
//                          the value scales as fp16 back to tensor memory, over
//                          the S they came from
//
// While the tensor cores work for one tile, the other tile's softmax runs.
// Bound: the MMAs, 4 x 128 x DIM flops per row and step; the converters' and
// softmax's instructions (about 1.2 a code and 4 a score) must fit beside them,
// which is why both scales stay factors of columns, the weights need no maximum
// (the reference moves only when a product with a value scale leaves fp16's
// range, as in kv4_rows.cu), and arithmetic goes in pairs (f32x2).
#include <cuda_runtime.h>

#include <atomic>

#include "kv4_attention.cuh"
#include "kv4_codes.cuh"
#include "ptx.cuh"

namespace lbg {
namespace {

constexpr int kThreads = 512;  // warps 0..3, 4..7 softmax, 8..11 converters, 12 MMAs
constexpr int kStep = kStepTokens;
constexpr int kMinSteps = 4;
constexpr int kScaleSlots = 4;

template <int DIM>
struct Smem {
  static constexpr int kTile = kStep * DIM * 2;  // bytes of 128 rows of fp16
  static constexpr int kQ = 0;                   // [2] queries
  static constexpr int kK = kQ + 2 * kTile;      // [2] keys
  static constexpr int kV = kK + 2 * kTile;      // [2] values
  static constexpr int kScales = kV + 2 * kTile; // [4][2][128] fp32: keys' x factor, values'
  static constexpr int kBars = kScales + kScaleSlots * 2 * kStep * 4;
  static constexpr int kNumBars = 8 + kScaleSlots + 1 + 7;
  static constexpr int kMisc = kBars + 8 * kNumBars;
  static constexpr int kBytes = kMisc + 64 + 1024;  // slack to align to 1024
};

// Chunk j (16 bytes) of row r of a 128-byte-swizzled block of rows of 128 bytes.
__device__ __forceinline__ uint32_t swizzled(int r, int j) {
  return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4));
}

// Descriptor of an operand whose rows (tokens) are the K dimension and whose
// 64 elements of a row the other one: blocks of 64 elements `block` bytes
// apart, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_rows_k(uint32_t addr, uint32_t block) {
  uint64_t d = smem_desc_sw128(addr);
  d &= ~((uint64_t)0x3FFF << 16);
  d |= (uint64_t)(block >> 4) << 16;
  return d;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Walks the steps of a run: which tile, head and step of the tile.
struct Cursor {
  int seq_tile, head, off;
  RowTile t;
  __device__ __forceinline__ void start(const Kv4AttnParams& p, const Run& run) {
    seq_tile = run.seq_tile;
    head = run.head;
    off = run.off;
    t = row_tile(p, seq_tile);
  }
  // to the next tile of the row of steps (the caller knows that there is one)
  __device__ __forceinline__ void next_tile(const Kv4AttnParams& p) {
    off = 0;
    if (++head == p.cache.heads) {
      head = 0;
      do t = row_tile(p, ++seq_tile);
      while (t.steps == 0);
    }
  }
};

// The steps of a tile that the rows of half X see: [from, to) within the tile.
struct HalfTile {
  int rows, from, to;
};
__device__ __forceinline__ HalfTile half_tile(const Kv4AttnParams& p, const RowTile& t, int x) {
  HalfTile h;
  h.rows = min(128, t.rows - 128 * x);
  h.from = h.to = 0;
  if (h.rows <= 0) {
    h.rows = 0;
    return h;
  }
  const int r0 = t.r0 + 128 * x;
  const int i0 = (int)p.by_group((uint32_t)r0), i1 = (int)p.by_group((uint32_t)(r0 + h.rows - 1));
  const int last = min(t.last, last_seen(p, t, i1));
  const int first = max(t.first, first_seen(p, last_seen(p, t, i0)));
  if (last > first) {
    h.from = (first - t.base) / kStep;
    h.to = (last - t.base + kStep - 1) / kStep;
  }
  return h;
}

template <typename T, int DIM>
__global__ void __launch_bounds__(kThreads, 1) kv4_tiles_kernel(const Kv4AttnParams p) {
  using S = Smem<DIM>;
  constexpr int kBlock = kStep * 128;
  constexpr uint32_t kIdescS = instr_desc(128, kStep);
  constexpr uint32_t kIdescO = instr_desc(128, DIM) | (1u << 16);  // B's rows are the K dimension
  constexpr uint32_t kColO = 256;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem), bar0 = sbase + S::kBars;
  auto k_full = [&](int i) { return bar0 + 8u * i; };
  auto k_empty = [&](int i) { return bar0 + 8u * (2 + i); };
  auto v_full = [&](int i) { return bar0 + 8u * (4 + i); };
  auto v_empty = [&](int i) { return bar0 + 8u * (6 + i); };
  auto scale_full = [&](int i) { return bar0 + 8u * (8 + i); };
  const uint32_t q_full = bar0 + 8u * (8 + kScaleSlots);
  auto s_full = [&](int x) { return q_full + 8u + 8u * x; };
  auto p_full = [&](int x) { return q_full + 24u + 8u * x; };
  auto o_full = [&](int x) { return q_full + 40u + 8u * x; };
  const uint32_t drain = q_full + 56u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);
  float* factor_slot = reinterpret_cast<float*>(smem + S::kMisc + 8);
  float* most_slots = reinterpret_cast<float*>(smem + S::kMisc + 16);  // [8]
  float* scales = reinterpret_cast<float*>(smem + S::kScales);

  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full(i), 128);
      mbar_init(k_empty(i), 1);
      mbar_init(v_full(i), 128);
      mbar_init(v_empty(i), 1);
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 128);
      mbar_init(o_full(i), 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) mbar_init(scale_full(i), 128);
    mbar_init(q_full, 256);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  const Run run = find_run<kThreads>(p, kMinSteps);  // (with a barrier of the block)
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (p.joins > 0 && !p.by_tile && threadIdx.x == 0) p.join[blockIdx.x].last_cta = -1;

  bool dead = false;
  auto wait = [&](uint32_t bar, uint32_t phase) {
    if (!dead) dead = !mbar_wait(bar, phase & 1u, abort_flag, p.status);
  };
  // the same for all lanes of a warp, which go on together
  auto warp_wait = [&](uint32_t bar, uint32_t phase) {
    wait(bar, phase);
    dead = __any_sync(0xffffffffu, dead);
  };

  if (warp >= 12) {
    // ---------------- the MMAs: one thread ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 12 && lane == 0 && run.count > 0) {
      Cursor c;
      c.start(p, run);
      uint32_t step = 0, tile = 0;      // of the run: steps so far, tiles so far
      uint32_t n_p[2] = {0, 0};         // weights of half X consumed so far
      for (int done = 0; done < run.count; ++tile) {
        const int count = min(c.t.steps - c.off, run.count - done);
        int from[2], to[2];  // of each half, in steps of this piece
        for (int x = 0; x < 2; ++x) {
          const HalfTile h = half_tile(p, c.t, x);
          from[x] = min(max(h.from - c.off, 0), count);
          to[x] = min(max(h.to - c.off, from[x]), count);
        }
        wait(q_full, tile);
        for (int j = 0; j <= count; ++j) {
          const uint32_t sj = step + j, sv = step + j - 1;  // run steps of the keys, values
          bool have_k = false, have_v = false;
          for (int x = 0; x < 2; ++x) {
            if (j > from[x] && j <= to[x]) {  // O_X += P_X V of step j - 1
              if (!have_v) wait(v_full(sv & 1), sv >> 1);
              have_v = true;
              wait(p_full(x), n_p[x]++);
              if (!dead) {
                tc_fence_after();
                const uint32_t vbase = sbase + S::kV + (sv & 1) * S::kTile;
#pragma unroll
                for (int k = 0; k < kStep / 16; ++k)
                  mma_f16_ts(tmem + kColO + 128 * x, tmem + 128 * x + 8 * k,
                             smem_desc_rows_k(vbase + 2048 * k, kBlock), kIdescO,
                             j - 1 > from[x] || k > 0);
                if (j == to[x]) mma_commit(o_full(x));
              }
            }
            if (j >= from[x] && j < to[x]) {  // S_X = Q_X K^T of step j
              if (!have_k) wait(k_full(sj & 1), sj >> 1);
              have_k = true;
              if (!dead) {
                tc_fence_after();
                const uint32_t qbase = sbase + S::kQ + x * S::kTile;
                const uint32_t kbase = sbase + S::kK + (sj & 1) * S::kTile;
#pragma unroll
                for (int k = 0; k < DIM / 16; ++k) {
                  const uint32_t at = (k / 4) * kBlock + (k % 4) * 32;
                  mma_f16(tmem + 128 * x, smem_desc_sw128(qbase + at), smem_desc_sw128(kbase + at),
                          kIdescS, k > 0);
                }
                mma_commit(s_full(x));
              }
            }
          }
          // (a step that neither half sees is converted all the same: its
          // barriers are passed on)
          if (j > 0) {
            if (!have_v) wait(v_full(sv & 1), sv >> 1);
            if (!dead) mma_commit(v_empty(sv & 1));
          }
          if (j < count) {
            if (!have_k) wait(k_full(sj & 1), sj >> 1);
            if (!dead) mma_commit(k_empty(sj & 1));
          }
        }
        step += count;
        done += count;
        if (done < run.count) c.next_tile(p);
      }
      // every MMA and commit has ended before the block does (with a limit, also
      // after a wait that ran out)
      volatile int go_on = 0;
      mma_commit(drain);
      mbar_wait(drain, 0, &go_on, p.status);
    }
  } else if (warp >= 8) {
    // ---------------- converters ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // lane -> 32 codes (16 bytes) of a token: LPT lanes a token, tokens whose
    // low three bits differ across a phase of 8 lanes (no bank conflicts)
    constexpr int LPT = DIM / 32, TPL = 32 / LPT, LOADS = 32 / TPL;
    const int cw = warp - 8, ctid = threadIdx.x - 256;
    const int row0 = cw * 32 + lane % TPL, chunk = lane / TPL;
    const int page_size = (int)p.cache.page_size;
    const uint32_t page16 = (uint32_t)page_size / 16;
    const int64_t block_bytes = kv4_block_bytes(DIM, page_size);
    Cursor c;
    if (run.count > 0) c.start(p, run);
    int tile_steps = 0;
    // this warp's two groups of 16 tokens: block of the page and token in it
    auto find = [&](const uint8_t* (&block)[2], int (&inside)[2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int token = c.t.base + c.off * kStep + cw * 32 + h * 16;
        block[h] = nullptr;
        inside[h] = 0;
        if (token >= c.t.last) continue;
        const uint32_t group = (uint32_t)token / 16, in_table = p.by_page16(group);
        const int page = __ldg(p.page_table + (int64_t)c.t.b * p.table_width + in_table);
        if ((uint32_t)page >= (uint32_t)p.cache.pages) {
          if (lane == 0) atomicOr(p.status, kStatusBadIndex);
          continue;
        }
        block[h] = p.cache.base + ((int64_t)page * p.cache.heads + c.head) * block_bytes;
        inside[h] = (int)(group - in_table * page16) * 16;
      }
    };
    uint4 raw_k[LOADS], raw_v[LOADS];
    uint32_t raw_s = 0;  // scales of token ctid: key, value << 16
    auto load = [&](const uint8_t* const (&block)[2], const int (&inside)[2]) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int r = lane % TPL + i * TPL, h = r / 16;  // token of the warp's 32
        raw_k[i] = raw_v[i] = make_uint4(0, 0, 0, 0);
        if (block[h] == nullptr) continue;
        const uint8_t* at = block[h] + (inside[h] + r % 16) * (DIM / 2) + chunk * 16;
        raw_k[i] = __ldg(reinterpret_cast<const uint4*>(at));
        raw_v[i] = __ldg(reinterpret_cast<const uint4*>(at + (int64_t)page_size * (DIM / 2)));
      }
      raw_s = 0;
      const uint8_t* b = lane < 16 ? block[0] : block[1];
      if (b) {
        const uint16_t* at = reinterpret_cast<const uint16_t*>(b + (int64_t)page_size * DIM) +
                             (lane < 16 ? inside[0] : inside[1]) + lane % 16;
        raw_s = (uint32_t)__ldg(at) | (uint32_t)__ldg(at + page_size) << 16;
      }
    };
    auto convert = [&](uint32_t dst, const uint4 (&raw)[LOADS]) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int r = row0 + i * TPL;
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t w8 = w[k] >> 8;
          const int at = chunk * 4 + k;
          st_shared_v4(dst + (at / 8) * kBlock + swizzled(r, at % 8), (int)codes0<false>(w[k]),
                       (int)codes0<true>(w[k]), (int)codes0<false>(w8), (int)codes0<true>(w8));
        }
      }
    };
    uint32_t tile = 0;
    const uint8_t* block[2];
    int inside[2];
    if (run.count > 0) {
      find(block, inside);
      load(block, inside);
    }
    float factor = 0.0f;
    for (int s = 0; s < run.count; ++s) {
      if (tile_steps == 0) {  // a new tile: its queries' factor
        tile_steps = min(c.t.steps - c.off, run.count - s);
        wait(q_full, tile++);
        factor = *reinterpret_cast<volatile float*>(factor_slot);
      }
      --tile_steps;
      // on to the next step, and its pages
      const uint8_t* next_block[2] = {nullptr, nullptr};
      int next_inside[2] = {0, 0};
      if (s + 1 < run.count) {
        if (++c.off == c.t.steps) c.next_tile(p);
        find(next_block, next_inside);
      }
      const int st = s & 1, use = s >> 1;
      float* sc = scales + (s % kScaleSlots) * 2 * kStep;
      sc[ctid] = __uint_as_float(raw_s << 16) * factor;
      sc[kStep + ctid] = __uint_as_float(raw_s & 0xffff0000u);
      mbar_arrive(scale_full(s % kScaleSlots));
      if (use > 0) wait(k_empty(st), use - 1);
      convert(sbase + S::kK + st * S::kTile, raw_k);
      fence_proxy_async_smem();
      mbar_arrive(k_full(st));
      if (use > 0) wait(v_empty(st), use - 1);
      convert(sbase + S::kV + st * S::kTile, raw_v);
      fence_proxy_async_smem();
      mbar_arrive(v_full(st));
      load(next_block, next_inside);
    }
  } else {
    // ---------------- softmax: thread = row ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int x = warp / 4, r = threadIdx.x;  // row of the 256
    const uint32_t lane_base = (uint32_t)(32 * (warp % 4)) << 16;
    const uint32_t ts = tmem + lane_base + 128 * x, to_ = tmem + lane_base + kColO + 128 * x;
    Cursor c;
    if (run.count > 0) c.start(p, run);
    uint32_t step = 0, n_s = 0, n_o = 0;
    for (int done = 0; done < run.count;) {
      const RowTile& t = c.t;
      const int count = min(t.steps - c.off, run.count - done);
      const HalfTile h = half_tile(p, t, x);
      const bool live = r < t.rows;
      const int qi = (int)p.by_group((uint32_t)(t.r0 + min(r, t.rows - 1)));
      // ---- queries to shared memory: fp16 times the tile's power of two (its
      // largest element goes to 2^14 .. 2^15), in the codes' order, those of odd
      // codes divided by 16.  (Every MMA of the tile before has ended.)
      {
        const T* src = static_cast<const T*>(p.q) + (int64_t)(t.q0 + qi) * p.q_stride +
                       (int64_t)(c.head * p.group + t.r0 + min(r, t.rows - 1) - qi * p.group) * DIM;
        float most = 0.0f;
#pragma unroll 4
        for (int i = 0; i < DIM / 8; ++i) {
          float v[8];
          load8(src + 8 * i, v);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (fabsf(v[k]) < INFINITY) most = fmaxf(most, fabsf(v[k]));
        }
#pragma unroll
        for (int i = 16; i >= 1; i >>= 1)
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, i));
        asm volatile("bar.sync 1, 256;" ::: "memory");  // (the slots' last readers are done)
        if (lane == 0) most_slots[warp] = most;
        asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll
        for (int i = 0; i < 8; ++i) most = fmaxf(most, most_slots[i]);
        int k2 = 0;
        if (most > 0.0f) k2 = min(max(14 - ((int)(__float_as_uint(most) >> 23) - 127), -103), 126);
        const float up = __uint_as_float((uint32_t)(127 + k2) << 23), up16 = up * 0.0625f;
        if (r == 0)
          *factor_slot = __uint_as_float((uint32_t)(127 + 24 - k2) << 23) * (p.scale * kLog2e);
        const uint32_t dst = sbase + S::kQ + x * S::kTile;
#pragma unroll 4
        for (int i = 0; i < DIM / 8; ++i) {
          float v[8];
          load8(src + 8 * i, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = live ? v[k] * (k & 1 ? up16 : up) : 0.0f;
          st_shared_v4(dst + (i / 8) * kBlock + swizzled(r % 128, i % 8), (int)pack_f16(v[0], v[4]),
                       (int)pack_f16(v[1], v[5]), (int)pack_f16(v[2], v[6]),
                       (int)pack_f16(v[3], v[7]));
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
      }
      // ---- the steps that this half sees
      const int from = min(max(h.from - c.off, 0), count);
      const int upto = min(max(h.to - c.off, from), count);
      const int seen_to = min(t.last, last_seen(p, t, qi));
      const int seen_from = max(t.first, first_seen(p, last_seen(p, t, qi)));
      // tokens that every row of the half sees
      const int hr0 = t.r0 + 128 * x;
      const int all_to = min(t.last, last_seen(p, t, (int)p.by_group((uint32_t)hr0)));
      const int all_from = max(t.first, first_seen(p, last_seen(p, t, (int)p.by_group(
                                            (uint32_t)(hr0 + max(h.rows, 1) - 1)))));
      float ref = -3.0e38f, m = -3.0e38f, l = 0.0f, wtop = 0.0f;
      for (int j = from; j < upto; ++j) {
        const uint32_t slot = (step + j) % kScaleSlots;
        warp_wait(scale_full(slot), (step + j) / kScaleSlots);
        warp_wait(s_full(x), n_s++);
        if (dead) break;
        tc_fence_after();
        const float* ks = scales + slot * 2 * kStep;
        const float* vs = ks + kStep;
        const int token0 = t.base + (c.off + j) * kStep;
        const bool masked = token0 < all_from || token0 + kStep > all_to;
        bool again = masked;
        if (!masked) {
          float sv[4][32];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, reinterpret_cast<uint32_t(&)[32]>(sv[q]));
          tmem_ld_wait();
          uint32_t pw[2][32];
          const uint64_t nref = pair(-ref, -ref);
          uint64_t sum0 = 0, sum1 = 0;
          __half2 most = __half2half2(__half(0.0f));
#pragma unroll
          for (int i = 0; i < 32; ++i) {  // four tokens
            const float* s4 = &sv[i / 8][i % 8 * 4];
            const ulonglong2 k4 = reinterpret_cast<const ulonglong2*>(ks)[i];
            const ulonglong2 v4 = reinterpret_cast<const ulonglong2*>(vs)[i];
            float x0, x1, x2, x3;
            unpair(fma2(pair(s4[0], s4[1]), k4.x, nref), x0, x1);
            unpair(fma2(pair(s4[2], s4[3]), k4.y, nref), x2, x3);
            const uint64_t p0 = pair(ex2(x0), ex2(x1)), p1 = pair(ex2(x2), ex2(x3));
            sum0 = add2(sum0, p0);
            sum1 = add2(sum1, p1);
            float w0, w1, w2, w3;
            unpair(mul2(p0, v4.x), w0, w1);
            unpair(mul2(p1, v4.y), w2, w3);
            const __half2 h0 = __floats2half2_rn(w0, w1), h1 = __floats2half2_rn(w2, w3);
            most = __hmax2(most, __hmax2(__habs2(h0), __habs2(h1)));
            pw[i / 16][i % 16 * 2] = *reinterpret_cast<const uint32_t*>(&h0);
            pw[i / 16][i % 16 * 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
          }
          float a, b, sum;
          unpair(add2(sum0, sum1), a, b);
          sum = a + b;
          again = sum > kFar || !__hble2(most, __half2half2(__half(32768.0f)));
          again = __any_sync(0xffffffffu, again);
          if (!again) {
            l += sum;
            tmem_st32(ts, pw[0]);
            tmem_st32(ts + 32, pw[1]);
          }
        }
        if (again) {
          // masked scores, or weights out of range: with care, 32 tokens at a time
          float high = m;
          auto hidden = [&](int token) { return token >= seen_to || token < seen_from; };
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t v[32];
            tmem_ld32(ts + 32 * q, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int n = 32 * q + i;
              if (!hidden(token0 + n)) high = fmaxf(high, __uint_as_float(v[i]) * ks[n]);
            }
          }
          float top = wtop * ex2(m - high);
          const float before = top;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t v[32];
            tmem_ld32(ts + 32 * q, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int n = 32 * q + i;
              if (!hidden(token0 + n))
                top = fmaxf(top, fabsf(ex2(__uint_as_float(v[i]) * ks[n] - high) * vs[n]));
            }
          }
          float next = ref;
          if (high > m || top > before) {
            const float lead = fminf(fmaxf(top, kLeastTop), 1.0e30f);
            next = high - (float)(10 - ((int)(__float_as_uint(lead) >> 23) - 127));
          }
          m = high;
          wtop = top;
          const float f = ex2(ref - next);
          const bool moved = next != ref;
          ref = next;
          l *= f;
          // (S of this step was committed after O += P V of the step before)
          if (j > from && __any_sync(0xffffffffu, moved)) {
#pragma unroll 1
            for (int q = 0; q < DIM / 32; ++q) {
              uint32_t v[32];
              tmem_ld32(to_ + 32 * q, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
              tmem_st32(to_ + 32 * q, v);
            }
          }
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t v[32], w[16];
            tmem_ld32(ts + 32 * q, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float w2[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int n = 32 * q + i + e;
                const float pj = hidden(token0 + n) ? 0.0f : ex2(fmaf(__uint_as_float(v[i + e]), ks[n], -ref));
                l += pj;
                // what a row does not see has weight 0 whatever its scale
                w2[e] = hidden(token0 + n) ? 0.0f : pj * vs[n];
              }
              w[i / 2] = pack_f16(w2[0], w2[1]);
            }
            tmem_st16(ts + 16 * q, w);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full(x));
      }
      // ---- the rows' results
      const bool whole = count == t.steps;
      const bool none = l == 0.0f;
      const float inv = none ? 0.0f : 1.0f / l;
      const float lse = none ? -INFINITY : ref + log2f(l);
      if (upto > from) {
        warp_wait(o_full(x), n_o++);
        tc_fence_after();
      }
      if (p.joins > 0 && c.off == 0 && (!whole || p.by_tile) && threadIdx.x == 0) {
        const int64_t last = (run.pos + done + t.steps - 1) / run.per;  // the CTA of its last step
        p.join[p.by_tile ? c.seq_tile * p.cache.heads + c.head : (int)blockIdx.x] =
            Kv4Join{c.seq_tile, c.head, (int)blockIdx.x, whole ? -1 : (int)last};
      }
      const int64_t share = ((int64_t)blockIdx.x * 2 + (c.off == 0)) * p.tile_rows + r;
      const int64_t at = out_row(p, t, c.head, t.r0 + min(r, t.rows - 1));
      if (h.rows > 0 && !dead) {
#pragma unroll 1
        for (int q = 0; q < DIM / 32; ++q) {
          uint32_t v[32];
          if (upto > from) {
            tmem_ld32(to_ + 32 * q, v);
            tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // columns 8 i .. of the accumulator are channels 0, 4, 1, 5, 2, 6, 3, 7 of
            // eight, in units of 2^-24 (2^-20 for odd codes)
            float ch[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int d = k / 2 + (k & 1) * 4;
              ch[d] = none ? 0.0f
                           : __uint_as_float(v[8 * i + k]) * ((d & 1 ? 1048576.0f : 16777216.0f) * inv);
            }
            if (!live) continue;
            if (whole) store8(static_cast<T*>(p.o) + at * DIM + 32 * q + 8 * i, ch);
            else store8(p.share_o + share * DIM + 32 * q + 8 * i, ch);
          }
        }
        if (live) {
          if (whole) {
            if (p.lse) p.lse[at] = lse * kLn2;
          } else {
            p.share_lse[share] = lse;
          }
        }
      }
      step += count;
      done += count;
      if (done < run.count) c.next_tile(p);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int DIM>
cudaError_t launch_tile(const Kv4AttnParams& p, cudaStream_t s) {
  auto kernel = kv4_tiles_kernel<T, DIM>;
  static std::atomic<uint64_t> set{0};  // devices on which the kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(set.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<DIM>::kBytes);
    if (e != cudaSuccess) return e;
    set |= uint64_t(1) << dev;
  }
  kernel<<<p.ctas, kThreads, Smem<DIM>::kBytes, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_tiles(int dtype, const Kv4AttnParams& p, cudaStream_t s) {
  if (dtype == LBGEMM_BF16)
    return p.cache.dim == 64 ? launch_tile<__nv_bfloat16, 64>(p, s)
                             : launch_tile<__nv_bfloat16, 128>(p, s);
  return p.cache.dim == 64 ? launch_tile<__half, 64>(p, s) : launch_tile<__half, 128>(p, s);
}

}  // namespace lbg
