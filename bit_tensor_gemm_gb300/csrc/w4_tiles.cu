// w4_tiles.cu -- products with 4-bit weights for many tokens, on tcgen05: tiles
// of 128 or 256 weight rows by up to 256 tokens.
//
//   linear  Y[m][n] = row_scale[n] * sum_k X[m][k] * (code * scale)[n][k]
//   up      h[pos][i] = silu(gate) * up for the picks (token, expert) in expert order
//   down    out[pos][n], which combine() adds up by token
//
// The weights are the MMA's A operand, read from tensor memory: converter warps
// turn a slice of 128 codes a row into halves (exactly, w4_codes.cuh), a row a
// lane, and store them into a slot of tensor memory.  Tokens are the B
// operand, brought by TMA (128-byte swizzle).  So shared memory carries a quarter of
// the weights' bytes of a product of halves, and is bound by the tokens: from 65
// tokens on a tile is a pair of CTAs' (cta_group::2, 128 weight rows in each), which
// halves the tokens that each of them brings and reads (4096 tokens x 11008 x 4096: 317 us
// with single CTAs of 128 x 256, at the rate of their fills, 258 with pairs).
//
// One persistent CTA an SM: warps for TMA of the codes (0), the MMAs (1, of a pair
// the even CTA's), TMA of the tokens (2), read-out (4..11), converters (12 on: four
// teams, of long slices three, that take slices in turn, a warp a quarter of the rows).
// The MMAs' warp goes through its loop with all lanes: operands that are the same in a
// warp stay in uniform registers, and an MMA is issued every 46 cycles; with one lane in
// the loop it was 99, and up to 128 tokens were bound by that.  Tiles of
// up to 128 tokens have two accumulators, so that a tile is read out beside the next
// one's MMAs.  A reader has a row a lane and turns 32 tokens through shared memory
// into vectors along the rows.  A linear layer with few tiles is cut along k and joined by join().
//
// Measured beyond L2: 4096 tokens x 11008 x 4096 in 215 us (1.71 PFLOP/s, what a plain product
// of 16-bit numbers reaches being 1.90), 64 x 19456 x 8192 in 25 us (3.4 TB/s of weights), 12 x
// 4096 x 11008 in 13.4; 4096 tokens, 6 of 64 experts of 2048 / 1024, in 350 us (0.87
// PFLOP/s: blocks of tokens three quarters full; 67 us of sorting, gathering and joining).
//
// In a pair the full barriers and the accumulators' empty ones are the even CTA's and
// count both; the commits of the MMAs go to both.  Every
// wait is bounded; on a time-out the CTAs wind down (copies in flight, own MMAs)
// before tensor memory is freed.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "attn_common.cuh"
#include "cluster.cuh"
#include "ffn.h"
#include "ptx.cuh"
#include "w4_codes.cuh"
#include "w4_kernels.h"

namespace lbg {
namespace {

constexpr int kReaders = 8;          // warps that read accumulators out
constexpr int kReadBytes = 32 * 80;  // a reader's room to turn 32 tokens of 32 rows: 64 bytes and a pad each
constexpr int kRows = 128;    // weight rows of a tile

enum Mode { kLinear, kUp, kDown };

constexpr int slice_for(int width) { return width <= 64 ? 256 : 128; }

// PAIR: the tile's tokens are split between the CTAs.
template <int BN, bool PAIR>
struct Layout {
  static constexpr int kTokens = PAIR ? BN / 2 : BN;  // that a CTA brings
  // Elements of k of a slice.  What a slice costs in waits and commits is as much as
  // its MMAs take below 128 tokens, so slices are longer there.
  static constexpr int kSlice = slice_for(BN);
  static constexpr int kSlotCols = kSlice / 2;
  static constexpr int kWBytes = kRows * kSlice / 2;
  static constexpr int kBoxes = kSlice / 64;         // of tokens
  static constexpr int kSlots = kSlice == 256 ? 3 : 4;  // slices of converted weights
  static constexpr int kTeams = kSlots;
  static constexpr int kThreads = 32 * (4 + kReaders + 4 * kTeams);
  static constexpr int kXStages = BN == 256 ? 4 : BN == 128 ? 8 : BN == 64 ? 3 : 6;
  static constexpr int kWStages = kSlice == 256 ? 6 : 8;
  static constexpr int kXBytes = kTokens * kSlice * 2;
  static constexpr int kAccs = BN == 256 ? 1 : 2;
  static constexpr int kWOffset = kXStages * kXBytes;
  static constexpr int kReadOffset = kWOffset + kWStages * kWBytes;
  static constexpr int kBarOffset = kReadOffset + kReaders * kReadBytes;
  // barriers: xfull, xempty, full, empty, wfull, wempty, accfull, accempty, done
  static constexpr int kBars = 2 * (kXStages + kSlots + kWStages + kAccs) + 1;
  static constexpr int kPeerIssued = kBarOffset + 8 * kBars;  // int64
  static constexpr int kTmemSlot = kPeerIssued + 8;
  static constexpr int kUsed = kTmemSlot + 8 + 1024;
  // more than half of an SM's, so that no two CTAs share its tensor memory
  static constexpr int kBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static constexpr int kACol = kAccs * BN;  // first column of the slots
  // A slot and a stage of codes are always the same team's: a team may be a round ahead
  // of another, and a barrier tells one round from the next only.
  static_assert(kSlots % kTeams == 0 && kWStages % kTeams == 0, "teams");
  static_assert(kACol + kSlots * kSlotCols <= 512, "tensor memory");
  static_assert(kBytes + 4 * (kTilesMaxExperts + 1) + 64 <= 232448, "shared memory");
};

template <typename T>
__host__ __device__ constexpr uint32_t instr(int m, int n) {  // fp32 sums, A and B of T, both K-major, m x n
  const uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}

// True in one lane of the warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity, int* status) {
  volatile int go_on = 0;
  return mbar_wait(bar, parity, &go_on, status);
}

// D (+)= A[tmem] . B[smem]^T over the pair: rows 0..127 of A and tokens 0..N/2 of B
// in the even CTA.
__device__ __forceinline__ void mma_pair_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A unit of work: a tile of rows by a block of tokens, whole or a part of k of it.
struct Unit {
  int expert, first, count;  // the block's tokens: place of the first, how many
  // Tokens that the MMAs take: whole thirty-twos for a pair (4096 tokens, 6 of 64 experts:
  // 367 us, 383 with whole blocks).
  int width;
  int row;                   // first row, in the expert
  int slice, end;            // slices of k
  int share;                 // of a part: its place among the shares (-1: a whole tile)
};
// A linear layer's tiles: `whole` ones, then the rest, each in `parts` parts.
template <int MODE, int BN, bool PAIR>
struct Units {
  static constexpr int kTileRows = PAIR ? 2 * kRows : kRows;
  const W4TilesParams& p;
  const int* before;  // blocks of tokens before an expert's
  int u, step, total, rank, expert = 0;
  __device__ __forceinline__ Units(const W4TilesParams& q, const int* b) : p(q), before(b) {
    if (MODE == kLinear)
      total = p.whole + (p.blocks * p.row_tiles - p.whole) * p.parts;
    else
      total = before[p.experts] * p.row_tiles;
    u = PAIR ? (int)cluster_index() : blockIdx.x;
    step = PAIR ? (int)cluster_count() : gridDim.x;
    rank = PAIR ? (int)cluster_rank() : 0;
  }
  __device__ __forceinline__ bool next(Unit& x) {
    if (u >= total) return false;
    int tile = u;
    x.share = -1;
    x.slice = 0;
    x.end = p.slices;
    if (MODE == kLinear && u >= p.whole) {
      x.share = u - p.whole;
      tile = x.share / p.parts;
      x.slice = (x.share - tile * p.parts) * p.part_slices;
      x.end = min(x.slice + p.part_slices, p.slices);
      tile += p.whole;
    }
    const int block = tile / p.row_tiles;
    x.row = (tile - block * p.row_tiles) * kTileRows + rank * kRows;
    if (MODE == kLinear) {
      x.expert = 0;
      x.first = block * BN;
      x.count = min(BN, p.m - x.first);
    } else {
      while (before[expert + 1] <= block) ++expert;
      x.expert = expert;
      const int skip = (block - before[expert]) * BN, at = p.offsets[expert];
      x.first = at + skip;
      x.count = min(BN, p.offsets[expert + 1] - x.first);
    }
    x.width = PAIR ? min(BN, (x.count + 31) / 32 * 32) : BN;
    u += step;
    return true;
  }
};

template <typename T, int MODE, int BN, bool PAIR>
__global__ void __launch_bounds__(Layout<BN, PAIR>::kThreads, 1)
    w4_tiles_kernel(const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_x, const W4TilesParams p) {
  using L = Layout<BN, PAIR>;
  constexpr int kSlice = L::kSlice, kSlotCols = L::kSlotCols, kWBytes = L::kWBytes;
  constexpr int XS = L::kXStages, SLOTS = L::kSlots, WS = L::kWStages, ACCS = L::kAccs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ int before[MODE == kLinear ? 1 : kTilesMaxExperts + 1];
  const uint32_t base = smem_addr(smem);
  const uint32_t bars = base + L::kBarOffset;
  auto xfull = [&](int i) { return bars + 8u * i; };
  auto xempty = [&](int i) { return bars + 8u * (XS + i); };
  auto full = [&](int i) { return bars + 8u * (2 * XS + i); };
  auto empty = [&](int i) { return bars + 8u * (2 * XS + SLOTS + i); };
  auto wfull = [&](int i) { return bars + 8u * (2 * (XS + SLOTS) + i); };
  auto wempty = [&](int i) { return bars + 8u * (2 * (XS + SLOTS) + WS + i); };
  auto accfull = [&](int i) { return bars + 8u * (2 * (XS + SLOTS + WS) + i); };
  auto accempty = [&](int i) { return bars + 8u * (2 * (XS + SLOTS + WS) + ACCS + i); };
  const uint32_t done = bars + 8u * (L::kBars - 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kTmemSlot + 4);
  volatile int64_t* peer_issued = reinterpret_cast<volatile int64_t*>(smem + L::kPeerIssued);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const bool even = !PAIR || cluster_rank() == 0;
  constexpr int CTAS = PAIR ? 2 : 1;
  // An arrival on the even CTA's barrier.  What the arrivals of the converters and
  // readers say is about tensor memory, which tcgen05's own waits and fences order: a
  // release to the other CTA (0.70 us a slice of 256 tokens with it, 0.58 without) has
  // nothing to add.
  auto arrive_even = [&](uint32_t bar) {
    if (!PAIR || even)
      mbar_arrive(bar);
    else
      mbar_arrive_cluster_relaxed(cluster_map(bar, 0));
  };
  auto commit = [&](uint32_t bar) {
    if (PAIR)
      mma_commit_pair(bar);
    else
      mma_commit(bar);
  };

  if (threadIdx.x == 0) {
    *peer_issued = 0;
    for (int i = 0; i < WS; ++i) mbar_init(wfull(i), 1), mbar_init(wempty(i), 4);
    for (int i = 0; i < XS; ++i) mbar_init(xfull(i), 1), mbar_init(xempty(i), 1);
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(full(i), 4 * CTAS);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < ACCS; ++i) mbar_init(accfull(i), 1), mbar_init(accempty(i), kReaders * CTAS);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_addr(tmem_slot), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_addr(tmem_slot), 512);
      tmem_relinquish();
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (MODE != kLinear) {
    for (int e = threadIdx.x; e < p.experts; e += L::kThreads)
      before[e + 1] = (p.offsets[e + 1] - p.offsets[e] + BN - 1) / BN;
    __syncthreads();
    if (warp == 0) {  // running sums
      int sum = 0;
      for (int e0 = 0; e0 < p.experts; e0 += 32) {
        const int e = e0 + lane;
        int v = e < p.experts ? before[e + 1] : 0;
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
          const int x = __shfl_up_sync(0xffffffffu, v, off);
          if (lane >= off) v += x;
        }
        if (e < p.experts) before[e + 1] = sum + v;
        sum += __shfl_sync(0xffffffffu, v, 31);
      }
      if (lane == 0) before[0] = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();  // both CTAs' barriers are there before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Units<MODE, BN, PAIR> units(p, before);
  int64_t issued = 0;  // copies of tokens
  Unit x;
  auto wait_warp = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status));
  };

  if (warp == 0) {
    // ---- TMA of the codes ----
    if (lane == 0) {
      tma_prefetch_desc(&map_w);
      int stage = 0, parity = 1;
      int64_t issued = 0;
      bool ok = true;
      while (ok && units.next(x))
        for (int s = x.slice; s < x.end; ++s) {
          if (!(ok = mbar_wait(wempty(stage), parity, abort_flag, p.status))) break;
          mbar_arrive_expect_tx(wfull(stage), kWBytes);
          tma_load_2d(base + L::kWOffset + stage * kWBytes, &map_w, wfull(stage), s * (kSlice / 2),
                      (int)(x.expert * p.n) + x.row);
          ++issued;
          if (++stage == WS) stage = 0, parity ^= 1;
        }
      if (!ok)  // wait for the copies still in flight
        for (int64_t i = min(issued, (int64_t)WS); i > 0; --i) {
          if (--stage < 0) stage = WS - 1, parity ^= 1;
          wait_drain(wfull(stage), parity ^ 1, p.status);
        }
    }
  } else if (warp == 2) {
    // ---- TMA of the tokens ----
    if (lane == 0) {
      tma_prefetch_desc(&map_x);
      int stage = 0, parity = 1;
      bool ok = true;
      while (ok && units.next(x))
        for (int s = x.slice; s < x.end; ++s) {
          if (!(ok = mbar_wait(xempty(stage), parity, abort_flag, p.status))) break;
          const uint32_t dst = base + stage * L::kXBytes;
          const int row = x.first + (even ? 0 : x.width / 2);
#pragma unroll
          for (int b = 0; b < L::kBoxes; ++b) {
            // (a box that would begin past the row is any other: no MMA reads it)
            const int k = s * kSlice + 64 * b < p.k ? s * kSlice + 64 * b : 0;
            if (PAIR) {
              if (even && b == 0) mbar_arrive_expect_tx(xfull(stage), 2 * L::kXBytes);
              tma_load_2d_pair(dst + b * L::kTokens * 128, &map_x, cluster_map(xfull(stage), 0), k,
                               row);
            } else {
              if (b == 0) mbar_arrive_expect_tx(xfull(stage), L::kXBytes);
              tma_load_2d(dst + b * L::kTokens * 128, &map_x, xfull(stage), k, row);
            }
          }
          ++issued;
          if (++stage == XS) stage = 0, parity ^= 1;
        }
      if (!ok && !PAIR)
        for (int64_t i = min(issued, (int64_t)XS); i > 0; --i) {
          if (--stage < 0) stage = XS - 1, parity ^= 1;
          wait_drain(xfull(stage), parity ^ 1, p.status);
        }
      if (PAIR && !even)
        st_cluster_u64(cluster_map(smem_addr((const void*)peer_issued), 0), (uint64_t)issued);
    }
  } else if (warp == 1) {
    // ---- the MMAs: the warp keeps step, so that what an MMA takes is the same in all its
    // lanes, and one lane issues them ----
    if (even) {
      constexpr int PIECES = kSlice / 16;
      const bool one = elect_one();
      int stage = 0, xparity = 0, slot = 0, parity = 0, acc = 0, cparity = 1;
      bool ok = true;
      while (ok && units.next(x)) {
        if (!(ok = wait_warp(accempty(acc), cparity))) break;
        tc_fence_after();
        const uint32_t idesc = instr<T>(kRows * CTAS, x.width);
        const uint32_t d = tmem + acc * BN;
        for (int s = x.slice; s < x.end; ++s) {
          if (!(ok = wait_warp(xfull(stage), xparity))) break;
          if (!(ok = wait_warp(full(slot), parity))) break;
          tc_fence_after();
          const uint64_t desc = smem_desc_sw128(base + stage * L::kXBytes);
          const uint32_t a = tmem + L::kACol + slot * kSlotCols;
          const int pieces = min(kSlice, p.k - s * kSlice) / 16;
          auto piece = [&](int i, uint32_t more) {
            const uint64_t b = desc + (i / 4) * (L::kTokens * 128 >> 4) + 2 * (i % 4);
            if (PAIR)
              mma_pair_ts(d, a + 8 * i, b, idesc, more);
            else
              mma_f16_ts(d, a + 8 * i, b, idesc, more);
          };
          if (one) {
            piece(0, s > x.slice ? 1u : 0u);
            if (pieces == PIECES) {
#pragma unroll
              for (int i = 1; i < PIECES; ++i) piece(i, 1u);
            } else {
              for (int i = 1; i < pieces; ++i) piece(i, 1u);
            }
            commit(empty(slot));
            commit(xempty(stage));
          }
          __syncwarp();
          if (++stage == XS) stage = 0, xparity ^= 1;
          if (++slot == SLOTS) slot = 0, parity ^= 1;
        }
        if (!ok) break;
        if (one) commit(accfull(acc));
        if (++acc == ACCS) acc = 0, cparity ^= 1;
      }
      if (one) commit(done);  // arrives once every MMA issued above has completed
    }
  } else if (warp >= 4 && warp < 4 + kReaders) {
    // ---- read-out: lane = row, columns = tokens; the readers of a quarter take 32 in turn ----
    const int quarter = warp & 3;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    uint8_t* turn = smem + L::kReadOffset + (warp - 4) * kReadBytes;
    // BYTES a token of this quarter's rows (up: pairs of rows), in 16-byte pieces
    constexpr int BYTES = MODE == kUp ? 32 : 64, LANES = BYTES / 16;
    T* const mine = reinterpret_cast<T*>(turn) + (MODE == kUp ? lane / 2 : lane);
    const int piece = lane % LANES;
    const int width = (int)(MODE == kUp ? p.n / 2 : p.n);
    int acc = 0, parity = 0;
    bool ok = true;
    while (ok && units.next(x)) {
      const int row0 = x.row + quarter * 32, row = row0 + lane;
      const float scale =
          row < p.n ? __ldg(p.row_scales + (int64_t)x.expert * p.n + row) : 0.0f;
      const int at = (MODE == kUp ? row0 / 2 : row0) + 8 * piece;
      const bool shared = MODE == kLinear && x.share >= 0;
      const bool turned = MODE == kUp || (MODE == kLinear && !shared && p.vector);
      // the 32 tokens from c0 on, from shared memory to their rows
      auto put = [&](int c0) {
        T* out = static_cast<T*>(p.out) + (int64_t)(x.first + c0) * p.out_stride + at;
#pragma unroll
        for (int j = lane / LANES; j < 32; j += 32 / LANES) {
          const uint4 o = *reinterpret_cast<const uint4*>(turn + j * 80 + 16 * piece);
          if (j < x.count - c0 && at < width) {
            if (at + 8 <= width) {
              *reinterpret_cast<uint4*>(out + j * p.out_stride) = o;
            } else {
              const T* e = reinterpret_cast<const T*>(&o);
              for (int i = 0; i < width - at; ++i) out[j * p.out_stride + i] = e[i];
            }
          }
        }
      };
      if (!(ok = wait_warp(accfull(acc), parity))) break;
      tc_fence_after();
      int last = -1;  // tokens that are in shared memory
#pragma unroll 1
      for (int c0 = (warp - 4) / 4 * 32; c0 < min(BN, x.count); c0 += 32 * (kReaders / 4)) {
        uint32_t v[32];
        tmem_ld32(tmem + lanes + acc * BN + c0, v);
        if (last >= 0) put(last);  // (beside the load)
        tmem_ld_wait();
        if (turned) {
          __syncwarp();
          if (MODE == kUp) {
            // rows 2i (gate) and 2i + 1 (up) sit in neighbouring lanes: the even one takes
            // token j, the odd one j + 1
            float h[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float a = __uint_as_float(v[2 * j]) * scale;
              const float b = __uint_as_float(v[2 * j + 1]) * scale;
              const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : b, 1);
              const float gate = lane & 1 ? other : a, up = lane & 1 ? b : other;
              h[j] = silu_times(gate, up);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
              mine[(2 * j + (lane & 1)) * (80 / 2)] = from_f32<T>(h[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              mine[j * (80 / 2)] = from_f32<T>(__uint_as_float(v[j]) * scale);
          }
          __syncwarp();
          last = c0;
        } else if (MODE == kDown || shared) {
          // down: [pick][n]; a share: [token of the tile][row of the tile]
          constexpr int TILE = Units<MODE, BN, PAIR>::kTileRows;
          const int64_t pitch = shared ? TILE : p.n;
          float* out = static_cast<float*>(shared ? p.shares : p.out) +
                       (shared ? ((int64_t)x.share * BN + c0) * TILE + row % TILE
                               : (int64_t)(x.first + c0) * p.n + row);
          if (row < p.n) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c0 + j < x.count) out[j * pitch] = __uint_as_float(v[j]) * scale;
          }
        } else {  // rows that are not aligned
          T* out = static_cast<T*>(p.out) + (int64_t)(x.first + c0) * p.out_stride + row;
          if (row < p.n) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c0 + j < x.count)
                out[j * p.out_stride] = from_f32<T>(__uint_as_float(v[j]) * scale);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_even(accempty(acc));
      if (++acc == ACCS) acc = 0, parity ^= 1;
      if (last >= 0) put(last);  // (beside the next tile's MMAs)
      __syncwarp();
    }
  } else if (warp >= 4 + kReaders) {
    // ---- converters: a row a lane, slices in turn by team ----
    const int quarter = warp & 3, team = (warp - 4 - kReaders) >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t scale_row = p.k / p.group;
    const int shift = p.group == 32 ? 5 : p.group == 64 ? 6 : 7;
    int index = 0;  // of the slice among all of this CTA
    bool ok = true;
    while (ok && units.next(x)) {
      const uint8_t* scales =
          p.scales + ((int64_t)x.expert * p.n + min(x.row + r, (int)p.n - 1)) * scale_row;
      const int skip = (team + L::kTeams - index % L::kTeams) % L::kTeams;
      int s = x.slice + skip;
      auto scale_at = [&](int slice, int piece) -> uint32_t {  // of 32 elements
        const int at = slice * kSlice + piece * 32;
        return at < p.k && slice < x.end ? __ldg(scales + (at >> shift)) : 0;
      };
      constexpr int PIECES = kSlice / 32;
      uint32_t ahead[PIECES];
#pragma unroll
      for (int q = 0; q < PIECES; ++q) ahead[q] = scale_at(s, q);
      for (int i = index + skip; s < x.end; s += L::kTeams, i += L::kTeams) {
        const int stage = i % WS, slot = i % SLOTS;
        uint32_t bytes[PIECES];
#pragma unroll
        for (int q = 0; q < PIECES; ++q) bytes[q] = ahead[q];
#pragma unroll
        for (int q = 0; q < PIECES; ++q) ahead[q] = scale_at(s + L::kTeams, q);
        if (!(ok = wait_warp(wfull(stage), (uint32_t)(i / WS) & 1u))) break;
        // 16-byte piece c of row r sits at piece c ^ (r / 2 % 4) of its 64 bytes, or
        // c ^ (r % 8) of 128: the swizzle by as many bytes
        const uint8_t* w = smem + L::kWOffset + stage * kWBytes + r * (kSlice / 2);
        const int turn = kSlice == 128 ? r >> 1 & 3 : r & 7;
#pragma unroll
        for (int half = 0; half < kSlice / 64; ++half) {
          uint32_t words[32];
          W4Scale<T> sc[2];
          w4_scales(bytes[2 * half], bytes[2 * half + 1], sc[0], sc[1]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint4 c = *reinterpret_cast<const uint4*>(w + (((2 * half + q) ^ turn) << 4));
            const uint32_t code[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t o[4];
              w4_word(code[j], sc[q], o);
#pragma unroll
              for (int k = 0; k < 4; ++k) words[16 * q + 4 * j + k] = o[k];
            }
          }
          if (half == 0) {
            if (!(ok = wait_warp(empty(slot), ((uint32_t)(i / SLOTS) & 1u) ^ 1u))) break;
            tc_fence_after();
          }
          tmem_st32(tmem + lanes + L::kACol + slot * kSlotCols + half * 32, words);
        }
        if (!ok) break;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_even(full(slot));
          mbar_arrive(wempty(stage));
        }
      }
      index += x.end - x.slice;
    }
  }

  __syncthreads();
  if (PAIR) {
    cluster_sync_all();  // the odd CTA's number of copies has reached the even one
    if (even && warp == 2 && lane == 0) {
      // Copies may be in flight only after a time-out, the last of the CTA that
      // issued more: one that the other never issued gets its half armed or completed
      // here, so that its phase ends when the issued half has landed.
      const int64_t peer = *peer_issued, most = max(issued, peer);
      for (int64_t j = max(most - XS, (int64_t)0); j < most; ++j) {
        const int stage = (int)(j % XS);
        if (j >= issued)
          mbar_arrive_expect_tx(xfull(stage), L::kXBytes);
        else if (j >= peer)
          mbar_complete_tx(xfull(stage), L::kXBytes);
        wait_drain(xfull(stage), (uint32_t)(j / XS) & 1u, p.status);
      }
    }
  }
  if (warp == 1) {
    if (lane == 0) wait_drain(done, 0, p.status);
    __syncwarp();
  }
  if (PAIR) {
    tc_fence_before();
    cluster_sync_all();  // no copy, MMA or arrival targets either CTA any more
  }
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

// From this width on a tile is a pair's.
constexpr int kPairWidth = 128;

template <typename T, int MODE, int BN>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& x, const W4TilesParams& p,
                   int64_t units, int sm_count, bool dependent, cudaStream_t s) {
  constexpr bool PAIR = BN >= kPairWidth;
  auto kernel = w4_tiles_kernel<T, MODE, BN, PAIR>;
  static std::atomic<uint64_t> set{0};  // devices on which the kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  constexpr int bytes = Layout<BN, PAIR>::kBytes;
  if (!(set.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    set |= uint64_t(1) << dev;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(PAIR ? 2 * (unsigned)std::min<int64_t>(units, sm_count / 2)
                          : (unsigned)std::min<int64_t>(units, sm_count));
  cfg.blockDim = dim3(Layout<BN, PAIR>::kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (PAIR) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim = {2, 1, 1};
    ++cfg.numAttrs;
  }
  if (dependent) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, kernel, w, x, p);
}

template <int MODE, int BN>
cudaError_t launch(int dtype, const CUtensorMap& w, const CUtensorMap& x, const W4TilesParams& p,
                   int64_t units, int sm_count, bool dependent, cudaStream_t s) {
  return dtype == LBGEMM_BF16
             ? launch<__nv_bfloat16, MODE, BN>(w, x, p, units, sm_count, dependent, s)
             : launch<__half, MODE, BN>(w, x, p, units, sm_count, dependent, s);
}

template <int MODE>
cudaError_t launch(int dtype, int bn, const CUtensorMap& w, const CUtensorMap& x,
                   const W4TilesParams& p, int64_t units, int sm_count, bool dependent,
                   cudaStream_t s) {
  if (bn == 32) return launch<MODE, 32>(dtype, w, x, p, units, sm_count, dependent, s);
  if (bn == 64) return launch<MODE, 64>(dtype, w, x, p, units, sm_count, dependent, s);
  if (bn == 128) return launch<MODE, 128>(dtype, w, x, p, units, sm_count, dependent, s);
  return launch<MODE, 256>(dtype, w, x, p, units, sm_count, dependent, s);
}

// ---- joining the parts of k of a linear layer ---------------------------------------
// Of the tiles that were cut: y = the sum of their shares, in order.  A block a token
// of a tile, its threads along the rows.
template <typename T>
__global__ void __launch_bounds__(256)
    join_kernel(const W4TilesParams p, int width, int tile_rows) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tile = blockIdx.x / width, token = blockIdx.x - tile * width;
  const int block = (p.whole + tile) / p.row_tiles;
  const int row = (p.whole + tile - block * p.row_tiles) * tile_rows + threadIdx.x;
  const int m = block * width + token;
  if (m >= p.m || row >= p.n) return;
  const float* share = p.shares + ((int64_t)tile * p.parts * width + token) * tile_rows + threadIdx.x;
  const int64_t step = (int64_t)width * tile_rows;
  float v = 0.0f;
#pragma unroll 4
  for (int q = 0; q < p.parts; ++q) v += share[q * step];
  static_cast<T*>(p.out)[m * p.out_stride + row] = from_f32<T>(v);
}

// ---- picks in expert order --------------------------------------------------------------
// Pieces of the list of picks: a histogram each, then each piece's places from the
// sums before it.  One piece does both at once.
constexpr int kSortThreads = 1024;
__global__ void __launch_bounds__(kSortThreads)
    count_kernel(const MoeSort q) {
  __shared__ int counts[kTilesMaxExperts];
  for (int e = threadIdx.x; e < q.experts; e += kSortThreads) counts[e] = 0;
  __syncthreads();
  const int first = blockIdx.x * q.piece, end = min(first + q.piece, q.picks);
  for (int i = first + threadIdx.x; i < end; i += kSortThreads) {
    const int e = q.ids[i];
    if (e >= 0 && e < q.experts) atomicAdd(&counts[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < q.experts; e += kSortThreads)
    q.counts[blockIdx.x * q.experts + e] = counts[e];
}
__global__ void __launch_bounds__(kSortThreads) place_kernel(const MoeSort q) {
  __shared__ int cursor[kTilesMaxExperts], sums[32];
  const int first = blockIdx.x * q.piece, end = min(first + q.piece, q.picks);
  const int e = threadIdx.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  cursor[threadIdx.x] = 0;  // (kSortThreads is kTilesMaxExperts)
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int before = 0, total = 0;  // of expert e: in pieces before this one, in all
  if (q.pieces == 1) {
    for (int i = threadIdx.x; i < q.picks; i += kSortThreads) {
      const int id = q.ids[i];
      if (id >= 0 && id < q.experts) atomicAdd(&cursor[id], 1);
    }
    __syncthreads();
    total = cursor[e];
  } else if (e < q.experts) {
    for (int c = 0; c < q.pieces; ++c) {
      const int n = q.counts[c * q.experts + e];
      total += n;
      if (c < (int)blockIdx.x) before += n;
    }
  }
  int v = total;  // running sum over the experts
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += x;
  }
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  int carry = 0;
  for (int w = 0; w < warp; ++w) carry += sums[w];
  v += carry;
  cursor[e] = v - total + before;
  if (blockIdx.x == 0 && e < q.experts) {
    q.offsets[e + 1] = v;
    if (e == 0) q.offsets[0] = 0;
  }
  __syncthreads();
  // (the order within an expert does not matter: a pick's sums are its own)
  for (int i = first + threadIdx.x; i < end; i += kSortThreads) {
    const int id = q.ids[i];
    int pos = -1;
    if (id >= 0 && id < q.experts) {
      pos = atomicAdd(&cursor[id], 1);
      q.token_of[pos] = i / q.top_k;
    } else if (id >= q.experts) {
      atomicOr(q.status, kStatusBadIndex);
    }
    q.pos_of[i] = pos;
  }
}

// (In this kernel and combine_kernel only the call's own inputs are __restrict__ or read by
// __ldg.  A dependent may be resident while the launch before it still writes, and what is
// loaded as constant for a kernel's whole life could be loaded before its wait.)

// ---- the picks' tokens in expert order -------------------------------------------------
// (tile::gather4 reads them where they are, but took 80 cycles for four pieces of 128
// bytes: 895 us for 24576 picks of 2048 elements against 64 experts)
__global__ void __launch_bounds__(256)
    gather_kernel(const uint16_t* __restrict__ x, int64_t x_stride, const int* offsets,
                  int experts, const int* token_of, int width, uint16_t* to) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int octets = width / 8, picks = offsets[experts];
  const int64_t total = (int64_t)picks * octets;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t pos = i / octets;
    const int c = (int)(i - pos * octets) * 8;
    *reinterpret_cast<uint4*>(to + pos * width + c) =
        *reinterpret_cast<const uint4*>(x + token_of[pos] * x_stride + c);
  }
}

// ---- a token's picks added up -------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256)
    combine_kernel(const float* out, const int* pos_of, const float* __restrict__ weights,
                   int64_t tokens, int hidden, int top_k, T* y, int64_t y_stride) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int octets = hidden / 8;
  const int64_t total = tokens * octets;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / octets;
    const int c = (int)(i - t * octets) * 8;
    float v[8] = {};
    for (int j = 0; j < top_k; ++j) {
      const int pos = pos_of[t * top_k + j];
      if (pos < 0) continue;
      const float w = __ldg(weights + t * top_k + j);
      float f[8];
      unpack8(load8_raw(out + (int64_t)pos * hidden + c), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += w * f[k];
    }
    store8(y + t * y_stride + c, v);
  }
}

template <typename F, typename... A>
cudaError_t launch_after(F kernel, int64_t blocks, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Tokens of a tile for a block of `tokens` on average.
int width_for(int64_t tokens) {
  return tokens <= 32 ? 32 : tokens <= 64 ? 64 : tokens <= 128 ? 128 : 256;
}

int tiles_of(int64_t rows, int width) {
  const int tile = width >= kPairWidth ? 2 * kRows : kRows;
  return (int)((rows + tile - 1) / tile);
}

bool maps(int dtype, const W4& w, int64_t rows, int64_t k, const void* x, int64_t x_rows,
          int64_t x_stride, int width, CUtensorMap* map_w, CUtensorMap* map_x) {
  return encode_map(map_w, LBGEMM_MAP_U8, w.codes, k / 2, rows, k / 2, slice_for(width) / 2, kRows,
                    slice_for(width) / 2) &&
         encode_map(map_x, dtype, x, k, x_rows, x_stride * 2, 64,
                    width >= kPairWidth ? width / 2 : width, 128);
}

int64_t round16(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Where a mixture's scratch lies.
struct MoeScratch {
  int64_t h, x, out, counts, offsets, token_of, pos_of, bytes;
  int pieces, piece;
};
MoeScratch moe_scratch(const MoeParams& m) {
  MoeScratch z;
  const int64_t picks = m.tokens * m.top_k;
  z.piece = (int)std::max<int64_t>(4096, (picks + 63) / 64);
  z.pieces = (int)((picks + z.piece - 1) / z.piece);
  z.h = 0;
  z.x = z.h + round16(picks * m.inter * 2);
  // (the tokens in expert order are read before the outputs are written)
  z.out = z.x;
  z.counts = z.out + round16(picks * m.hidden * 4);
  z.offsets = z.counts + round16((int64_t)z.pieces * m.experts * 4);
  z.token_of = z.offsets + round16((m.experts + 1) * 4);
  z.pos_of = z.token_of + round16(picks * 4);
  z.bytes = z.pos_of + round16(picks * 4);
  return z;
}

// How a linear layer is cut: tiles that do not make half a wave (of the SMs, or pairs)
// are cut along k, so that they take one as a whole.  A part has 512 elements at least.
void cut_linear(const W4LinearParams& l, int sm_count, int* bn, W4TilesParams* p) {
  *bn = width_for(l.m);
  p->blocks = (int)((l.m + *bn - 1) / *bn);
  p->row_tiles = tiles_of(l.n, *bn);
  const int slice = slice_for(*bn);
  p->slices = p->part_slices = (int)((l.k + slice - 1) / slice);
  const int64_t tiles = (int64_t)p->blocks * p->row_tiles;
  const int slots = *bn >= kPairWidth ? sm_count / 2 : sm_count;
  const int rest = (int)(tiles % slots);
  p->whole = (int)tiles;
  p->parts = 1;
  if (rest == 0 || 2 * rest > slots) return;
  const int parts = std::min(slots / rest, p->slices / (512 / slice));
  if (parts < 2) return;
  p->part_slices = (p->slices + parts - 1) / parts;
  p->parts = (p->slices + p->part_slices - 1) / p->part_slices;
  p->whole = (int)tiles - rest;
}

}  // namespace

size_t w4_tiles_linear_scratch(const W4LinearParams& l, int sm_count) {
  W4TilesParams p;
  int bn;
  cut_linear(l, sm_count, &bn, &p);
  const size_t shares = ((size_t)p.blocks * p.row_tiles - p.whole) * p.parts;
  return shares * bn * (bn >= kPairWidth ? 2 * kRows : kRows) * sizeof(float);
}

cudaError_t launch_w4_tiles_linear(int dtype, const W4LinearParams& l, void* scratch, int sm_count,
                                   int* launches, cudaStream_t s) {
  W4TilesParams p;
  int bn;
  cut_linear(l, sm_count, &bn, &p);
  p.n = l.n;
  p.k = (int)l.k;
  p.group = l.group;
  p.scales = l.w.scales;
  p.row_scales = l.w.row_scales;
  p.out = l.y;
  p.out_stride = l.y_stride;
  p.vector = l.m == 1 || l.y_stride % 8 == 0;
  p.shares = static_cast<float*>(scratch);
  p.m = (int)l.m;
  p.status = l.status;
  CUtensorMap map_w, map_x;
  // (a single row's stride may be anything)
  if (!maps(dtype, l.w, l.n, l.k, l.x, l.m, l.m > 1 ? l.x_stride : l.k, bn, &map_w, &map_x))
    return cudaErrorInvalidValue;
  const int64_t cut = (int64_t)p.blocks * p.row_tiles - p.whole;
  cudaError_t e = launch<kLinear>(dtype, bn, map_w, map_x, p, p.whole + cut * p.parts, sm_count,
                                  false, s);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (cut == 0) return e;
  const int rows = bn >= kPairWidth ? 2 * kRows : kRows;
  e = dtype == LBGEMM_BF16
          ? launch_after(join_kernel<__nv_bfloat16>, cut * bn, rows, s, p, bn, rows)
          : launch_after(join_kernel<__half>, cut * bn, rows, s, p, bn, rows);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

size_t w4_tiles_moe_scratch(const MoeParams& m) { return (size_t)moe_scratch(m).bytes; }

cudaError_t launch_w4_tiles_moe(int dtype, const MoeParams& m, void* scratch, int sm_count,
                                int* launches, cudaStream_t s) {
  const MoeScratch z = moe_scratch(m);
  uint8_t* at = static_cast<uint8_t*>(scratch);
  const int64_t picks = m.tokens * m.top_k;
  MoeSort q;
  q.ids = m.ids;
  q.picks = (int)picks;
  q.top_k = m.top_k;
  q.experts = m.experts;
  q.piece = z.piece;
  q.pieces = z.pieces;
  q.counts = reinterpret_cast<int*>(at + z.counts);
  q.offsets = reinterpret_cast<int*>(at + z.offsets);
  q.token_of = reinterpret_cast<int*>(at + z.token_of);
  q.pos_of = reinterpret_cast<int*>(at + z.pos_of);
  q.status = m.status;
  cudaError_t e;
  if (q.pieces > 1) {
    count_kernel<<<q.pieces, kSortThreads, 0, s>>>(q);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    *launches += 1;
    e = launch_after(place_kernel, q.pieces, kSortThreads, s, q);
  } else {
    place_kernel<<<1, kSortThreads, 0, s>>>(q);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  *launches += 1;

  // Blocks of tokens for the average expert.
  const int bn = width_for((picks + m.experts - 1) / m.experts);
  const int slice = slice_for(bn);
  W4TilesParams p;
  p.experts = m.experts;
  p.offsets = q.offsets;
  p.group = m.group;
  p.m = (int)picks;
  p.status = m.status;
  CUtensorMap map_w, map_x;
  p.n = 2 * (int64_t)m.inter;
  p.k = m.hidden;
  p.row_tiles = tiles_of(p.n, bn);
  p.slices = (p.k + slice - 1) / slice;
  p.scales = m.up.scales;
  p.row_scales = m.up.row_scales;
  p.out = at + z.h;
  p.out_stride = m.inter;
  uint16_t* x = reinterpret_cast<uint16_t*>(at + z.x);
  e = launch_after(gather_kernel, std::min<int64_t>((picks * (m.hidden / 8) + 255) / 256, 16 * sm_count),
                   256, s, static_cast<const uint16_t*>(m.x), m.x_stride, (const int*)q.offsets,
                   m.experts, (const int*)q.token_of, m.hidden, x);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (!maps(dtype, m.up, m.experts * p.n, p.k, x, picks, m.hidden, bn, &map_w, &map_x))
    return cudaErrorInvalidValue;
  const int64_t units = INT32_MAX;  // (known on the device only)
  e = launch<kUp>(dtype, bn, map_w, map_x, p, units, sm_count, true, s);
  if (e != cudaSuccess) return e;
  *launches += 1;
  // Tiles with few slices spend their time on the fp32 rows that they write: blocks of 128
  // have a second accumulator for the next tile (64 experts of 2048 / 1024: 348 us, 366 with
  // 256; 8 of 4096 / 2048: 348 and 361; of 2048 / 4096: 335 and 320).
  const int down_bn = m.inter <= 2048 ? std::min(bn, 128) : bn;
  const int down_slice = slice_for(down_bn);
  p.n = m.hidden;
  p.k = m.inter;
  p.row_tiles = tiles_of(p.n, down_bn);
  p.slices = (p.k + down_slice - 1) / down_slice;
  p.scales = m.down.scales;
  p.row_scales = m.down.row_scales;
  p.out = at + z.out;
  if (!maps(dtype, m.down, m.experts * p.n, p.k, at + z.h, picks, m.inter, down_bn, &map_w,
            &map_x))
    return cudaErrorInvalidValue;
  e = launch<kDown>(dtype, down_bn, map_w, map_x, p, units, sm_count, true, s);
  if (e != cudaSuccess) return e;
  *launches += 1;
  const float* out = reinterpret_cast<const float*>(at + z.out);
  const int64_t blocks = std::min<int64_t>((m.tokens * (m.hidden / 8) + 255) / 256, 16 * sm_count);
  if (dtype == LBGEMM_BF16)
    e = launch_after(combine_kernel<__nv_bfloat16>, blocks, 256, s, out, (const int*)q.pos_of,
                     m.weights, m.tokens, m.hidden, m.top_k, static_cast<__nv_bfloat16*>(m.y),
                     m.y_stride);
  else
    e = launch_after(combine_kernel<__half>, blocks, 256, s, out, (const int*)q.pos_of, m.weights,
                     m.tokens, m.hidden, m.top_k, static_cast<__half*>(m.y), m.y_stride);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

}  // namespace lbg
