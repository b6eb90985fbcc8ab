// kv4_attention.cu -- attention of new tokens over the 4-bit paged cache.
//
//   t_ij = scale * ks_j * (q_i . kc_j)       kc, vc codes; ks, vs their scales
//   o_i  = sum_j softmax_j(t_ij) vs_j vc_j,  lse_i = log sum_j exp(t_ij)
//
// The plainest kernel: one warp per query row, its head's channels spread over
// the lanes, one cached token at a time with the running maximum m and sum l
// of the softmax.
#include <cuda_runtime.h>

#include "attn.h"
#include "attn_common.cuh"

namespace lbg {
namespace {

constexpr int kWarps = 4;

template <typename T, int DIM>
__global__ void __launch_bounds__(kWarps * 32) kv4_attention_kernel(const Kv4AttnParams p) {
  constexpr int C = DIM / 32;  // channels of a lane, consecutive
  const int lane = threadIdx.x % 32;
  const int64_t work = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  const int64_t row = work / p.heads_q;
  const int head = (int)(work - row * p.heads_q);
  if (row >= p.total_q) return;
  // the sequence of this row
  int b = 0;
  while (b < p.batch && row >= p.cu_q[b + 1]) ++b;
  if (b >= p.batch) {
    atomicOr(p.status, kStatusBadIndex);
    return;
  }
  const int n = p.cu_q[b + 1] - p.cu_q[b];
  int len = p.kv_lens[b];
  if (len > p.max_kv || len < 0) {
    atomicOr(p.status, kStatusBadIndex);
    len = len < 0 ? 0 : p.max_kv;
  }
  const int position = len - n + (int)(row - p.cu_q[b]);
  const int last = p.causal ? min(len, position + 1) : len;  // one past the last seen
  const int first = p.window ? max(0, position - p.window + 1) : 0;
  const T* q = static_cast<const T*>(p.q) + row * p.q_stride + head * DIM + lane * C;
  float x[C], o[C] = {};
#pragma unroll
  for (int i = 0; i < C; ++i) x[i] = to_f32(q[i]) * p.scale;
  float m = -INFINITY, l = 0.0f;
  for (int j = first; j < last; ++j) {
    const int page = p.page_table[b * p.table_width + j / p.cache.page_size];
    if (page < 0 || page >= p.cache.pages) {
      atomicOr(p.status, kStatusBadIndex);
      continue;
    }
    const int64_t at = j % p.cache.page_size;
    const uint8_t* block = p.cache.base + ((int64_t)page * p.cache.heads + head / p.group) *
                                              kv4_block_bytes(DIM, p.cache.page_size);
    const uint8_t* kc = block + at * (DIM / 2);
    const uint8_t* vc = kc + p.cache.page_size * (DIM / 2);
    const __nv_bfloat16* sc =
        reinterpret_cast<const __nv_bfloat16*>(block + p.cache.page_size * DIM) + at;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int ch = lane * C + i;
      dot += x[i] * (float)nibble_value(kc[ch / 2] >> (4 * (ch & 1)));
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    const float t = dot * __bfloat162float(sc[0]);
    const float next = fmaxf(m, t);
    const float keep = m == next ? 1.0f : expf(m - next), pj = expf(t - next);
    const float pv = pj * __bfloat162float(sc[p.cache.page_size]);
    l = l * keep + pj;
    m = next;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int ch = lane * C + i;
      o[i] = o[i] * keep + pv * (float)nibble_value(vc[ch / 2] >> (4 * (ch & 1)));
    }
  }
  const bool empty = last <= first;
  T* out = static_cast<T*>(p.o) + (row * p.heads_q + head) * DIM + lane * C;
#pragma unroll
  for (int i = 0; i < C; ++i) out[i] = from_f32<T>(empty ? 0.0f : o[i] / l);
  if (p.lse && lane == 0) p.lse[row * p.heads_q + head] = empty ? -INFINITY : m + logf(l);
}

template <typename T>
void launch_typed(const Kv4AttnParams& p, cudaStream_t s) {
  const int64_t rows = (int64_t)p.total_q * p.heads_q;
  const unsigned blocks = (unsigned)((rows + kWarps - 1) / kWarps);
  if (p.cache.dim == 64) kv4_attention_kernel<T, 64><<<blocks, kWarps * 32, 0, s>>>(p);
  else kv4_attention_kernel<T, 128><<<blocks, kWarps * 32, 0, s>>>(p);
}

}  // namespace

cudaError_t launch_kv4_attention(int dtype, const Kv4AttnParams& p, int, int* launches,
                                 cudaStream_t s) {
  if (dtype == LBGEMM_BF16) launch_typed<__nv_bfloat16>(p, s);
  else launch_typed<__half>(p, s);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace lbg
