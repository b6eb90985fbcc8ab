// api_checks.h -- argument checks shared by the C entries of the attention and
// the feed-forward operators.
#pragma once
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "attn.h"
#include "lbgemm.h"

namespace lbg {

inline lbgemm_status bad(lbgemm_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return report_error(st, buf);
}

inline int64_t elem_size(int dtype) { return dtype == LBGEMM_F32 ? 4 : 2; }

inline bool aligned(const void* p, int64_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

inline lbgemm_status check_dtype(int dtype, bool f32) {
  if (dtype == LBGEMM_BF16 || dtype == LBGEMM_F16 || (f32 && dtype == LBGEMM_F32))
    return LBGEMM_OK;
  return bad(LBGEMM_ERR_INVALID_ARG, "dtype %d is not taken by this call", dtype);
}

constexpr int64_t kMaxStride = int64_t(1) << 40;

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

}  // namespace lbg
