// Argument checks shared by the C ABI's translation units (api.cpp,
// api_mx_product.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "trace.h"

namespace trace_api {

struct Range {
  uintptr_t lo;
  uint64_t len;
};

inline bool overlaps(Range a, Range b) {
  if (a.len == 0 || b.len == 0) return false;
  return a.lo < b.lo + b.len && b.lo < a.lo + a.len;
}

inline Range rng(const void* p, uint64_t len) { return Range{reinterpret_cast<uintptr_t>(p), len}; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// n = rows * cols with cols % 16 == 0 and 2n bytes addressable.
inline trace_status site_size(int64_t rows, int64_t cols, uint64_t* n_out) {
  if (rows < 0 || cols < 0 || (cols % 16) != 0) return TRACE_E_SHAPE;
  int64_t n = 0;
  if (__builtin_mul_overflow(rows, cols, &n) || n > (INT64_MAX / 4)) return TRACE_E_SHAPE;
  *n_out = (uint64_t)n;
  return TRACE_OK;
}

// n = rows * cols with cols % 32 == 0.
inline trace_status mx_site_size(int64_t rows, int64_t cols, uint64_t* n_out) {
  if (cols % 32 != 0) return TRACE_E_SHAPE;
  return site_size(rows, cols, n_out);
}

// TRACE_OK or TRACE_E_HIP, which trace_last_hip_error() then explains.
trace_status hip_status(hipError_t e);

// Outputs must not overlap any input nor each other; `inplace_ok` lists an
// (output, input) pair that may coincide exactly.
inline trace_status check_alias(const Range* outs, int nout, const Range* ins, int nin, int inplace_out = -1,
                                int inplace_in = -1) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j) {
      if (i == inplace_out && j == inplace_in && outs[i].lo == ins[j].lo && outs[i].len == ins[j].len)
        continue;
      if (overlaps(outs[i], ins[j])) return TRACE_E_ALIAS;
    }
    for (int k = i + 1; k < nout; ++k)
      if (overlaps(outs[i], outs[k])) return TRACE_E_ALIAS;
  }
  return TRACE_OK;
}

}  // namespace trace_api
