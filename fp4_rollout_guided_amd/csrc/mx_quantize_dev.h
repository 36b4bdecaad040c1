// Device helpers of the MXFP4 quantiser, on 8-element vectors (four packed
// bf16 pairs).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"
#include "fp4_block.h"

namespace trace_dev {

// The value of lane ^ 2: a DPP quad permutation [2, 3, 0, 1].
__device__ __forceinline__ uint32_t quad_swap(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false);
}

// Largest magnitude's bf16 bits over a vector, NaN excluded (a signed 16-bit
// maximum of m + 0x7f puts NaN halves below every other value).
__device__ __forceinline__ uint32_t vec_amax_bits(const uint32_t (&w)[4]) {
  typedef short s16x2_t __attribute__((ext_vector_type(2)));
  s16x2_t best = {0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t m = (w[k] & 0x7fff7fffu) + 0x007f007fu;
    s16x2_t v;
    __builtin_memcpy(&v, &m, 4);
    best = __builtin_elementwise_max(best, v);
  }
  const int lo = best.x, hi = best.y;
  const int m = lo > hi ? lo : hi;
  return m > 0x7f ? (uint32_t)(m - 0x7f) : 0u;
}

// E2M1 codes of a vector under inverse scale inv (nibble j = element j) and
// its clip-mask byte: round to nearest even, saturating at 6; a NaN element
// gets code 0 and mask bit 0.
__device__ __forceinline__ uint32_t e2m1_codes8(const uint32_t (&w)[4], float inv, uint32_t& keep) {
  float q[8];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    q[j] = half_elem(w, j) * inv;
    bad |= __builtin_amdgcn_class(q[j], kBadClass);
  }
  keep = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) keep |= (fabsf(q[j]) <= 6.f ? 1u : 0u) << j;
  if (bad) {  // NaN and infinities: the conversion's own results are not these
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = is_nan_f(q[j]) ? 0.f : __builtin_amdgcn_fmed3f(q[j], -6.f, 6.f);
  }
  uint32_t c = 0;
  c = FP4_RNE(c, q[0], q[1], 0);
  c = FP4_RNE(c, q[2], q[3], 1);
  c = FP4_RNE(c, q[4], q[5], 2);
  c = FP4_RNE(c, q[6], q[7], 3);
  return c;
}

}  // namespace trace_dev
