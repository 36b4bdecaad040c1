// Device helpers of the MXFP4 and MXFP8 quantisers, on 8-element vectors (four
// packed bf16 pairs).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"
#include "e8m0.h"
#include "fp4_block.h"
#include "mx8_block.h"

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

// Codes, scale byte and clip-mask byte of a lane's vector.  The four lanes of
// a 32-element block hold consecutive vectors and are active together; MXFP4
// codes are in .x.
template <bool kFp4>
__device__ __forceinline__ uint2 quantize_vector(const uint4& v, uint32_t& scale, uint32_t& keep) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t amax = vec_amax_bits(w);
  const uint32_t near = pair_swap(amax);
  amax = amax > near ? amax : near;
  const uint32_t far = quad_swap(amax);
  amax = amax > far ? amax : far;
  scale = mx_scale_byte<kFp4 ? kE2M1Emax : kE4M3Emax>(amax);
  const float inv = e8m0_inverse(scale);
  if constexpr (kFp4) {
    return make_uint2(e2m1_codes8(w, inv, keep), 0);
  } else {
    float q[8];
    uint32_t nan_bits;
    mx8_quotients<8>(w, inv, q, nan_bits);
    keep = mx8_keep_bits<8>(q) & ~nan_bits;
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __builtin_amdgcn_fmed3f(q[j], -448.f, 448.f);
    uint32_t C[2];
    fp8_rne_codes<8>(q, C);
    return make_uint2(C[0], C[1]);
  }
}

}  // namespace trace_dev
