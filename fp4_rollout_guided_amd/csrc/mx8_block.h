// MXFP8 (E4M3) element machinery shared by the capture and forward kernels
// (mx8_kernels.hip) and the quantiser (mx_quantize.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"

namespace trace_dev {

constexpr uint32_t kLow = 0x01010101u;   // bit 0 of every byte
constexpr uint32_t kSign = 0x80808080u;  // bit 7 of every byte

// Element j of a lane's N elements held as N / 2 packed bf16 pairs.
template <int N>
__device__ __forceinline__ float lane_elem(const uint32_t (&w)[N / 2], int j) {
  return (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
}

// Quotients of a lane's N elements under inverse scale inv; NaN quotients (a
// NaN element, or an infinity times the zero of a zero-scale block) become
// the zero the format gives them -- +0 for a NaN element, the element's
// signed zero otherwise -- and their elements are flagged in *nan_bits (a
// NaN element's mask bit is 0).
template <int N>
__device__ __forceinline__ void mx8_quotients(const uint32_t (&w)[N / 2], float inv, float (&q)[N],
                                              uint32_t& nan_bits) {
  bool bad = false;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    q[j] = lane_elem<N>(w, j) * inv;
    bad |= __builtin_amdgcn_class(q[j], 0x003);  // signalling or quiet NaN
  }
  nan_bits = 0;
  if (bad) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float xv = lane_elem<N>(w, j);
      if (is_nan_f(q[j])) {
        q[j] = is_nan_f(xv) ? 0.f : copysignf(0.f, xv);
        nan_bits |= is_nan_f(xv) ? (1u << j) : 0u;
      }
    }
  }
}

// Clip-mask word: bit j set when |q_j| <= 448 (the sign bit of 448 - |q_j|
// is clear exactly then, infinities included).
template <int N>
__device__ __forceinline__ uint32_t mx8_keep_bits(const float (&q)[N]) {
  uint32_t clip = 0;
#pragma unroll
  for (int j = N - 1; j >= 0; --j) clip = __builtin_amdgcn_alignbit(clip, __float_as_uint(448.f - fabsf(q[j])), 31);
  return ~clip & ((1u << N) - 1u);
}

// Round-to-nearest-even E4M3FN codes of the clipped quotients, dword k
// holding elements 4k..4k+3 (byte j = element 4k + j).
template <int N>
__device__ __forceinline__ void fp8_rne_codes(const float (&qc)[N], uint32_t (&C)[N / 4]) {
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(qc[4 * k], qc[4 * k + 1], 0, false);
    C[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(qc[4 * k + 2], qc[4 * k + 3], (int)lo, true);
  }
}

}  // namespace trace_dev
