// libtrace microscaled products for gfx950: y = A W^T on MXFP4 weights and
// MXFP4 or MXFP8 activations, for one weight or one per group of packed rows
// (routed experts).
//
//   y[m, n] = sum over k of 2^(sa[m, k/32] - 127) a[m, k] * 2^(sw[n, k/32] - 127) w[n, k]
//
// The scaled matrix instructions take the codes and the E8M0 bytes as they
// are stored; sums are fp32, rounded once to bf16.  W is the instruction's
// first operand, so a lane's consecutive results are consecutive n of one row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"
#include "fp4_block.h"
#include "launch.h"
#include "launch_mx.h"
#include "mx_mfma.h"

namespace trace_dev {

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const bf16x2 p = __builtin_convertvector((f32x2){a, b}, bf16x2);
  uint32_t u;
  __builtin_memcpy(&u, &p, 4);
  return u;
}

// ---------------------------------------------------------------------------
// Few rows.  A workgroup owns 16 columns of W's rows n times kNF and up to
// 16 * kMF rows of one group; its kWaves waves take the 128-long steps of k
// in turn and their partial sums meet in LDS, added in the order of the
// waves.  Operands go straight from memory to registers: no row of W is used
// twice, and this is bound by W's bytes (or, for one token, by latency).
// ---------------------------------------------------------------------------
template <int kFmt, int kMF, int kNF, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void mx_skinny_kernel(trace_host::MxProductArgs p, uint32_t col_tiles) {
  __shared__ v4f sums[kWaves][kMF * kNF][64];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t r = lane & 15, g = lane >> 4;
  const uint64_t row_tile = blockIdx.x / col_tiles;
  const uint32_t n0 = (uint32_t)(blockIdx.x - row_tile * col_tiles) * (16 * kNF);
  RowTile t;
  if (p.offsets) {
    if (!find_row_tile(p.offsets, p.groups, p.rows, 16 * kMF, row_tile, t)) return;
  } else {
    t.group = 0;
    t.first = row_tile * (16 * kMF);
    t.count = (uint32_t)(p.rows - t.first < 16 * kMF ? p.rows - t.first : 16 * kMF);
  }
  const bool behind = t.group >= p.groups;  // rows of no group: zeros
  const uint32_t blocks = p.k / 32;
  const uint32_t a_pitch = kFmt == trace_host::kE2M1 ? p.k / 2 : p.k;
  v4f acc[kMF][kNF] = {};
  if (!behind) {
    const uint8_t* wc = p.w_codes + ((uint64_t)t.group * p.n + n0) * (p.k / 2);
    const uint8_t* ws = p.w_scales + ((uint64_t)t.group * p.n + n0) * blocks;
    uint32_t w_row[kNF];
#pragma unroll
    for (int f = 0; f < kNF; ++f) {
      const uint32_t n = 16 * f + r;
      w_row[f] = n0 + n < p.n ? n : r;  // past the last column: any row of the tile, its results are dropped
    }
    const uint8_t* ac[kMF];
    const uint8_t* as[kMF];
    bool a_ok[kMF];
#pragma unroll
    for (int f = 0; f < kMF; ++f) {
      const uint32_t m = 16 * f + r;
      a_ok[f] = m < t.count;
      uint64_t src = t.first + (a_ok[f] ? m : 0);
      if (p.row_index) {
        const int64_t i = p.row_index[src];
        a_ok[f] = a_ok[f] && i >= 0 && i < (int64_t)p.src_rows;
        src = a_ok[f] ? (uint64_t)i : 0;
      }
      ac[f] = p.a_codes + src * a_pitch;
      as[f] = p.a_scales + src * blocks;
    }
    const uint32_t steps = (p.k + 127) / 128;
    for (uint32_t s = wave; s < steps; s += kWaves) {
      const uint32_t b = 4 * s + g;  // this lane's block of k
      const bool in = b < blocks;
      v8i wv[kNF], av[kMF];
      int wsc[kNF], asc[kMF];
#pragma unroll
      for (int f = 0; f < kNF; ++f) {
        v4i c = {0, 0, 0, 0};
        wsc[f] = 127;
        if (in) {
          c = *reinterpret_cast<const v4i*>(wc + (uint64_t)w_row[f] * (p.k / 2) + 16 * b);
          wsc[f] = ws[(uint64_t)w_row[f] * blocks + b];
        }
        wv[f] = widen(c);
      }
#pragma unroll
      for (int f = 0; f < kMF; ++f) {
        v4i c = {0, 0, 0, 0}, d = {0, 0, 0, 0};
        asc[f] = 127;
        if (kFmt == trace_host::kE2M1) {
          if (in && a_ok[f]) c = *reinterpret_cast<const v4i*>(ac[f] + 16 * b);
          av[f] = widen(c);
        } else {
          const uint32_t k0 = 128 * s + 16 * g;
          if (k0 < p.k && a_ok[f]) c = *reinterpret_cast<const v4i*>(ac[f] + k0);
          if (k0 + 64 < p.k && a_ok[f]) d = *reinterpret_cast<const v4i*>(ac[f] + k0 + 64);
          av[f] = join(c, d);
        }
        if (in && a_ok[f]) asc[f] = as[f][b];
      }
#pragma unroll
      for (int i = 0; i < kMF; ++i)
#pragma unroll
        for (int j = 0; j < kNF; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              wv[j], av[i], acc[i][j], kSelE2M1, kFmt == trace_host::kE2M1 ? kSelE2M1 : kSelE4M3, 0, wsc[j], 0, asc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kMF; ++i)
#pragma unroll
    for (int j = 0; j < kNF; ++j) sums[wave][i * kNF + j][lane] = acc[i][j];
  __syncthreads();
  for (uint32_t f = wave; f < kMF * kNF; f += kWaves) {
    v4f v = sums[0][f][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += sums[w][f][lane];
    const uint32_t m = 16 * (f / kNF) + r, n = n0 + 16 * (f % kNF) + 4 * g;
    if (m < t.count && n < p.n)
      *reinterpret_cast<uint2*>(p.y + (t.first + m) * p.n + n) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
  }
}

}  // namespace trace_dev

namespace trace_host {

using namespace trace_dev;

template <int kFmt, int kMF, int kNF, int kWaves>
static hipError_t launch_skinny(const MxProductArgs& p, hipStream_t stream) {
  const uint32_t cols = (p.n + 16 * kNF - 1) / (16 * kNF);
  const uint64_t row_tiles = p.offsets ? max_row_tiles(p.rows, p.groups, 16 * kMF) : (p.rows + 16 * kMF - 1) / (16 * kMF);
  if (row_tiles * cols * (64 * kWaves) > 0xffffffffull) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((mx_skinny_kernel<kFmt, kMF, kNF, kWaves>), dim3((unsigned)(row_tiles * cols)), dim3(64 * kWaves),
                     0, stream, p, cols);
  return hipGetLastError();
}

template <int kFmt>
static hipError_t launch_product(const MxProductArgs& p, hipStream_t stream) {
  return launch_skinny<kFmt, 2, 2, 4>(p, stream);
}

hipError_t launch_mx_product(MxFormat fmt, const MxProductArgs& p, hipStream_t stream) {
  return fmt == kE2M1 ? launch_product<kE2M1>(p, stream) : launch_product<kE4M3>(p, stream);
}

}  // namespace trace_host
