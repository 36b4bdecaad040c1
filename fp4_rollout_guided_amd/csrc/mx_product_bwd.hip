// libtrace gradients of the microscaled products for gfx950, for one weight
// or one per group of packed rows:
//
//   to the activations  gx[m, k] = sum over n of gy[m, n] W[n, k]
//   to the weights      gw[n, k] = sum over m of gy[m, n] A[m, k]
//
// W and A are the codes' values; the rounding that made them passes the
// gradient straight through inside its clip range, so each result is zeroed
// where its tensor's clip mask is 0.  gy is bf16 and the codes' values are
// exact in bf16, so both run on the bf16 matrix instructions with fp32 sums,
// rounded once.
//
// Both are one kernel: D[p, k] = sum over c of G(p, c) Q[c, k], where Q's
// codes lie row by row along k and are turned into bf16 on the way into LDS.
// The matrix instruction wants eight consecutive c of one k per lane, so Q
// (and, for the weights, gy) is read back from LDS transposed
// (ds_read_b64_tr_b16: 16 lanes read four rows of 16 values, lane i gets
// column i).  Q is the first operand: a lane's results are consecutive k.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"
#include "fp4_block.h"
#include "launch.h"
#include "launch_mx.h"
#include "mx_mfma.h"

namespace trace_dev {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr uint32_t kTileP = 128, kTileK = 128, kTileC = 32;
// Row pitch of a tile that is read transposed: 64 bytes more than a multiple
// of 256, so that the four rows that 32 lanes read together lie in different
// LDS banks.
constexpr uint32_t kTrPitch = 2 * kTileK + 64;

// The E8M0 byte as the float whose exponent the scaling conversions use.
__device__ __forceinline__ float e8m0_operand(uint32_t b) { return __uint_as_float(b << 23); }

// 16 codes to bf16: out[i] holds elements 2i and 2i + 1.
template <int kFmt>
__device__ __forceinline__ void decode16(const uint32_t (&c)[4], float s, uint32_t (&out)[8]) {
  bf16x2 v[8];
  if (kFmt == trace_host::kE2M1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[4 * i] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], s, 0);
      v[4 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], s, 1);
      v[4 * i + 2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], s, 2);
      v[4 * i + 3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], s, 3);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, false);
      v[2 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, true);
    }
  }
  __builtin_memcpy(out, v, sizeof(v));
}

// Eight consecutive c (rows 16 kk + 8 h ..) of one of 32 columns from a tile
// of kTrPitch-byte rows; kSwap: the columns' bits 2 and 3 trade places.
template <bool kSwap>
__device__ __forceinline__ v8bf read_transposed(const char* tile, uint32_t col0, uint32_t kk, uint32_t lane) {
  const uint32_t j = lane & 15;
  const uint32_t q = kSwap ? (((j & 1) << 1) | ((j & 3) >> 1)) : (j & 3);
  const uint32_t row = 16 * kk + 8 * (lane >> 5) + (j >> 2);
  const uint32_t at = row * kTrPitch + 2 * (col0 + 16 * ((lane >> 4) & 1) + 4 * q);
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(tile + at));
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(tile + at + 4 * kTrPitch));
  v8bf out;
  __builtin_memcpy(&out, &lo, 8);
  __builtin_memcpy(reinterpret_cast<char*>(&out) + 8, &hi, 8);
  return out;
}

// kWeight: D = gw of one group (p = n, c = the group's rows m); otherwise
// D = gx of a row tile (p = m, c = n).  parts > 1 (kWeight, one group only):
// the contraction's part blockIdx.y, as fp32 to p.partial.
template <bool kWeight, int kFmt>
__global__ __launch_bounds__(256) void mx_grad_kernel(trace_host::MxGradArgs p, uint32_t k_tiles, uint32_t p_tiles,
                                                      uint32_t parts) {
  __shared__ __attribute__((aligned(16))) char g_tile[kWeight ? kTileC * kTrPitch : kTileP * 2 * kTileC];
  __shared__ __attribute__((aligned(16))) char q_tile[kTileC * kTrPitch];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t k0 = (blockIdx.x % k_tiles) * kTileK;
  const uint64_t outer = blockIdx.x / k_tiles;
  RowTile t{0, 0, 0};       // rows of the tile (gx) or of the group (gw)
  uint32_t p0 = 0;          // first n (gw)
  uint64_t c_begin = 0, c_end = p.n;
  if (kWeight) {
    p0 = (uint32_t)(outer % p_tiles) * kTileP;
    t.group = (uint32_t)(outer / p_tiles);
    if (p.offsets) {
      t.count = group_rows(p.offsets, t.group, p.groups, p.rows, t.first);
    } else {
      t.count = (uint32_t)p.rows;
    }
    const uint32_t steps = (t.count + kTileC - 1) / kTileC;
    c_begin = (uint64_t)(blockIdx.y * (uint64_t)steps / parts) * kTileC;
    c_end = (uint64_t)((blockIdx.y + 1) * (uint64_t)steps / parts) * kTileC;
    if (c_end > t.count) c_end = t.count;
  } else if (p.offsets) {
    if (!find_row_tile(p.offsets, p.groups, p.rows, kTileP, outer, t)) return;
    if (t.group >= p.groups) c_end = 0;  // rows of no group: zeros
  } else {
    t.first = outer * kTileP;
    t.count = (uint32_t)(p.rows - t.first < kTileP ? p.rows - t.first : kTileP);
  }
  const uint32_t q_pitch = kFmt == trace_host::kE2M1 ? p.k / 2 : p.k;
  const uint32_t blocks = p.k / 32;
  const uint8_t* qc = p.q_codes + (kWeight ? 0 : (uint64_t)t.group * p.n * q_pitch);
  const uint8_t* qs = p.q_scales + (kWeight ? 0 : (uint64_t)t.group * p.n * blocks);
  const uint32_t wp = (wave >> 1) * 64, wk = (wave & 1) * 64;
  v16f acc[2][2] = {};  // [k fragment][p fragment]
  for (uint64_t c0 = c_begin; c0 < c_end; c0 += kTileC) {
    __syncthreads();
    // gy
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (kWeight) {
        const uint32_t c = threadIdx.x / 16 + 16 * i, col = 8 * (threadIdx.x & 15);
        if (c0 + c < c_end && p0 + col < p.n)
          v = *reinterpret_cast<const uint4*>(p.grad_y + (t.first + c0 + c) * p.n + p0 + col);
        *reinterpret_cast<uint4*>(g_tile + c * kTrPitch + 2 * col) = v;
      } else {
        const uint32_t m = threadIdx.x / 4 + 64 * i, ch = threadIdx.x & 3;
        if (m < t.count && c0 + 8 * ch < c_end)
          v = *reinterpret_cast<const uint4*>(p.grad_y + (t.first + m) * p.n + c0 + 8 * ch);
        *reinterpret_cast<uint4*>(g_tile + m * 64 + 16 * (ch ^ ((m >> 1) & 3))) = v;
      }
    }
    // Q: 16 codes of row c
    {
      const uint32_t c = threadIdx.x / 8, k = k0 + 16 * (threadIdx.x & 7);
      uint32_t code[4] = {0, 0, 0, 0};
      float s = 1.f;
      bool ok = c0 + c < c_end && k < p.k;
      uint64_t row = c0 + c;
      if (kWeight) {
        row += t.first;
        if (p.row_index && ok) {
          const int64_t src = p.row_index[row];
          ok = src >= 0 && src < (int64_t)p.src_rows;
          row = (uint64_t)src;
        }
      }
      if (ok) {
        s = e8m0_operand(qs[row * blocks + k / 32]);
        if (kFmt == trace_host::kE2M1) {
          const uint2 v = *reinterpret_cast<const uint2*>(qc + row * q_pitch + k / 2);
          code[0] = v.x; code[1] = v.y;
        } else {
          const uint4 v = *reinterpret_cast<const uint4*>(qc + row * q_pitch + k);
          code[0] = v.x; code[1] = v.y; code[2] = v.z; code[3] = v.w;
        }
      }
      uint32_t out[8];
      decode16<kFmt>(code, s, out);
      uint4* dst = reinterpret_cast<uint4*>(q_tile + c * kTrPitch + 32 * (threadIdx.x & 7));
      dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
      dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
    __syncthreads();
#pragma unroll
    for (uint32_t kk = 0; kk < 2; ++kk) {
      v8bf q[2], gg[2];
#pragma unroll
      for (uint32_t f = 0; f < 2; ++f) {
        q[f] = read_transposed<true>(q_tile, wk + 32 * f, kk, lane);
        if (kWeight) {
          gg[f] = read_transposed<false>(g_tile, wp + 32 * f, kk, lane);
        } else {
          const uint32_t m = wp + 32 * f + (lane & 31), ch = 2 * kk + (lane >> 5);
          gg[f] = *reinterpret_cast<const v8bf*>(g_tile + m * 64 + 16 * (ch ^ ((m >> 1) & 3)));
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q[i], gg[j], acc[i][j], 0, 0, 0);
    }
  }
  // register e of a fragment: k = 16 (e / 8) + 8 (lane / 32) + e % 8
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t pp = wp + 32 * j + (lane & 31);
    if (kWeight ? p0 + pp >= p.n : pp >= t.count) continue;
    const uint64_t row = kWeight ? (uint64_t)t.group * p.n + p0 + pp : t.first + pp;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 16; e += 8) {
        const uint32_t k = k0 + wk + 32 * i + 2 * e + 8 * (lane >> 5);
        if (k >= p.k) continue;
        const v16f& a = acc[i][j];
        if (kWeight && parts > 1) {
          float* dst = p.partial + ((uint64_t)blockIdx.y * p.n + p0 + pp) * p.k + k;
          *reinterpret_cast<v4f*>(dst) = (v4f){a[e], a[e + 1], a[e + 2], a[e + 3]};
          *reinterpret_cast<v4f*>(dst + 4) = (v4f){a[e + 4], a[e + 5], a[e + 6], a[e + 7]};
          continue;
        }
        const uint32_t keep = p.mask ? p.mask[(row * p.k + k) / 8] : 0xffu;
        uint32_t out[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const float lo = (keep >> (2 * h)) & 1 ? a[e + 2 * h] : 0.f, hi = (keep >> (2 * h + 1)) & 1 ? a[e + 2 * h + 1] : 0.f;
          const bf16x2 v = __builtin_convertvector((f32x2){lo, hi}, bf16x2);
          __builtin_memcpy(&out[h], &v, 4);
        }
        *reinterpret_cast<uint4*>(p.grad + row * p.k + k) = make_uint4(out[0], out[1], out[2], out[3]);
      }
  }
}

// Sum of the contraction's parts, in their order, rounded and masked.
__global__ __launch_bounds__(kThreads) void mx_grad_join_kernel(const float* __restrict__ partial, uint32_t parts,
                                                                uint64_t nvec, const uint8_t* __restrict__ mask,
                                                                uint4* __restrict__ grad) {
  const uint64_t stride = (uint64_t)gridDim.x * kThreads;
  for (uint64_t g = (uint64_t)blockIdx.x * kThreads + threadIdx.x; g < nvec; g += stride) {
    v4f a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
    for (uint32_t s = 0; s < parts; ++s) {
      const v4f* src = reinterpret_cast<const v4f*>(partial) + 2 * (s * nvec + g);
      a += src[0];
      b += src[1];
    }
    const uint32_t keep = mask ? mask[g] : 0xffu;
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    uint32_t out[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const float lo = (keep >> (2 * h)) & 1 ? v[2 * h] : 0.f, hi = (keep >> (2 * h + 1)) & 1 ? v[2 * h + 1] : 0.f;
      const bf16x2 w = __builtin_convertvector((f32x2){lo, hi}, bf16x2);
      __builtin_memcpy(&out[h], &w, 4);
    }
    grad[g] = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

}  // namespace trace_dev

namespace trace_host {

using namespace trace_dev;

hipError_t launch_mx_grad_input(const MxGradArgs& p, hipStream_t stream) {
  const uint32_t k_tiles = (p.k + kTileK - 1) / kTileK;
  const uint64_t row_tiles = p.offsets ? max_row_tiles(p.rows, p.groups, kTileP) : (p.rows + kTileP - 1) / kTileP;
  if (row_tiles * k_tiles * 256 > 0xffffffffull) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((mx_grad_kernel<false, kE2M1>), dim3((unsigned)(row_tiles * k_tiles)), dim3(256), 0, stream, p,
                     k_tiles, 1u, 1u);
  return hipGetLastError();
}

uint32_t mx_grad_weight_parts(uint64_t rows, uint32_t groups, uint32_t n, uint32_t k) {
  (void)rows; (void)groups; (void)n; (void)k;
  return 1;
}

hipError_t launch_mx_grad_weight(MxFormat fmt, const MxGradArgs& p, hipStream_t stream) {
  const uint32_t k_tiles = (p.k + kTileK - 1) / kTileK, p_tiles = (p.n + kTileP - 1) / kTileP;
  const uint64_t tiles = (uint64_t)k_tiles * p_tiles * p.groups;
  if (tiles * 256 > 0xffffffffull) return hipErrorInvalidConfiguration;
  const uint32_t parts = mx_grad_weight_parts(p.rows, p.groups, p.n, p.k);
  const dim3 grid((unsigned)tiles, parts), block(256);
  if (fmt == kE2M1)
    hipLaunchKernelGGL((mx_grad_kernel<true, kE2M1>), grid, block, 0, stream, p, k_tiles, p_tiles, parts);
  else
    hipLaunchKernelGGL((mx_grad_kernel<true, kE4M3>), grid, block, 0, stream, p, k_tiles, p_tiles, parts);
  if (parts > 1) {
    const uint64_t nvec = (uint64_t)p.n * p.k / 8;
    const uint64_t g = (nvec + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(mx_grad_join_kernel, dim3((unsigned)(g < kMaxGroups ? g : kMaxGroups)), block, 0, stream,
                       p.partial, parts, nvec, p.mask, reinterpret_cast<uint4*>(p.grad));
  }
  return hipGetLastError();
}

}  // namespace trace_host
