// libtrace gradients of the microscaled products for gfx950, for one weight
// or one per group of packed rows:
//
//   to the activations  gx[m, k] = sum over n of gy[m, n] W[n, k]
//   to the weights      gw[n, k] = sum over m of gy[m, n] A[m, k]
//
// W and A are the codes' values; the rounding that made them passes the
// gradient straight through inside its clip range, so each result is zeroed
// where its tensor's clip mask is 0.  gy is bf16 and the codes' values are exact
// in bf16 from 2^-130 up to its largest, 2^128 (past that they are infinite; no
// finite tensor's rounding writes such), so both run on the bf16 matrix
// instructions with fp32 sums, rounded once or, for packed rows that are summed
// further, left as they are.
//
// Both are one kernel: D[p, k] = sum over c of G(p, c) Q[c, k], where Q's
// codes lie row by row along k and are turned into bf16 on the way into LDS.
// The matrix instruction wants eight consecutive c of one k per lane, so Q
// (and, for the weights, gy) is read back from LDS transposed
// (ds_read_b64_tr_b16: 16 lanes read four rows of 16 values, lane i gets
// column i).  Q is the first operand: a lane's results are consecutive k.
//
// Measured: 16384 x 4096 x 2048 at 1.07 PFLOP/s (gx 259 us, gw and the sum of its
// two parts 253 us), the matrix units busy 55% of the time and LDS half of it:
// writing the decoded tiles and reading them back transposed take as long as the
// arithmetic and are under it only in part.  Experts' weights (128 of 1536 x
// 2048, 512 rows each) take 515 us alone and 640 behind the other kernels of a
// backward pass, a quarter of it their 805 MB.
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

// The E8M0 byte as the float whose exponent the scaling conversions use.
__device__ __forceinline__ float e8m0_operand(uint32_t b) { return __uint_as_float(b << 23); }

// Eight codes to bf16: out[i] holds elements 2i and 2i + 1.
template <int kFmt>
__device__ __forceinline__ uint4 decode8(const uint32_t* c, float s) {
  bf16x2 v[4];
  if (kFmt == trace_host::kE2M1) {
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[0], s, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[0], s, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[0], s, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[0], s, 3);
  } else {
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], s, false);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], s, true);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], s, false);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], s, true);
  }
  uint4 out;
  __builtin_memcpy(&out, v, sizeof(out));
  return out;
}

// This wave's LDS accesses are done; meet the workgroup's other waves.  Loads
// to registers stay under way.
__device__ __forceinline__ void grad_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ v8bf transposed(const char* at, uint32_t pitch) {
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)at);
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + 4 * pitch));
  v8bf out;
  __builtin_memcpy(&out, &lo, 8);
  __builtin_memcpy(reinterpret_cast<char*>(&out) + 8, &hi, 8);
  return out;
}

// kWeight: D = gw of one group (p = n, c = the group's rows m); otherwise
// D = gx of a row tile (p = m, c = n).  A workgroup of 2 x 2 waves owns
// 64 kKF k times 64 kPF p, each wave a quarter as kKF x kPF results of
// 32 x 32.  The contraction runs in stages of kC, in two LDS buffers with one
// barrier per stage; the next stage is decoded and placed in LDS, and the two
// after it fetched to registers, under the arithmetic.
//
// LDS layouts.  Q is [c][k]: 64 bytes per block of 32 k, a lane's four
// 16-byte pieces of a block permuted by the row's and the block's low bits so
// that sixteen lanes write different banks; rows are 64 bytes more than a
// multiple of 256 apart, so that the four rows that 32 lanes read transposed
// lie in different banks.  gy is [c][p] likewise for gw; for gx it is [p][c]
// with its pieces permuted by the row's bits.
// kF32: results in fp32 (gx of packed rows, which are summed further).
// parts > 1 (kWeight, one group only): the contraction's part blockIdx.y, as
// fp32 to p.partial.
template <bool kWeight, int kFmt, bool kGather, bool kF32, int kKF, int kPF, int kPerCu>
__global__ __launch_bounds__(256, kPerCu) void mx_grad_kernel(trace_host::MxGradArgs p, uint32_t k_tiles,
                                                              uint32_t p_tiles, uint32_t parts) {
  constexpr bool kFp4 = kFmt == trace_host::kE2M1;
  constexpr uint32_t kK = 64 * kKF, kP = 64 * kPF;
  constexpr uint32_t kC = 256 * 32 / kK;              // one block of Q per lane and stage
  constexpr uint32_t kQPitch = 2 * kK + 64, kGPitch = kWeight ? 2 * kP + 64 : 2 * kC;
  constexpr uint32_t kQBytes = kC * kQPitch, kGBytes = kWeight ? kC * kGPitch : kP * kGPitch;
  constexpr uint32_t kGLoads = kP * kC * 2 / 4096;    // 16-byte loads per lane and stage
  constexpr uint32_t kQDwords = kFp4 ? 4 : 8;
  __shared__ __attribute__((aligned(256))) char q_buf[2][kQBytes];
  __shared__ __attribute__((aligned(256))) char g_buf[2][kGBytes];

  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint64_t tiles;
  if (kWeight)
    tiles = (uint64_t)p.groups * p_tiles * k_tiles;
  else
    tiles = (p.offsets ? count_row_tiles(p.offsets, p.groups, p.rows, kP) : (p.rows + kP - 1) / kP) * k_tiles;
  const uint64_t tile = xcd_tile(blockIdx.x, tiles);
  if (tile >= tiles) return;
  const uint64_t outer = tile / k_tiles;
  const uint32_t k0 = (uint32_t)(tile - outer * k_tiles) * kK;
  RowTile t{0, 0, 0};  // rows of the tile (gx) or of the group (gw)
  uint32_t p0 = 0;     // first n (gw)
  uint32_t c_begin = 0, c_end = p.n;
  if (kWeight) {
    t.group = (uint32_t)(outer / p_tiles);
    p0 = (uint32_t)(outer - (uint64_t)t.group * p_tiles) * kP;
    if (p.offsets)
      t.count = group_rows(p.offsets, t.group, p.groups, p.rows, t.first);
    else
      t.count = (uint32_t)p.rows;
    const uint64_t steps = (t.count + kC - 1) / kC;
    c_begin = (uint32_t)(blockIdx.y * steps / parts) * kC;
    c_end = (uint32_t)((blockIdx.y + 1) * steps / parts) * kC;
    if (c_end > t.count) c_end = t.count;
  } else if (p.offsets) {
    if (!find_row_tile(p.offsets, p.groups, p.rows, kP, outer, t)) return;
    if (t.group >= p.groups) c_end = 0;  // rows of no group: zeros
  } else {
    t.first = outer * kP;
    t.count = (uint32_t)(p.rows - t.first < kP ? p.rows - t.first : kP);
  }
  const uint32_t length = c_end > c_begin ? c_end - c_begin : 0;
  const uint32_t stages = (length + kC - 1) / kC;
  const uint32_t q_pitch = kFp4 ? p.k / 2 : p.k, blocks = p.k / 32;

  // Q: this lane's row of a stage and its block of the tile's k.  Columns
  // past p.k and rows p past the end read something valid: their results are
  // dropped.  Rows c past the end, and rows without a source, are zeros.
  const uint32_t q_row = threadIdx.x / (kK / 32), q_blk = threadIdx.x % (kK / 32);
  const uint32_t q_col = k0 + 32 * q_blk < p.k ? k0 + 32 * q_blk : k0;
  const uint64_t q_first = kWeight ? t.first + c_begin : (uint64_t)(t.group < p.groups ? t.group : 0) * p.n;
  const uint8_t* qc = p.q_codes + (kFp4 ? q_col / 2 : q_col);
  const uint8_t* qs = p.q_scales + q_col / 32;
  const uint16_t* g_from[kGLoads];
  uint32_t g_c[kGLoads];  // c within the stage
#pragma unroll
  for (uint32_t i = 0; i < kGLoads; ++i) {
    if (kWeight) {
      g_c[i] = (threadIdx.x + 256 * i) / (kP / 8);
      const uint32_t col = 8 * ((threadIdx.x + 256 * i) % (kP / 8));
      g_from[i] = p.grad_y + (t.first + c_begin + g_c[i]) * p.n + (p0 + col < p.n ? p0 + col : p0);
    } else {
      const uint32_t m = (threadIdx.x + 256 * i) / (kC / 8);
      g_c[i] = 8 * ((threadIdx.x + 256 * i) % (kC / 8));
      g_from[i] = p.grad_y + (t.first + (m < t.count ? m : 0)) * p.n + g_c[i];
    }
  }

  struct Held {  // a stage on its way to LDS
    uint32_t q[kQDwords], q_scale;
    v4i g[kGLoads];
  };
  Held held[2];
  int64_t q_index = 0;  // kGather: the source row of the stage to be fetched next
  const auto fetch_index = [&](uint32_t st, bool may_end) -> int64_t {
    const uint32_t c = kC * st + q_row;
    return kGather && (!may_end || c < length) ? p.row_index[q_first + c] : -1;
  };
  // may_end: the stage may end early
  const auto fetch = [&](uint32_t st, Held& to, bool may_end) {
    const uint32_t c = kC * st + q_row;
    uint64_t row = q_first + c;
    bool ok = !may_end || c < length;
    if (kGather) {
      ok = ok && q_index >= 0 && q_index < (int64_t)p.src_rows;
      row = ok ? (uint64_t)q_index : 0;
    }
    to.q_scale = 127;
#pragma unroll
    for (uint32_t d = 0; d < kQDwords; ++d) to.q[d] = 0;
    if ((!may_end && !kGather) || ok) {
      __builtin_memcpy(to.q, __builtin_assume_aligned(qc + row * q_pitch, 16), 4 * kQDwords);
      to.q_scale = qs[row * blocks];
    }
#pragma unroll
    for (uint32_t i = 0; i < kGLoads; ++i) {
      v4i v = {0, 0, 0, 0};
      if (!may_end || kC * st + g_c[i] < length)
        v = *reinterpret_cast<const v4i*>(g_from[i] + (uint64_t)kC * st * (kWeight ? p.n : 1));
      to.g[i] = v;
    }
  };
  const uint32_t q_swap = ((q_blk >> 2) & 1) | ((q_row & 1) << 1);
  const auto place = [&](uint32_t st, const Held& from) {
    char* q = q_buf[st & 1] + q_row * kQPitch + 64 * q_blk;
    const float s = e8m0_operand(from.q_scale);
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(q + 16 * (i ^ q_swap)) = decode8<kFmt>(from.q + (kFp4 ? i : 2 * i), s);
    char* g = g_buf[st & 1];
#pragma unroll
    for (uint32_t i = 0; i < kGLoads; ++i) {
      const uint32_t id = threadIdx.x + 256 * i;
      if (kWeight) {
        *reinterpret_cast<v4i*>(g + id / (kP / 8) * kGPitch + 16 * (id % (kP / 8))) = from.g[i];
      } else {
        const uint32_t m = id / (kC / 8), piece = id % (kC / 8);
        *reinterpret_cast<v4i*>(g + m * kGPitch + 16 * (piece ^ (kC == 32 ? (m >> 2) & 3 : (m >> 1) & 7))) = from.g[i];
      }
    }
  };

  // Where this lane reads.  Transposed: lane j of 16 reads row j / 4 and four
  // of the 16 columns, and gets column j.  Q's columns 4..7 and 8..11 of every
  // 16 trade places, so that a lane's eight consecutive results are eight
  // consecutive k.
  const uint32_t wk = 32 * kKF * (wave >> 1), wp = 32 * kPF * (wave & 1);
  const uint32_t h = lane >> 5, r = lane & 31, j = lane & 15, half = (lane >> 4) & 1;
  const uint32_t quad = ((j & 1) << 1) | ((j >> 1) & 1);
  const uint32_t tr_row = 8 * h + (j >> 2);
  // piece 2 half + quad / 2 of the block, permuted by the row's lowest bit
  // here and by bit 2 of the block below; rows 4 apart have the same bit
  const uint32_t q_at = tr_row * kQPitch + 16 * ((2 * half + (quad >> 1)) ^ (2 * (tr_row & 1))) + 8 * (quad & 1);
  const uint32_t g_at = kWeight ? tr_row * kGPitch + 2 * (wp + 16 * half + 4 * (j & 3))
                                : (wp + r) * kGPitch + 16 * (h ^ (kC == 32 ? (r >> 2) & 3 : (r >> 1) & 7));
  v16f acc[kKF][kPF] = {};
  constexpr uint32_t kSteps = kC / 16;
  v8bf qf[2][kKF], gf[2][kPF];
  // operands of k-step kk of a stage
  const auto read_step = [&](uint32_t st, uint32_t kk, v8bf(&qv)[kKF], v8bf(&gv)[kPF]) {
    const char* q = q_buf[st & 1] + 16 * kk * kQPitch;
    const char* g = g_buf[st & 1];
#pragma unroll
    for (uint32_t f = 0; f < kPF; ++f) {
      if (kWeight)
        gv[f] = transposed(g + 16 * kk * kGPitch + g_at + 64 * f, kGPitch);
      else
        gv[f] = *reinterpret_cast<const v8bf*>(g + (g_at ^ (32 * kk)) + 32 * f * kGPitch);
    }
#pragma unroll
    for (uint32_t f = 0; f < kKF; ++f) {
      const uint32_t blk = wk / 32 + f;
      qv[f] = transposed(q + (q_at ^ (16 * ((blk >> 2) & 1))) + 64 * blk, kQPitch);
    }
  };
  const auto multiply = [&](const v8bf(&qv)[kKF], const v8bf(&gv)[kPF]) {
#pragma unroll
    for (int a = 0; a < kKF; ++a)
#pragma unroll
      for (int b = 0; b < kPF; ++b) acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qv[a], gv[b], acc[a][b], 0, 0, 0);
  };
  // One stage, whose first k-step has been read: each further step is read
  // under the arithmetic of the one before, and the next stage's first step
  // under the last one's.  next: what holds stage st + 1, and then st + 3.
  // steady: stages st + 1 to st + 4 exist in full.  A wave at its arithmetic
  // goes before one that decodes (16384 x 4096 x 2048, gx: 255 us against 267,
  // gw: 247 against 267).
  const auto stage = [&](uint32_t st, Held& next, bool steady) {
    read_step(st, 1, qf[1], gf[1]);
    __builtin_amdgcn_s_setprio(0);
    if (steady || st + 1 < stages) place(st + 1, next);
    if (steady || st + 3 < stages) fetch(st + 3, next, !steady);
    if (steady || st + 4 < stages) q_index = fetch_index(st + 4, !steady);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (uint32_t kk = 0; kk + 1 < kSteps; ++kk) {
      __builtin_amdgcn_s_setprio(1);
      multiply(qf[kk & 1], gf[kk & 1]);
      if (kk + 2 < kSteps) read_step(st, kk + 2, qf[kk & 1], gf[kk & 1]);
    }
    __builtin_amdgcn_sched_barrier(0);
    grad_barrier();
    if (steady || st + 1 < stages) read_step(st + 1, 0, qf[kSteps & 1], gf[kSteps & 1]);
    multiply(qf[(kSteps - 1) & 1], gf[(kSteps - 1) & 1]);
    __builtin_amdgcn_sched_barrier(0);
  };
  static_assert(kSteps % 2 == 0, "a stage starts with the first of the two sets of operands");
  if (stages) {
    q_index = fetch_index(0, true);
    const int64_t index1 = fetch_index(1, true), index2 = fetch_index(2, true), index3 = fetch_index(3, true);
    fetch(0, held[0], true);
    q_index = index1;
    if (stages > 1) fetch(1, held[1], true);
    place(0, held[0]);
    q_index = index2;
    if (stages > 2) fetch(2, held[0], true);
    q_index = index3;
    grad_barrier();
    read_step(0, 0, qf[0], gf[0]);
  }
  uint32_t st = 0;
  for (; (st + 6) * kC <= length; st += 2) {
    stage(st, held[1], true);
    stage(st + 1, held[0], true);
  }
  for (; st < stages; st += 2) {
    stage(st, held[1], false);
    if (st + 1 < stages) stage(st + 1, held[0], false);
  }

  // register e of a result: k = 16 (e / 8) + 8 h + e % 8, p = lane % 32
  const bool masked = p.mask && !(kWeight && parts > 1);
  uint32_t keep[kPF][kKF];
#pragma unroll
  for (int b = 0; b < kPF; ++b) {
    const uint32_t pp = wp + 32 * b + r;
    const bool in = kWeight ? p0 + pp < p.n : pp < t.count;
    const uint64_t row = kWeight ? (uint64_t)t.group * p.n + p0 + pp : t.first + pp;
#pragma unroll
    for (int a = 0; a < kKF; ++a) {
      const uint32_t k = k0 + wk + 32 * a;  // the mask's bits of 32 k are a dword, at any byte multiple of 4 of the mask
      keep[b][a] = ~0u;
      if (masked && in && k < p.k) __builtin_memcpy(&keep[b][a], p.mask + (row * p.k + k) / 8, 4);
    }
  }
  if (kWeight && parts > 1) {
#pragma unroll
    for (int b = 0; b < kPF; ++b) {
      const uint32_t pp = p0 + wp + 32 * b + r;
      if (pp >= p.n) continue;
#pragma unroll
      for (int a = 0; a < kKF; ++a) {
        if (k0 + wk + 32 * a >= p.k) continue;
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
          float* dst = p.partial + ((uint64_t)blockIdx.y * p.n + pp) * p.k + k0 + wk + 32 * a + 2 * e + 8 * h;
          const v16f& v = acc[a][b];
          *reinterpret_cast<v4f*>(dst) = (v4f){v[e], v[e + 1], v[e + 2], v[e + 3]};
          *reinterpret_cast<v4f*>(dst + 4) = (v4f){v[e + 4], v[e + 5], v[e + 6], v[e + 7]};
        }
      }
    }
    return;
  }
  // every wave has passed the barrier after its last LDS read
  if constexpr (kF32) {  // 64 columns at a time
    const RowBlock<16> block{q_buf[0] + 512 * 16 * wave};
    static_assert(4 * 512 * 16 <= 2 * kQBytes && kKF % 2 == 0 && !kWeight, "four waves' blocks fit the tiles' buffers");
#pragma unroll
    for (int b = 0; b < kPF; ++b) {
#pragma unroll
      for (int a0 = 0; a0 < kKF; a0 += 2) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            const uint32_t bits = keep[b][a0 + a] >> (2 * e + 8 * h);
            float v[8];
#pragma unroll
            for (int d = 0; d < 8; ++d) v[d] = (bits >> d) & 1 ? acc[a0 + a][b][e + d] : 0.f;
            put_f32(block, r, 8 * a + e / 2 + 2 * h, v);
          }
        block.drain([&](uint32_t row, uint32_t piece, uint4 v) {
          const uint32_t pp = wp + 32 * b + row, k = k0 + wk + 32 * a0 + 4 * piece;
          if (k < p.k && pp < t.count) store_result(static_cast<float*>(p.grad) + (t.first + pp) * p.k + k, v, p.stream_out);
        });
      }
    }
    return;
  }
  const RowBlock<4 * kKF> block{q_buf[0] + 512 * 4 * kKF * wave};
  static_assert(4 * 512 * 4 * kKF <= 2 * kQBytes, "four waves' blocks fit the tiles' buffers");
#pragma unroll
  for (int b = 0; b < kPF; ++b) {
#pragma unroll
    for (int a = 0; a < kKF; ++a)
#pragma unroll
      for (int e = 0; e < 16; e += 8) {
        const v16f& v = acc[a][b];
        const uint32_t bits = keep[b][a] >> (2 * e + 8 * h);
        uint32_t out[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const float lo = (bits >> (2 * d)) & 1 ? v[e + 2 * d] : 0.f, hi = (bits >> (2 * d + 1)) & 1 ? v[e + 2 * d + 1] : 0.f;
          const bf16x2 w = __builtin_convertvector((f32x2){lo, hi}, bf16x2);
          __builtin_memcpy(&out[d], &w, 4);
        }
        block.put(r, 4 * a + e / 4 + h, make_uint4(out[0], out[1], out[2], out[3]));
      }
    block.drain([&](uint32_t row, uint32_t piece, uint4 v) {
      const uint32_t pp = wp + 32 * b + row, k = k0 + wk + 8 * piece;
      if (k < p.k && (kWeight ? p0 + pp < p.n : pp < t.count)) {
        const uint64_t to = kWeight ? (uint64_t)t.group * p.n + p0 + pp : t.first + pp;
        store_result(static_cast<uint16_t*>(p.grad) + to * p.k + k, v, p.stream_out);
      }
    });
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

// Whether tiles of 128 x 256 fill the compute units (16384 x 4096 x 2048: 258 us
// against 393 in tiles of 64 x 128).
static bool big_tiles(uint64_t p, uint32_t k) { return (p + 127) / 128 * ((k + 255) / 256) >= 512; }

template <bool kF32, int kKF, int kPF, int kPerCu>
static hipError_t grad_input(const MxGradArgs& p, hipStream_t stream) {
  const uint32_t k_tiles = (p.k + 64 * kKF - 1) / (64 * kKF);
  const uint64_t row_tiles = p.offsets ? max_row_tiles(p.rows, p.groups, 64 * kPF) : (p.rows + 64 * kPF - 1) / (64 * kPF);
  const uint64_t grid = (row_tiles * k_tiles + 7) / 8 * 8;
  if (grid * 256 > 0xffffffffull) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((mx_grad_kernel<false, kE2M1, false, kF32, kKF, kPF, kPerCu>), dim3((unsigned)grid), dim3(256), 0, stream,
                     p, k_tiles, 1u, 1u);
  return hipGetLastError();
}

hipError_t launch_mx_grad_input(const MxGradArgs& args, hipStream_t stream) {
  MxGradArgs p = args;
  p.stream_out = past_cache((p.f32 ? 4 : 2) * p.rows * p.k);
  if (p.f32) return big_tiles(p.rows, p.k) ? grad_input<true, 4, 2, 2>(p, stream) : grad_input<true, 2, 1, 2>(p, stream);
  return big_tiles(p.rows, p.k) ? grad_input<false, 4, 2, 2>(p, stream) : grad_input<false, 2, 1, 2>(p, stream);
}

// Tiles and parts of a weight's gradient.  Tiles of 128 x 256 where, with the
// contraction over one weight's rows in up to a part per 1024 rows, they fill
// the compute units twice; else tiles of 64 x 128 and a part per 1024 rows.  The
// parts' sums are written and read once more, so fewer rows to a part cost more
// than they save (2000 x 768 x 2048: 19 us, 28 in three parts; 4096 x 512 x 512:
// 15 us in four parts, 21 in two).
struct GradWeightPlan {
  bool big;
  uint32_t parts;
};
static GradWeightPlan grad_weight_plan(uint64_t rows, uint32_t groups, uint32_t n, uint32_t k) {
  const uint64_t weights = groups ? groups : 1;
  const uint64_t big = (uint64_t)((n + 127) / 128) * ((k + 255) / 256) * weights;
  const uint64_t small = (uint64_t)((n + 63) / 64) * ((k + 127) / 128) * weights;
  if (big >= 512) return {true, 1};
  if (groups || small == 0) return {false, 1};
  const uint64_t big_parts = (512 + big - 1) / big, small_parts = (512 + small - 1) / small;
  if (big_parts <= rows / 1024 && big_parts <= 8) return {true, (uint32_t)big_parts};
  const uint64_t most = rows / 1024 < 32 ? rows / 1024 : 32;
  const uint64_t parts = small_parts < most ? small_parts : most;
  return {false, parts > 1 ? (uint32_t)parts : 1u};
}

uint32_t mx_grad_weight_parts(uint64_t rows, uint32_t groups, uint32_t n, uint32_t k) {
  return grad_weight_plan(rows, groups, n, k).parts;
}

template <int kFmt, int kKF, int kPF, int kPerCu>
static hipError_t grad_weight(const MxGradArgs& p, uint32_t parts, hipStream_t stream) {
  const uint32_t k_tiles = (p.k + 64 * kKF - 1) / (64 * kKF), p_tiles = (p.n + 64 * kPF - 1) / (64 * kPF);
  const uint64_t tiles = ((uint64_t)k_tiles * p_tiles * p.groups + 7) / 8 * 8;
  if (tiles * 256 > 0xffffffffull) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)tiles, parts), block(256);
  if (p.row_index)
    hipLaunchKernelGGL((mx_grad_kernel<true, kFmt, true, false, kKF, kPF, kPerCu>), grid, block, 0, stream, p, k_tiles, p_tiles, parts);
  else
    hipLaunchKernelGGL((mx_grad_kernel<true, kFmt, false, false, kKF, kPF, kPerCu>), grid, block, 0, stream, p, k_tiles, p_tiles, parts);
  return hipGetLastError();
}

template <int kFmt>
static hipError_t grad_weight(const MxGradArgs& p, hipStream_t stream) {
  const GradWeightPlan plan = grad_weight_plan(p.rows, p.offsets ? p.groups : 0, p.n, p.k);
  const uint32_t parts = plan.parts;
  const hipError_t st = plan.big ? grad_weight<kFmt, 4, 2, 2>(p, parts, stream) : grad_weight<kFmt, 2, 1, 2>(p, parts, stream);
  if (st != hipSuccess || parts == 1) return st;
  const uint64_t nvec = (uint64_t)p.n * p.k / 8;
  const uint64_t g = (nvec + kThreads - 1) / kThreads;
  hipLaunchKernelGGL(mx_grad_join_kernel, dim3((unsigned)(g < kMaxGroups ? g : kMaxGroups)), dim3(kThreads), 0, stream,
                     p.partial, parts, nvec, p.mask, static_cast<uint4*>(p.grad));
  return hipGetLastError();
}

hipError_t launch_mx_grad_weight(MxFormat fmt, const MxGradArgs& args, hipStream_t stream) {
  MxGradArgs p = args;
  p.stream_out = past_cache(2 * (uint64_t)p.groups * p.n * p.k);
  return fmt == kE2M1 ? grad_weight<kE2M1>(p, stream) : grad_weight<kE4M3>(p, stream);
}

}  // namespace trace_host
