// Tiles of bf16 products with fp32 sums (gfx950), for the loss over the
// vocabulary and its gradients:  D[i, j] = sum over c of I(i, c) J(j, c).
//
// A workgroup of four waves, kWI x kWJ of them, owns 32 kWI kI results i times
// 32 kWJ kJ results j, each wave kI x kJ blocks of the 32x32x16 instruction.  A
// lane holds one j and, in consecutive registers, eight consecutive i at a time.
//
// Each operand lies in memory either along c (rows i or j of consecutive c) or
// across it (rows c of consecutive i or j).  Stages of 64 c are copied straight
// to LDS, 1 KiB (64 lanes' 16 bytes) per instruction, kRing stages in turn, one
// barrier per stage; the copies run kRing - 1 stages ahead of the arithmetic.
// Place i of a copy's KiB belongs to lane i, so the lanes choose which 16 bytes
// they fetch: pieces are permuted by their row's bits, so that the rows that are
// read together lie in different banks.  Operands across c are read back
// transposed (ds_read_b64_tr_b16: 16 lanes read four rows of 16 values, lane i
// gets column i).
//
// The copies are written as assembly: the compiler would wait for all of them
// before each read of LDS.  They have no result registers; the barrier below waits
// for them.  Nothing else in these kernels uses M0.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"
#include "fp4_block.h"
#include "mx_mfma.h"

namespace trace_dev {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr uint32_t kStageC = 64;  // c of a stage

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// Copies 16 bytes per lane to lds + 16 * lane.
__device__ __forceinline__ void copy_to_lds(const void* from, uint32_t lds) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(lds));
#endif
}

// All but the last kLeft copies of this wave have arrived and its LDS reads are
// done; meet the workgroup's other waves.
template <uint32_t kLeft>
__device__ __forceinline__ void stage_barrier() {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLeft) : "memory");
#endif
}

// An operand of a tile: kRows rows i (or j) of a stage.  Both ways a stage has
// 128 kRows bytes.
template <uint32_t kRows, bool kAcross>
struct TileOperand {
  static_assert(!kAcross || kRows == 128 || kRows == 256, "rows of 256 or 512 bytes");
  static constexpr uint32_t kBytes = 128 * kRows;
  static constexpr uint32_t kCopies = kBytes / 4096;  // per wave
  static constexpr uint32_t kPitch = kAcross ? 2 * kRows : 128;

  // What this lane fetches with copy n of its wave: the row of the operand in
  // memory and its first of eight columns.
  static __device__ __forceinline__ void place(uint32_t wave, uint32_t n, uint32_t& row, uint32_t& col) {
    const uint32_t at = 1024 * (wave * kCopies + n) + 16 * (threadIdx.x & 63);
    row = at / kPitch;
    const uint32_t piece = at % kPitch / 16;
    col = 8 * (kAcross ? piece ^ ((row & 3) << 2) : piece ^ ((row >> 1) & 7));
  }

  // Operand registers of k-step kk, rows first + 32 f + (lane % 32).  kSwap:
  // rows 4..7 and 8..11 of every 16 trade places (a lane's eight consecutive
  // results are then eight consecutive i).
  template <bool kSwap>
  static __device__ __forceinline__ v8bf read(const char* stage, uint32_t first, uint32_t f, uint32_t kk) {
    const uint32_t lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
    if constexpr (kAcross) {
      const uint32_t j = lane & 15, half = (lane >> 4) & 1;
      const uint32_t quad = kSwap ? ((j & 1) << 1) | ((j >> 1) & 1) : j & 3;
      const uint32_t row = 8 * h + (j >> 2);  // and four rows on, whose low bits are the same
      const uint32_t piece = first / 8 + 4 * f + 2 * half + (quad >> 1);
      const char* at = stage + (16 * kk + row) * kPitch + 16 * (piece ^ ((row & 3) << 2)) + 8 * (quad & 1);
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)at);
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + 4 * kPitch));
      v8bf out;
      __builtin_memcpy(&out, &lo, 8);
      __builtin_memcpy(reinterpret_cast<char*>(&out) + 8, &hi, 8);
      return out;
    } else {
      const uint32_t row = first + 32 * f + (kSwap ? (r & 0x13) | ((r & 4) << 1) | ((r & 8) >> 1) : r);
      return *reinterpret_cast<const v8bf*>(stage + row * kPitch + 16 * ((2 * kk + h) ^ ((row >> 1) & 7)));
    }
  }
};

template <int kI_, int kJ_, int kWI_, int kWJ_, bool kAcrossI, bool kAcrossJ, int kRing_>
struct Tile {
  static constexpr int kI = kI_, kJ = kJ_, kWI = kWI_, kWJ = kWJ_;
  static constexpr uint32_t kRing = kRing_;
  static constexpr uint32_t kRowsI = 32 * kI * kWI, kRowsJ = 32 * kJ * kWJ;
  using I = TileOperand<kRowsI, kAcrossI>;
  using J = TileOperand<kRowsJ, kAcrossJ>;
  static constexpr uint32_t kStageBytes = I::kBytes + J::kBytes;
  static constexpr uint32_t kLds = kRing * kStageBytes;
  static constexpr uint32_t kCopies = I::kCopies + J::kCopies;
  static_assert(kWI * kWJ == 4, "four waves");
  static_assert(kCopies * (kRing - 2) < 64, "copies that the wait can count");

  // This wave's first row of the tile's I and J.
  static __device__ __forceinline__ uint32_t wave_i() {
    return 32 * kI * (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / kWJ);
  }
  static __device__ __forceinline__ uint32_t wave_j() {
    return 32 * kJ * (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % kWJ);
  }

  // from_i(n, stage), from_j(n, stage): where this lane's 16 bytes of copy n of a
  // stage lie.  Leaves every wave past its last read of the ring.
  template <class FromI, class FromJ>
  static __device__ __forceinline__ void multiply(char* ring, uint32_t stages, FromI from_i, FromJ from_j,
                                                  v16f (&acc)[kI][kJ]) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t base = __builtin_amdgcn_readfirstlane(lds_address(ring));
    const auto fetch = [&](uint32_t st, uint32_t slot) {
      const uint32_t to = base + slot * kStageBytes;
#pragma unroll
      for (uint32_t n = 0; n < I::kCopies; ++n) copy_to_lds(from_i(n, st), to + 1024 * (wave * I::kCopies + n));
#pragma unroll
      for (uint32_t n = 0; n < J::kCopies; ++n)
        copy_to_lds(from_j(n, st), to + I::kBytes + 1024 * (wave * J::kCopies + n));
    };
    const uint32_t wi = wave_i(), wj = wave_j();
    v8bf fi[2][kI], fj[2][kJ];
    const auto read = [&](uint32_t slot, uint32_t kk, v8bf(&a)[kI], v8bf(&b)[kJ]) {
      const char* from = ring + slot * kStageBytes;
#pragma unroll
      for (uint32_t f = 0; f < kI; ++f) a[f] = I::template read<true>(from, wi, f, kk);
#pragma unroll
      for (uint32_t f = 0; f < kJ; ++f) b[f] = J::template read<false>(from + I::kBytes, wj, f, kk);
    };
    const auto multiply_step = [&](const v8bf(&a)[kI], const v8bf(&b)[kJ]) {
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    };
    if (stages == 0) return;
#pragma unroll
    for (uint32_t s = 0; s < kRing - 1; ++s)
      if (s < stages) fetch(s, s);
    stage_barrier<0>();
    read(0, 0, fi[0], fj[0]);
    uint32_t slot = 0;
    for (uint32_t st = 0; st < stages; ++st) {
      const uint32_t ahead = slot == 0 ? kRing - 1 : slot - 1;  // the slot of stage st - 1, free since the last barrier
      const bool more = st + kRing - 1 < stages;
      if (more) fetch(st + kRing - 1, ahead);
#pragma unroll
      for (uint32_t kk = 0; kk < 3; ++kk) {
        read(slot, kk + 1, fi[(kk + 1) & 1], fj[(kk + 1) & 1]);
        multiply_step(fi[kk & 1], fj[kk & 1]);
      }
      slot = slot + 1 == kRing ? 0 : slot + 1;
      if (more)
        stage_barrier<kCopies * (kRing - 2)>();
      else
        stage_barrier<0>();
      if (st + 1 < stages) read(slot, 0, fi[0], fj[0]);
      multiply_step(fi[1], fj[1]);
    }
  }
};

}  // namespace trace_dev
