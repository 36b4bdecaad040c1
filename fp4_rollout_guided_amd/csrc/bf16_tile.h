// Tiles of bf16 products with fp32 sums (gfx950), for the loss over the
// vocabulary and its gradients:  D[i, j] = sum over c of I(i, c) J(j, c).
//
// A workgroup of four waves, kWI x kWJ of them, owns 16 kWI kI results i times
// 16 kWJ kJ results j, each wave kI x kJ blocks of the 16x16x32 instruction.  A
// lane holds one j and four consecutive i, or (I along c, below) in the registers
// of two neighbouring blocks eight.
//
// Each operand lies in memory either along c (rows i or j of consecutive c) or
// across it (rows c of consecutive i or j).  Stages of 64 c are copied straight
// to LDS, 1 KiB (64 lanes' 16 bytes) per instruction, a few stages in turn, one
// barrier per stage.  Place i of a copy's KiB belongs to lane i, so the lanes
// choose which 16 bytes they fetch: pieces are permuted by their row's bits, so
// that the rows that are read together lie in different banks.  Operands across c
// are read back transposed (ds_read_b64_tr_b16: 16 lanes read four rows of 16
// values, lane i gets column i).
//
// What bounds the largest tile (256 x 256) is power: at full use of the matrix
// units the clock falls from 2.4 to some 1.8 GHz.  The 16x16x32 instruction does
// 1.67 PFLOP/s alone where 32x32x16 does 1.51 (it moves fewer bytes of sums for a
// product), and 1.40 against 1.30 with the reads of LDS under it.
//
// The copies are written as assembly: the compiler would wait for all of them
// before each read of LDS.  They have no result registers; the barrier below waits
// for them.  Nothing else in these kernels uses M0.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_math.h"
#include "fp4_block.h"
#include "mx_mfma.h"

namespace trace_dev {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr uint32_t kStageC = 64;  // c of a stage

// This lane's number in its wave, by a value that is not known before this point:
// or what a tile's end computes from it would fill registers throughout its loop.
__device__ __forceinline__ uint32_t late_lane() {
  uint32_t lane = threadIdx.x & 63;
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("" : "+v"(lane));
#endif
  return lane;
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// Where the next copies go in LDS: lds + 16 * lane, and kAt bytes on below.
__device__ __forceinline__ void copies_to(uint32_t lds) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0" ::"s"(lds));
#endif
}
// Copies 16 bytes per lane from base + off + kAt, in the lanes that `lanes` has:
// all of them or none (all are active here).  kStream: past the caches, for what
// is read once.
template <uint32_t kAt, bool kStream>
__device__ __forceinline__ void copy_to_lds(const char* base, uint32_t off, uint64_t lanes) {
  static_assert(kAt < 4096, "the instruction's offset");
#ifdef __HIP_DEVICE_COMPILE__
  if constexpr (kStream)
    asm volatile("s_mov_b64 exec, %3\n\tglobal_load_lds_dwordx4 %0, %1 offset:%2 nt\n\ts_mov_b64 exec, -1" ::"v"(off),
                 "s"(base), "n"(kAt), "s"(lanes));
  else
    asm volatile("s_mov_b64 exec, %3\n\tglobal_load_lds_dwordx4 %0, %1 offset:%2\n\ts_mov_b64 exec, -1" ::"v"(off),
                 "s"(base), "n"(kAt), "s"(lanes));
#endif
}

// A loop whose index is a constant.
template <uint32_t kFrom, uint32_t kTo, class F>
__device__ __forceinline__ void unrolled(const F& f) {
  if constexpr (kFrom < kTo) {
    f(std::integral_constant<uint32_t, kFrom>());
    unrolled<kFrom + 1, kTo>(f);
  }
}

// This wave's LDS reads are done (and, of its copies, all but the last kLeft);
// meet the workgroup's other waves.
__device__ __forceinline__ void reads_barrier() {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#endif
}
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

  // How a row's pieces are permuted.  Along c, 16 lanes read one piece of 16 rows
  // that differ in bits 0 to 3, or 0, 1, 3 and 4 (kPairs below), two rows to 256
  // bytes; across it, 32 lanes read 32 bytes of eight rows that differ in bits 0, 1
  // and 3.
  static __device__ __forceinline__ uint32_t swap(uint32_t row) {
    return kAcross ? (row & 3) << 2 | ((row >> 2) & 2) : ((row >> 1) & 1) | ((row >> 2) & 2) | (((row ^ (row >> 2)) & 4));
  }

  // What this lane fetches with copy n of its wave: the row of the operand in
  // memory and its first of eight columns.
  static __device__ __forceinline__ void place(uint32_t wave, uint32_t lane, uint32_t n, uint32_t& row, uint32_t& col) {
    const uint32_t at = 1024 * (wave * kCopies + n) + 16 * lane;
    row = at / kPitch;
    col = 8 * ((at % kPitch / 16) ^ swap(row));
  }

  // Operand registers of k-step kk (32 c): block f, 16 rows from first + 16 f,
  // this lane's (lane % 16).  kPairs: blocks 2 q and 2 q + 1 share 32 rows, the
  // first with those whose bit 2 is 0 (a lane's results in both are then eight
  // consecutive ones); across c that would read half of the banks.
  template <bool kPairs>
  static __device__ __forceinline__ v8bf read(const char* stage, uint32_t first, uint32_t f, uint32_t kk) {
    const uint32_t lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4;
    if constexpr (kAcross) {
      static_assert(!kPairs);
      const uint32_t row = 8 * g + (q >> 2), run = q & 3;  // and four rows on, which are permuted alike
      const uint32_t piece = first / 8 + 2 * f + (run >> 1);
      const char* at = stage + (32 * kk + row) * kPitch + 16 * (piece ^ swap(row)) + 8 * (run & 1);
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)at);
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + 4 * kPitch));
      v8bf out;
      __builtin_memcpy(&out, &lo, 8);
      __builtin_memcpy(reinterpret_cast<char*>(&out) + 8, &hi, 8);
      return out;
    } else {
      const uint32_t row = first + (kPairs ? 32 * (f / 2) + 8 * (q >> 2) + 4 * (f & 1) + (q & 3) : 16 * f + q);
      return *reinterpret_cast<const v8bf*>(stage + row * kPitch + 16 * ((4 * kk + g) ^ swap(row)));
    }
  }
};

template <int kI_, int kJ_, int kWI_, int kWJ_, bool kAcrossI, bool kAcrossJ, int kRing_, bool kStreamI = false>
struct Tile {
  static constexpr int kI = kI_, kJ = kJ_, kWI = kWI_, kWJ = kWJ_;
  static constexpr uint32_t kRing = kRing_;  // stages in LDS
  static constexpr bool kStreams = kStreamI;
  static constexpr bool kPairs = !kAcrossI && kI % 2 == 0;

  // The wave's row i of element e of block b, in lane group g (lane / 16).
  static __device__ __forceinline__ uint32_t row_of(uint32_t b, uint32_t g, uint32_t e) {
    return kPairs ? 32 * (b / 2) + 8 * g + 4 * (b & 1) + e : 16 * b + 4 * g + e;
  }
  static constexpr uint32_t kRowsI = 16 * kI * kWI, kRowsJ = 16 * kJ * kWJ;
  using I = TileOperand<kRowsI, kAcrossI>;
  using J = TileOperand<kRowsJ, kAcrossJ>;
  static constexpr uint32_t kStageBytes = I::kBytes + J::kBytes, kLds = kRing * kStageBytes;
  static constexpr uint32_t kCopies = I::kCopies + J::kCopies;
  static_assert(kWI * kWJ == 4 && kRing >= 2, "four waves");
  static_assert(kCopies * (kRing - 1) < 64 && kLds <= 163840, "what the wait can count; LDS");

  // This wave's first row of the tile's I and J.
  static __device__ __forceinline__ uint32_t wave_i() {
    return 16 * kI * (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / kWJ);
  }
  static __device__ __forceinline__ uint32_t wave_j() {
    return 16 * kJ * (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % kWJ);
  }

  // Where an operand's copies come from: base + stage * step, the same for all
  // lanes, and each lane's place in a stage for each of its wave's copies.
  template <class Operand>
  struct Source {
    const char* base;
    uint64_t step;
    uint32_t off[Operand::kCopies];
  };

  // Sums of `stages` stages.  From stage `whole` on (the last one, or none) lanes
  // would pass an operand's end: before its copies shorten(from_i, from_j) moves
  // their places.  half: of the last stage only the first k-step counts.  first
  // (with kStreamI): the stage to begin with, then on to `whole` and round.  Leaves
  // every wave past its last read of the ring that matters.
  //
  // A stage is two k-steps; under the arithmetic of each the next one's operands
  // are read.  Half way through the first, when all waves have read the stage's
  // second half, its slot is free, and the copies of the stage kRing on go there:
  // they have more than kRing - 1 stages' time.  The order is the program's own
  // (sched_barrier): the compiler would gather the reads before their use,
  // where they are waited for.  There is one copy of the arithmetic, since branches
  // around products would move their sums between registers; past the last stage
  // the copies run with no lanes, and the reads find an old stage.
  template <class Shorten>
  static __device__ __forceinline__ void multiply(char* ring, uint32_t stages, uint32_t whole, bool half,
                                                  Source<I>& from_i, Source<J>& from_j, Shorten shorten,
                                                  v4f (&acc)[kI][kJ], uint32_t first = 0) {
    constexpr uint32_t kProducts = kI * kJ, kFragments = kI + kJ;
    constexpr uint32_t kHalf = (kProducts + 1) / 2, kReadsEach = (kFragments + kHalf - 1) / kHalf;
    // the product after which a slot is free, products to a copy and copies to a product after that
    constexpr uint32_t kRead = (kFragments + kReadsEach - 1) / kReadsEach - 1;  // the last product that reads follow
    constexpr uint32_t kFree = kRead > kProducts * 5 / 16 ? kRead : kProducts * 5 / 16, kLeft = kProducts - kFree;
    constexpr uint32_t kEvery = kLeft / kCopies < 1 ? 1 : (kLeft / kCopies > 2 ? 2 : kLeft / kCopies);
    constexpr uint32_t kAtOnce = kLeft / kCopies < 1 ? (kCopies + kLeft - 1) / kLeft : 1;
    if (stages == 0) return;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // this wave's part of slot 0 of either operand
    const uint32_t to_i = __builtin_amdgcn_readfirstlane(lds_address(ring)) + 1024 * I::kCopies * wave;
    const uint32_t to_j = __builtin_amdgcn_readfirstlane(lds_address(ring)) + I::kBytes + 1024 * J::kCopies * wave;
    // the instruction's offset moves the place in memory too
#pragma unroll
    for (uint32_t n = 0; n < I::kCopies; ++n) from_i.off[n] += 4096 - 1024 * (n % 4);
#pragma unroll
    for (uint32_t n = 0; n < J::kCopies; ++n) from_j.off[n] += 4096 - 1024 * (n % 4);
    const char* next_i = from_i.base - 4096 + (kStreamI ? first * from_i.step : 0);
    const char* next_j = from_j.base - 4096 + (kStreamI ? first * from_j.step : 0);
    uint32_t place = first;
    const auto advance = [&]() {
      next_i += from_i.step;
      next_j += from_j.step;
      if (kStreamI && ++place == whole) {
        next_i -= whole * from_i.step;
        next_j -= whole * from_j.step;
        place = 0;
      }
    };
    const auto to_last = [&]() {
      shorten(from_i, from_j);
      if (kStreamI) {
        next_i = from_i.base - 4096 + whole * from_i.step;
        next_j = from_j.base - 4096 + whole * from_j.step;
      }
    };
    uint64_t lanes = ~0ull;
    const auto copy = [&](auto n, uint32_t slot) {
      constexpr uint32_t kN = decltype(n)::value;
      if constexpr (kN < J::kCopies) {
        if constexpr (kN % 4 == 0) copies_to(to_j + slot * kStageBytes + 1024 * kN);
        copy_to_lds<1024 * (kN % 4), false>(next_j, from_j.off[kN], lanes);
      } else if constexpr (kN < kCopies) {
        constexpr uint32_t kM = kN - J::kCopies;
        if constexpr (kM % 4 == 0) copies_to(to_i + slot * kStageBytes + 1024 * kM);
        copy_to_lds<1024 * (kM % 4), kStreamI>(next_i, from_i.off[kM], lanes);
      }
    };
    const uint32_t wi = wave_i(), wj = wave_j();
    v8bf fi[2][kI], fj[2][kJ];
    // fragment f of a k-step, in the order of their first use
    const auto read = [&](auto f, uint32_t slot, uint32_t kk) {
      constexpr uint32_t kF = decltype(f)::value;
      const char* from = ring + slot * kStageBytes;
      if constexpr (kF == 0 || (kF > kJ && kF < kFragments))
        fi[kk][kF == 0 ? 0 : kF - kJ] = I::template read<kPairs>(from, wi, kF == 0 ? 0 : kF - kJ, kk);
      else if constexpr (kF <= kJ)
        fj[kk][kF - 1] = J::template read<false>(from + I::kBytes, wj, kF - 1, kk);
    };
    // k-step kk; under it `under` is called after each product
    const auto products = [&](uint32_t kk, const auto& under) {
      unrolled<0, kProducts>([&](auto m) {
        constexpr uint32_t kM = decltype(m)::value;
        acc[kM / kJ][kM % kJ] =
            __builtin_amdgcn_mfma_f32_16x16x32_bf16(fi[kk][kM / kJ], fj[kk][kM % kJ], acc[kM / kJ][kM % kJ], 0, 0, 0);
        under(m);
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    const auto read_under = [&](auto m, uint32_t slot, uint32_t kk) {
      constexpr uint32_t kM = decltype(m)::value;
      unrolled<kM * kReadsEach, (kM + 1) * kReadsEach>([&](auto f) { read(f, slot, kk); });
    };
#pragma unroll
    for (uint32_t s = 0; s < kRing; ++s) {
      if (s >= stages) continue;
      if (s == whole) to_last();
      unrolled<0, kCopies>([&](auto n) { copy(n, s); });
      advance();
    }
    stage_barrier<0>();
    unrolled<0, kFragments>([&](auto f) { read(f, 0, 0); });
    uint32_t slot = 0;
#pragma unroll 1
    for (uint32_t st = 0; st < stages; ++st) {
      if (st + kRing >= whole) {
        if (st + kRing >= stages)
          lanes = 0;
        else
          to_last();
      }
      products(0, [&](auto m) {
        constexpr uint32_t kM = decltype(m)::value;
        read_under(m, slot, 1);
        if constexpr (kM == kFree) reads_barrier();
        if constexpr (kM >= kFree && (kM - kFree) % kEvery == 0)
          unrolled<(kM - kFree) / kEvery * kAtOnce, (kM - kFree) / kEvery * kAtOnce + kAtOnce>(
              [&](auto n) { copy(n, slot); });
      });
      if (st + kRing < stages)
        stage_barrier<kCopies * (kRing - 1)>();
      else
        stage_barrier<0>();
      __builtin_amdgcn_sched_barrier(0);
      advance();
      slot = slot + 1 == kRing ? 0 : slot + 1;
      if (half && st + 1 == stages) {
#pragma unroll
        for (int f = 0; f < kI; ++f) fi[1][f] = v8bf{};
#pragma unroll
        for (int f = 0; f < kJ; ++f) fj[1][f] = v8bf{};
      }
      products(1, [&](auto m) { read_under(m, slot, 0); });
#ifdef __HIP_DEVICE_COMPILE__
      // sums that fill half of the registers stay in that half, whatever follows the loop
      if constexpr (kProducts == 64)
#pragma unroll
        for (int i = 0; i < kI; ++i)
#pragma unroll
          for (int j = 0; j < kJ; ++j) asm volatile("" : "+a"(acc[i][j]));
#endif
    }
  }
};

}  // namespace trace_dev
