// Operands of the scaled matrix instructions and the row groups of the
// microscaled products (gfx950).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 and 32x32x64: lane l holds row l % R of
// an operand (R = 16 or 32) and, with group g = l / R, either 32 E2M1 codes
// of the block k = 32 g .. 32 g + 31 (16 bytes), or 32 E4M3 codes in two runs
// of 16: k = 16 g .. 16 g + 15 and K/2 + 16 g .. (K = 128 or 64).  Either way
// the lane's scale operand carries the E8M0 byte of block g of its row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"

namespace trace_dev {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

// Format selectors of the instruction.
constexpr int kSelE4M3 = 0;
constexpr int kSelE2M1 = 4;

// A 16-byte operand: the instruction reads four registers for E2M1.
__device__ __forceinline__ v8i widen(v4i v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }
__device__ __forceinline__ v8i widen(v8i v) { return v; }
__device__ __forceinline__ v8i join(v4i a, v4i b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// Results leave through LDS, 32 rows of kPieces 16-byte pieces at a time: a
// lane's registers hold pieces of one row, and stores straight from them would
// write 32 bytes of each of 32 rows at once; memory takes whole lines more
// than twice as fast.  Each wave has 512 kPieces bytes of its own.  The pieces
// of a row are permuted by the row's bits, for the LDS banks.
template <int kPieces>
struct RowBlock {
  static_assert(kPieces == 8 || kPieces == 16, "rows of 128 or 256 bytes");
  char* lds;
  __device__ __forceinline__ char* at(uint32_t row, uint32_t piece) const {
    return lds + row * (16 * kPieces) + 16 * ((piece ^ (kPieces == 16 ? row : row >> 1)) & (kPieces - 1));
  }
  __device__ __forceinline__ void put(uint32_t row, uint32_t piece, uint4 v) const {
    *reinterpret_cast<uint4*>(at(row, piece)) = v;
  }
  // store(row, piece, v) for every piece of the block, a row's pieces on
  // consecutive lanes.
  template <typename Store>
  __device__ __forceinline__ void drain(Store store) const {
    const uint32_t lane = threadIdx.x & 63;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (uint32_t i = 0; i < kPieces / 2; ++i) {
      const uint32_t row = (lane + 64 * i) / kPieces, piece = lane % kPieces;
      store(row, piece, *reinterpret_cast<const uint4*>(at(row, piece)));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
};

// Eight consecutive results of a row in fp32: pieces `piece` and the next.
__device__ __forceinline__ void put_f32(const RowBlock<16>& block, uint32_t row, uint32_t piece, const float (&v)[8]) {
  uint4 u[2];
  __builtin_memcpy(u, v, sizeof(u));
  block.put(row, piece, u[0]);
  block.put(row, piece + 1, u[1]);
}

// 16 bytes of a result.  One larger than the last-level cache (past_cache)
// goes past it, since its reader will not find it there: the weights' gradient
// of 128 x 1536 x 2048, 805 MB, takes 521 us against 607, the product's 537 MB
// of 131072 x 2048 x 768 211 against 259.
__device__ __forceinline__ void store_result(void* at, uint4 v, bool stream) {
  if (stream)
    store_vec<true>(reinterpret_cast<uint4*>(at), v);
  else
    *reinterpret_cast<uint4*>(at) = v;
}

// A row tile of one group: rows [first, first + count), count <= the tile's
// height; group == groups stands for the rows behind the last group.
struct RowTile {
  uint32_t group;
  uint32_t count;
  uint64_t first;
};

// offsets[i] within [0, rows].
__device__ __forceinline__ uint64_t clamped_offset(const int64_t* __restrict__ offsets, uint32_t i, uint64_t rows) {
  const int64_t v = offsets[i];
  return v <= 0 ? 0 : ((uint64_t)v > rows ? rows : (uint64_t)v);
}

// Rows of group g: offsets that decrease give an empty group, and the rows
// behind offsets[groups] form one more.
__device__ __forceinline__ uint32_t group_rows(const int64_t* __restrict__ offsets, uint32_t g, uint32_t groups,
                                               uint64_t rows, uint64_t& first) {
  first = clamped_offset(offsets, g, rows);
  const uint64_t end = g < groups ? clamped_offset(offsets, g + 1, rows) : rows;
  return end > first ? (uint32_t)(end - first) : 0u;
}

// Inclusive prefix of v over the wave's 64 lanes by DPP moves (a shuffle
// through LDS takes ten times as long, and every tile waits for this),
// saturating: offsets that overlap could pass 32 bits.
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t add_moved(uint32_t v) {
  return __builtin_elementwise_add_sat(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, kRows, 0xf, false));
}
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v) {
  v = add_moved<0x111, 0xf>(v);  // one lane up within 16, then 2, 4 and 8
  v = add_moved<0x112, 0xf>(v);
  v = add_moved<0x114, 0xf>(v);
  v = add_moved<0x118, 0xf>(v);
  v = add_moved<0x142, 0xa>(v);     // lane 15 to the second 16, lane 47 to the fourth
  return add_moved<0x143, 0xc>(v);  // lane 31 to the upper half
}

// Finds row tile `tile` (tiles of `height` rows, group by group; the rows
// behind the last group come last).  Every lane of the wave must call it
// with the same arguments: the wave adds up 64 groups' tiles at a time.
// Returns false past the last tile.
__device__ __forceinline__ bool find_row_tile(const int64_t* __restrict__ offsets, uint32_t groups, uint64_t rows,
                                              uint32_t height, uint64_t tile, RowTile& out) {
  const uint32_t lane = threadIdx.x & 63;
  uint64_t before = 0;
  for (uint32_t g0 = 0; g0 <= groups; g0 += 64) {
    const uint32_t g = g0 + lane;
    uint64_t first = 0;
    const uint32_t count = g <= groups ? group_rows(offsets, g, groups, rows, first) : 0u;
    const uint32_t tiles = (count + height - 1) / height;
    const uint32_t sum = wave_prefix(tiles);
    const uint32_t all = (uint32_t)__builtin_amdgcn_readlane((int)sum, 63);
    if (tile < before + all) {
      const uint64_t hit = __ballot(tile < before + sum);
      const int at = __ffsll((long long)hit) - 1;  // the first group whose tiles reach past `tile`
      const uint32_t cnt = (uint32_t)__builtin_amdgcn_readlane((int)count, at);
      const uint32_t start = at ? (uint32_t)__builtin_amdgcn_readlane((int)sum, at - 1) : 0u;
      const uint32_t flo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)first, at);
      const uint32_t fhi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(first >> 32), at);
      const uint32_t in = (uint32_t)(tile - (before + start)) * height;
      out.group = g0 + (uint32_t)at;
      out.first = (((uint64_t)fhi << 32) | flo) + in;
      out.count = cnt - in < height ? cnt - in : height;
      return true;
    }
    before += all;
  }
  return false;
}

// Row tiles of all groups and of the rows behind them; called like
// find_row_tile.
__device__ __forceinline__ uint64_t count_row_tiles(const int64_t* __restrict__ offsets, uint32_t groups, uint64_t rows,
                                                    uint32_t height) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t sum = 0;
  for (uint32_t g = lane; g <= groups; g += 64) {
    uint64_t first;
    sum = __builtin_elementwise_add_sat(sum, (group_rows(offsets, g, groups, rows, first) + height - 1) / height);
  }
  return (uint32_t)__builtin_amdgcn_readlane((int)wave_prefix(sum), 63);
}

// Workgroups go to the 8 XCDs (each with an L2 of its own) in turn.  The
// tiles are dealt out so that each XCD works through one run of consecutive
// tiles, which share operands: the tile of this workgroup, or `tiles` where
// it has none.
__device__ __forceinline__ uint64_t xcd_tile(uint64_t block, uint64_t tiles) {
  const uint64_t run = (tiles + 7) / 8;
  const uint64_t at = block / 8, tile = (block % 8) * run + at;
  return at < run && tile < tiles ? tile : tiles;
}

// Most row tiles that `rows` rows in `groups` groups (and the rows behind
// them) can make: every group but one ends in a partial tile.
inline uint64_t max_row_tiles(uint64_t rows, uint32_t groups, uint32_t height) {
  const uint64_t parts = (uint64_t)groups + 1;
  const uint64_t most = rows / height + parts;
  return most < rows ? most : rows;
}

}  // namespace trace_dev
