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

// ---------------------------------------------------------------------------
// Many rows.  A workgroup of four waves owns a 256 x 256 tile of y, each wave
// 128 n x 128 m of it as 4 x 4 blocks of the 32x32x64 instruction (256
// accumulator registers, one wave per SIMD).
//
// The operands pass through LDS in stages of 128 k, two buffers, one barrier
// per stage.  Loads run up to three stages ahead of the arithmetic, in
// registers until their buffer is free.  (Copying to LDS without registers
// was slower: the compiler waits for every copy under way before each LDS
// read.)  Lane i's 16 bytes lie at place i of a 1 KiB chunk, so the lanes
// choose which 16 bytes they fetch: the pieces of a row are permuted by the
// row's bits, so that the eight rows that the reads of eight lanes touch lie
// in different banks.
//
// Scale bytes go through registers, 16 blocks (512 k) of a row at a time,
// into a double buffer of dwords [stage][row]; the instruction picks its byte.
//
// W's rows 4..7 and 8..11 of every 16 trade places on the way to the
// instruction: a lane's eight consecutive result registers are then eight
// consecutive n, stored as 16 bytes.
// ---------------------------------------------------------------------------

// This wave's LDS accesses are done; meet the workgroup's other waves.  Loads
// to registers stay under way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Scale bytes of blocks b .. b + 15 of a row (0x7f past its last block).
__device__ __forceinline__ v4i scale_span(const uint8_t* __restrict__ row, uint32_t b, uint32_t blocks) {
  v4i s = {0x7f7f7f7f, 0x7f7f7f7f, 0x7f7f7f7f, 0x7f7f7f7f};
  if (b + 16 <= blocks) {
    __builtin_memcpy(&s, row + b, 16);
  } else {
#pragma unroll
    for (uint32_t d = 0; d < 4; ++d) {
      const uint32_t at = b + 4 * d;
      int v = 0x7f7f7f7f;
      if (at + 4 <= blocks) {
        __builtin_memcpy(&v, row + at, 4);
      } else if (at < blocks) {
#pragma unroll
        for (uint32_t j = 0; j < 3; ++j)
          if (at + j < blocks) v = (v & ~(0xff << (8 * j))) | ((int)row[at + j] << (8 * j));
      }
      s[d] = v;
    }
  }
  return s;
}

// 32 codes of an activation row.
template <int kFmt>
struct Operand {
  using type = v4i;
};
template <>
struct Operand<trace_host::kE4M3> {
  using type = v8i;
};

// A number as a type, for lambdas that need it at compile time.
template <uint32_t kValue>
struct Constant {
  static constexpr uint32_t value = kValue;
};

template <int kFmt, bool kGather>
__global__ __launch_bounds__(256, 1) void mx_tile_kernel(trace_host::MxProductArgs p, uint32_t col_tiles) {
  constexpr bool kFp4 = kFmt == trace_host::kE2M1;
  constexpr uint32_t kTile = 256;
  constexpr uint32_t kABytes = kFp4 ? 64 : 128;                // per row and stage
  constexpr uint32_t kStageBytes = kTile * (64 + kABytes);
  constexpr uint32_t kALoads = kABytes / 16, kLoads = 4 + kALoads;  // 16-byte loads per lane and stage
  constexpr uint32_t kAhead = kFp4 ? 2 : 1;                    // stages in registers
  __shared__ __attribute__((aligned(1024))) char ring[2 * kStageBytes];
  __shared__ int scale_buf[2][4][2 * kTile];  // [span][stage of the span][W's rows, A's rows]

  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t row_tiles = p.offsets ? count_row_tiles(p.offsets, p.groups, p.rows, kTile)
                                       : (p.rows + kTile - 1) / kTile;
  const uint64_t tiles = row_tiles * col_tiles;
  const uint64_t tile = xcd_tile(blockIdx.x, tiles);
  if (tile >= tiles) return;
  const uint64_t row_tile = tile / col_tiles;
  const uint32_t n0 = (uint32_t)(tile - row_tile * col_tiles) * kTile;
  RowTile t;
  if (p.offsets) {
    if (!find_row_tile(p.offsets, p.groups, p.rows, kTile, row_tile, t)) return;
  } else {
    t.group = 0;
    t.first = row_tile * kTile;
    t.count = (uint32_t)(p.rows - t.first < kTile ? p.rows - t.first : kTile);
  }
  const bool behind = t.group >= p.groups;  // rows of no group: zeros
  const uint32_t blocks = p.k / 32;
  const uint32_t w_pitch = p.k / 2, a_pitch = kFp4 ? p.k / 2 : p.k;
  const uint32_t stages = behind ? 0 : (p.k + 127) / 128;

  // what this lane fetches: W's rows 64 wave + 16 j + lane / 4, and A's rows
  // 64 wave + 16 j + lane / 4 (4 pieces a row) or + 8 j + lane / 8 (8 pieces)
  const uint32_t w_piece = (lane & 3) ^ (((lane >> 3) & 1) | ((lane >> 4) & 2));
  const uint32_t a_piece = kFp4 ? (lane & 3) ^ ((lane >> 3) & 3) : (lane & 7) ^ (lane >> 3);
  const uint64_t weight = behind ? 0 : t.group;
  const uint8_t* wc = p.w_codes + (weight * p.n + n0) * w_pitch;
  uint32_t w_from[4];
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j) {
    const uint32_t n = 64 * wave + 16 * j + lane / 4;
    w_from[j] = (n0 + n < p.n ? n : 0) * w_pitch;  // past the last column: any row, dropped at the end
  }
  // source rows of packed rows m of the tile; rows past the tile's and rows
  // without a source read row 0 and are dropped or cleared at the end
  const auto packed_row = [&](uint32_t m) -> uint64_t { return t.first + (m < t.count ? m : 0); };
  const auto has_source = [&](int64_t i) -> bool { return !kGather || (i >= 0 && i < (int64_t)p.src_rows); };
  int64_t a_index[kALoads], r_index[4], s_index;
  const uint32_t h = lane >> 5, r = lane & 31;
  const uint32_t wn = 128 * (wave >> 1), wm = 128 * (wave & 1);
#pragma unroll
  for (uint32_t j = 0; j < kALoads; ++j) {
    const uint64_t row = packed_row(kFp4 ? 64 * wave + 16 * j + lane / 4 : 64 * wave + 8 * j + lane / 8);
    a_index[j] = kGather ? p.row_index[row] : (int64_t)row;
  }
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j) r_index[j] = kGather ? p.row_index[packed_row(wm + r + 32 * j)] : 0;
  s_index = kGather ? p.row_index[packed_row(threadIdx.x)] : (int64_t)packed_row(threadIdx.x);
  const uint8_t* a_from[kALoads];
#pragma unroll
  for (uint32_t j = 0; j < kALoads; ++j)
    a_from[j] = p.a_codes + (has_source(a_index[j]) ? (uint64_t)a_index[j] : 0) * a_pitch;
  uint32_t sources = 0;  // which of this lane's four result rows have a source row
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j) sources |= (has_source(r_index[j]) ? 1u : 0u) << j;
  v4i held[kAhead][kLoads];  // stages on their way to LDS
  // may_end: the stage may hold fewer than 128 k; pieces past the end are zeros
  const auto fetch = [&](uint32_t st, v4i(&to)[kLoads], bool may_end) {
    const uint32_t left = p.k - 128 * st;
    const bool w_in = !may_end || 32 * w_piece < left;
    const bool a_in = !may_end || (kFp4 ? 32 : 16) * a_piece < left;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
      v4i v = {0, 0, 0, 0};
      if (w_in) v = *reinterpret_cast<const v4i*>(wc + 64 * st + (w_from[j] + 16 * w_piece));
      to[j] = v;
    }
#pragma unroll
    for (uint32_t j = 0; j < kALoads; ++j) {
      v4i v = {0, 0, 0, 0};
      if (a_in) v = *reinterpret_cast<const v4i*>(a_from[j] + kABytes * st + 16 * a_piece);
      to[4 + j] = v;
    }
  };
  const auto place = [&](uint32_t st, const v4i(&from)[kLoads]) {
    char* to = ring + (st & 1) * kStageBytes + 16 * lane;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) *reinterpret_cast<v4i*>(to + 1024 * (4 * wave + j)) = from[j];
#pragma unroll
    for (uint32_t j = 0; j < kALoads; ++j)
      *reinterpret_cast<v4i*>(to + 64 * kTile + 1024 * (kALoads * wave + j)) = from[4 + j];
  };
  // scale rows: thread i carries W's row i and A's row i
  const uint8_t* ws_row = p.w_scales + (weight * p.n + n0 + (n0 + threadIdx.x < p.n ? threadIdx.x : 0)) * blocks;
  const uint8_t* as_row = p.a_scales + (has_source(s_index) ? (uint64_t)s_index : 0) * blocks;
  v4i w_span, a_span;
  const auto load_span = [&](uint32_t span) {
    w_span = scale_span(ws_row, 16 * span, blocks);
    a_span = scale_span(as_row, 16 * span, blocks);
  };
  const auto store_span = [&](uint32_t span) {
#pragma unroll
    for (uint32_t d = 0; d < 4; ++d) {
      scale_buf[span & 1][d][threadIdx.x] = w_span[d];
      scale_buf[span & 1][d][kTile + threadIdx.x] = a_span[d];
    }
  };

  v16f acc[4][4] = {};  // [W fragment][A fragment]
  const uint32_t w_row = wn + ((r & 0x13) | ((r & 4) << 1) | ((r & 8) >> 1));  // bits 2 and 3 trade places
  const uint32_t w_at = w_row * 64 + 16 * (h ^ (((w_row >> 1) & 1) | ((w_row >> 2) & 2)));
  const uint32_t a_row_in = wm + r;
  const uint32_t a_at = 64 * kTile + (kFp4 ? a_row_in * 64 + 16 * (h ^ ((r >> 1) & 3)) : a_row_in * 128 + 16 * (h ^ (r & 7)));

  using AFrag = typename Operand<kFmt>::type;
  v4i wf[2][4];
  AFrag af[2][4];
  uint32_t wsc[2][4], asc[2][4];  // of this stage and the next
  // Fragments of k-step kk (64 k) of a stage.
  const auto read_step = [&](uint32_t st, uint32_t kk, v4i(&w)[4], AFrag(&a)[4]) {
    const char* from = ring + (st & 1) * kStageBytes;
#pragma unroll
    for (uint32_t f = 0; f < 4; ++f) w[f] = *reinterpret_cast<const v4i*>(from + ((w_at ^ (32 * kk)) + 2048 * f));
#pragma unroll
    for (uint32_t f = 0; f < 4; ++f) {
      if constexpr (kFp4) {
        a[f] = *reinterpret_cast<const v4i*>(from + ((a_at ^ (32 * kk)) + 2048 * f));
      } else {
        a[f] = join(*reinterpret_cast<const v4i*>(from + ((a_at ^ (64 * kk)) + 4096 * f)),
                    *reinterpret_cast<const v4i*>(from + ((a_at ^ (64 * kk) ^ 32) + 4096 * f)));
      }
    }
  };
  const auto read_scales = [&](uint32_t st, uint32_t(&w)[4], uint32_t(&a)[4]) {
    const int* from = scale_buf[(st >> 2) & 1][st & 3];
#pragma unroll
    for (uint32_t f = 0; f < 4; ++f) {
      w[f] = (uint32_t)from[w_row + 32 * f];
      a[f] = (uint32_t)from[kTile + a_row_in + 32 * f];
    }
  };
  const auto multiply = [&](const v4i(&w)[4], const AFrag(&a)[4], const uint32_t(&ws)[4], const uint32_t(&as)[4], auto sel) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(w[i]), widen(a[j]), acc[i][j], kSelE2M1,
                                                                    kFp4 ? kSelE2M1 : kSelE4M3, decltype(sel)::value,
                                                                    (int)ws[i], decltype(sel)::value, (int)as[j]);
  };
  // One stage, whose first step and scales have been read.  Under the first
  // step's arithmetic the second step is read, the next stage is placed in
  // LDS and the one kAhead + 1 further is fetched; under the second step's the
  // next stage's first step is read.  kSteady: those stages exist, in full.
  const auto stage = [&](uint32_t st, auto part, auto steady) {
    constexpr uint32_t kPart = decltype(part)::value;  // st % 4
    constexpr bool kSteady = decltype(steady)::value;
    constexpr uint32_t kNow = kPart & 1, kNext = kNow ^ 1, kHeld = (kPart + 1) % kAhead;
#pragma unroll
    for (int f = 0; f < 4; ++f) {  // byte 0: this lane's block of step 0; byte 2: of step 1
      wsc[kNow][f] >>= 8 * h;
      asc[kNow][f] >>= 8 * h;
    }
    read_step(st, 1, wf[1], af[1]);
    if (kPart == 2 && (kSteady || st + 2 < stages)) store_span((st >> 2) + 1);
    if (kSteady || st + 1 < stages) place(st + 1, held[kHeld]);
    if (kPart == 0 && (kSteady || st + 4 < stages)) load_span((st >> 2) + 1);
    if (kSteady || st + 1 + kAhead < stages) fetch(st + 1 + kAhead, held[kHeld], !kSteady);
    multiply(wf[0], af[0], wsc[kNow], asc[kNow], Constant<0>());
    if (kSteady) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);                // matrix instructions
        __builtin_amdgcn_sched_group_barrier(0x100, kFp4 ? 1 : 2, 0);     // LDS reads
        __builtin_amdgcn_sched_group_barrier(0x200, kFp4 ? 1 : 2, 0);     // LDS writes
        __builtin_amdgcn_sched_group_barrier(0x020, kFp4 ? 1 : 2, 0);     // loads
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (kSteady || st + 1 < stages) {
      lds_barrier();
      read_step(st + 1, 0, wf[0], af[0]);
      read_scales(st + 1, wsc[kNext], asc[kNext]);
    }
    multiply(wf[1], af[1], wsc[kNow], asc[kNow], Constant<2>());
    if (kSteady) {
#pragma unroll
      for (int i = 0; i < 12; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, kFp4 ? 1 : 2, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  if (stages) {
    load_span(0);
    v4i first[kLoads];
    fetch(0, first, true);
#pragma unroll
    for (uint32_t i = 0; i < kAhead; ++i)
      if (1 + i < stages) fetch(1 + i, held[(1 + i) % kAhead], true);
    store_span(0);
    place(0, first);
    lds_barrier();
    read_step(0, 0, wf[0], af[0]);
    read_scales(0, wsc[0], asc[0]);
    uint32_t st = 0;
    for (; st + 5 + kAhead < stages; st += 4) {
      stage(st, Constant<0>(), Constant<1>());
      stage(st + 1, Constant<1>(), Constant<1>());
      stage(st + 2, Constant<2>(), Constant<1>());
      stage(st + 3, Constant<3>(), Constant<1>());
    }
    for (; st < stages; st += 4) {
      stage(st, Constant<0>(), Constant<0>());
      if (st + 1 < stages) stage(st + 1, Constant<1>(), Constant<0>());
      if (st + 2 < stages) stage(st + 2, Constant<2>(), Constant<0>());
      if (st + 3 < stages) stage(st + 3, Constant<3>(), Constant<0>());
    }
  }
  // register e of a block: n = 16 (e / 8) + 8 h + e % 8, m = lane % 32
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t m = wm + 32 * j + r;
    if (m >= t.count) continue;
    const bool ok = (sources >> j) & 1;
    uint16_t* row = p.y + (t.first + m) * p.n;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 16; e += 8) {
        const uint32_t n = n0 + wn + 32 * i + 2 * e + 8 * h;
        if (n >= p.n) continue;
        const v16f& a = acc[i][j];
        uint4 v = make_uint4(bf16_pair(a[e], a[e + 1]), bf16_pair(a[e + 2], a[e + 3]), bf16_pair(a[e + 4], a[e + 5]),
                             bf16_pair(a[e + 6], a[e + 7]));
        if (!ok) v = make_uint4(0, 0, 0, 0);  // no source row
        *reinterpret_cast<uint4*>(row + n) = v;
      }
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
static hipError_t launch_tile(const MxProductArgs& p, hipStream_t stream) {
  const uint32_t cols = (p.n + 255) / 256;
  const uint64_t row_tiles = p.offsets ? max_row_tiles(p.rows, p.groups, 256) : (p.rows + 255) / 256;
  const uint64_t grid = (row_tiles * cols + 7) / 8 * 8;
  if (grid * 256 > 0xffffffffull) return hipErrorInvalidConfiguration;
  if (p.row_index)
    hipLaunchKernelGGL((mx_tile_kernel<kFmt, true>), dim3((unsigned)grid), dim3(256), 0, stream, p, cols);
  else
    hipLaunchKernelGGL((mx_tile_kernel<kFmt, false>), dim3((unsigned)grid), dim3(256), 0, stream, p, cols);
  return hipGetLastError();
}

template <int kFmt>
static hipError_t launch_product(const MxProductArgs& p, hipStream_t stream) {
  if (p.rows >= 128 && p.src_rows > 0) return launch_tile<kFmt>(p, stream);
  return launch_skinny<kFmt, 2, 2, 4>(p, stream);
}

hipError_t launch_mx_product(MxFormat fmt, const MxProductArgs& p, hipStream_t stream) {
  return fmt == kE2M1 ? launch_product<kE2M1>(p, stream) : launch_product<kE4M3>(p, stream);
}

}  // namespace trace_host
