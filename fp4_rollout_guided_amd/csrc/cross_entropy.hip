// libtrace softmax cross entropy over a large vocabulary for gfx950, and its
// gradients, without keeping the logits:
//
//   z[t, v] = scale * sum over k of x[t, k] w[v, k]
//   lse[t] = log(sum over v of exp(z[t, v])),  loss[t] = lse[t] - z[t, target[t]]
//   P[t, v] = scale * grad_loss[t] * (exp(z[t, v] - lse[t]) - (v == target[t]))
//   grad_x = P W,  grad_w = P^T X
//
// Forward: each tile of logits leaves the maximum and the sum of its columns for
// every token, and the target's logit where it has it; one more launch joins the
// tiles.  Backward: a slice of the vocabulary at a time, the logits are computed
// again and P is written in bf16 to the workspace; then the slice's part of
// grad_x is added to fp32 sums, and its rows of grad_w are finished.
//
// Tokens without a target (prompts, padding) are taken out before: the rows
// that remain are listed, and for the backward pass packed, so that ignored rows
// are neither read nor paid for.
//
// The matrix instructions want P in bf16.  Its largest entry in a row as a rule is
// the target's, p - 1: a rounding there is a factor on the token's whole part of the
// gradients.  So a row is written over |p - 1|, which leaves the target's entry near -1
// and all others below one, and the factor |p - 1| scale grad_loss goes onto the sums
// of grad_x in fp32, and for grad_w onto the token's row of x, whose elements
// are then rounded each by itself.  Against 64 bits (norm of the difference over the
// norm) grad_x is off by its own rounding to bf16, 0.0017, and grad_w by 1.4 times
// that, 0.0024; P rounded as it is makes 0.0024 of both.
//
// The divisor comes from a dot product of its own, summed in another order than the
// tile's logit: the target's entry is -1 up to the difference of the two, some
// 2^-24 of the logits' size over 1 - p.  For a token so confident that 1 - p falls to that size
// the entry can be anything, of either sign, and others may pass one; times the
// factor it is still the gradient as far as fp32 logits know it.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bf16_tile.h"
#include "device_math.h"
#include "fp4_block.h"
#include "launch.h"
#include "launch_step.h"

namespace trace_dev {

using trace_host::CrossEntropyArgs;

constexpr uint32_t kTileT = 256;  // tokens and vocabulary of the largest tile
constexpr uint32_t kPlanThreads = 1024;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// What the kernels of a call pass on in its workspace.
struct CrossEntropyPlan {
  uint32_t count;     // tokens with a target
  float grad_top;     // the largest finite |grad_loss| among them, or 1 where that is 0: a unit for rows of x
  uint32_t parts;     // of grad_x's contraction
  uint32_t pad[29];
};
static_assert(sizeof(CrossEntropyPlan) == 128, "a line of its own");

__host__ __device__ inline uint32_t tiles_of(uint32_t n, uint32_t each) { return (n + each - 1) / each; }

// The time of a stage of `tiles` tiles of 256 or (small) 128, in units of 0.05 us.  A
// compute unit holds one tile of 256 at a time (1.65 us), one of 128 (0.5) or two of
// them (0.9).  So tiles of 128 win where those of 256 leave many units idle, in their
// only or their last turn: grad_w of 1000 x 10007 x 1056, 5 us of 135.
__host__ __device__ inline uint64_t stage_time(uint64_t tiles, bool small) {
  if (!small) return (tiles + 255) / 256 * 33;
  const uint32_t rest = tiles % 512;
  return tiles / 512 * 18 + (rest == 0 ? 0 : (rest <= 256 ? 10 : 18));
}

// grad_x's contraction over a slice goes in parts, to fill the card, whose sums are
// written and read again.  Its time in `parts`, in units of 0.05 us: the stages, 3 us to
// start and end a turn, and 7 TB/s for `sums` elements of a part.  2000 tokens of k = 2048 go
// in 4 parts of one turn rather than in 16 of four: 840 -> 736 us with the rest of the
// gradients; 509 of k = 1056 in 7 of tiles of 128 rather than in 16 of 256: 94 -> 82.
__host__ __device__ inline uint64_t parts_time(uint64_t tiles, uint32_t parts, uint32_t stages, uint64_t sums, bool small) {
  const uint64_t turn = small ? 512 : 256;
  return stage_time(tiles * parts, small) * tiles_of(stages, parts) + (tiles * parts + turn - 1) / turn * 60 +
         parts * sums / 43750;
}
struct PartsRule {
  uint32_t most;    // parts, up to 64; 0: none are wanted
  uint32_t stages;  // of a slice
  uint32_t k;
  bool small;
};
// The best number of parts for `count` tokens, by one wave: a lane to a number.
__device__ __forceinline__ uint32_t best_parts(const PartsRule& rule, uint32_t count) {
  const uint32_t lane = threadIdx.x & 63, edge = rule.small ? 128 : 256;
  const uint64_t tiles = (uint64_t)tiles_of(count, edge) * tiles_of(rule.k, edge);
  uint64_t best = ~0ull;
  if (lane < rule.most)
    best = parts_time(tiles, lane + 1, rule.stages, (uint64_t)tiles_of(count, edge) * edge * rule.k, rule.small) << 6 | lane;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const uint64_t o = __shfl_xor(best, d);
    best = o < best ? o : best;
  }
  return (uint32_t)(best & 63) + 1;
}

// list[i]: the i-th token with a target; at[t]: the place of token t, or -1.
__global__ __launch_bounds__(kPlanThreads) void cross_entropy_plan_kernel(const int64_t* __restrict__ targets,
                                                                          const float* __restrict__ grad_loss,
                                                                          uint32_t tokens, uint32_t vocab,
                                                                          PartsRule rule, CrossEntropyPlan* plan,
                                                                          int32_t* list, int32_t* at) {
  constexpr uint32_t kWaves = kPlanThreads / 64, kEach = 8;
  __shared__ uint32_t part[kWaves];
  __shared__ uint32_t tops[kWaves];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t before = 0, top = 0;
  for (uint64_t t0 = 0; t0 < tokens; t0 += kPlanThreads * kEach) {
    // a wave's kEach * 64 tokens follow each other
    bool has[kEach];
    uint64_t mask[kEach];
    uint32_t mine = 0;
    int64_t v[kEach];
    uint32_t g[kEach];
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {  // all loads under way at once
      const uint64_t t = t0 + (wave * kEach + i) * 64 + lane;
      v[i] = t < tokens ? targets[t] : -1;
      g[i] = t < tokens && grad_loss ? __float_as_uint(grad_loss[t]) & 0x7fffffffu : 0u;
    }
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
      has[i] = v[i] >= 0 && v[i] < (int64_t)vocab;
      if (has[i] && g[i] < 0x7f800000u) top = g[i] > top ? g[i] : top;
    }
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
      mask[i] = __ballot(has[i]);
      mine += (uint32_t)__popcll(mask[i]);
    }
    __syncthreads();
    if (lane == 0) part[wave] = mine;
    __syncthreads();
    uint32_t place = before;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) {
      place += w < wave ? part[w] : 0u;
      before += part[w];
    }
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
      const uint64_t t = t0 + (wave * kEach + i) * 64 + lane;
      const uint32_t p = place + (uint32_t)__popcll(mask[i] & ((1ull << lane) - 1));
      if (t < tokens) {
        at[t] = has[i] ? (int32_t)p : -1;
        if (has[i]) list[p] = (int32_t)t;
      }
      place += (uint32_t)__popcll(mask[i]);
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top, d);
    top = o > top ? o : top;
  }
  if (lane == 0) tops[wave] = top;
  if (wave == 0 && rule.most) {
    const uint32_t parts = best_parts(rule, before);
    if (lane == 0) plan->parts = parts;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (uint32_t w = 1; w < kWaves; ++w) top = tops[w] > top ? tops[w] : top;
    plan->count = before;
    plan->grad_top = top ? __uint_as_float(top) : 1.f;
  }
}

__device__ __forceinline__ uint32_t two_bf16(float a, float b) {
  const bf16x2 p = __builtin_convertvector((f32x2){a, b}, bf16x2);
  uint32_t u;
  __builtin_memcpy(&u, &p, 4);
  return u;
}

__device__ __forceinline__ float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }

// The rows with a target: x packed, zeros up to the next multiple of kTileT.
__global__ __launch_bounds__(256) void cross_entropy_pack_kernel(CrossEntropyArgs p,
                                                                 const CrossEntropyPlan* __restrict__ plan,
                                                                 const int32_t* __restrict__ list, uint4* rows) {
  const uint32_t vecs = p.k / 8, count = plan->count;
  const uint64_t all = (uint64_t)tiles_of(count, kTileT) * kTileT * vecs;
  const uint64_t stride = (uint64_t)gridDim.x * 256;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += stride) {
    const uint32_t r = (uint32_t)(i / vecs), c = (uint32_t)(i - (uint64_t)r * vecs);
    rows[i] = r < count ? reinterpret_cast<const uint4*>(p.x)[(uint64_t)list[r] * vecs + c] : make_uint4(0, 0, 0, 0);
  }
}

// What the backward pass knows of a packed row: 1 / |p - 1|, lse in powers of two,
// the target, and the factor |p - 1| scale grad_loss of its gradients.  All zero for
// rows past the last one.
struct PackedRow {
  float over;
  float lse2;
  int32_t target;
  float factor;
};

// A row of the backward pass with its facts: x of token t, and x times factor over
// grad_top; p of its target by a product of its own.  By a workgroup; part: four floats
// that the row before has not used.
__device__ __forceinline__ void pack_row(const CrossEntropyArgs& p, const float* grad_loss, const float* lse, uint32_t t,
                                         int32_t target, float grad_top, float* part, uint4* to, uint4* to_scaled,
                                         PackedRow* about) {
  const uint32_t vecs = p.k / 8;
  const uint4* const x = reinterpret_cast<const uint4*>(p.x) + (uint64_t)t * vecs;
  const uint4* const w = reinterpret_cast<const uint4*>(p.w) + (uint64_t)target * vecs;
  float dot = 0.f;
  for (uint32_t c = threadIdx.x; c < vecs; c += 256) {
    const uint4 a = x[c], b = w[c];
    to[c] = a;
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dot = fmaf(bf16_lo(u[i]), bf16_lo(v[i]), dot);
      dot = fmaf(bf16_hi(u[i]), bf16_hi(v[i]), dot);
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
  __syncthreads();
  dot = part[0] + part[1] + part[2] + part[3];
  // p near one: |p - 1| is what the roundings of p leave, and 2^-20 will do
  const float lse2 = lse[t] * kLog2e, rest = fabsf(1.f - exp2_of(dot * p.scale * kLog2e - lse2));
  const float over = 1.f / (rest < 0x1p-20f ? 0x1p-20f : rest);  // a NaN stays
  const float factor = grad_loss[t] * p.scale / over, by = factor / grad_top;
  if (threadIdx.x == 0) *about = PackedRow{over, lse2, target, factor};
  for (uint32_t c = threadIdx.x; c < vecs; c += 256) {
    const uint4 a = x[c];
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = two_bf16(bf16_lo(u[i]) * by, bf16_hi(u[i]) * by);
    to_scaled[c] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}
__device__ __forceinline__ void clear_row(uint32_t vecs, uint4* to, uint4* to_scaled, PackedRow* about) {
  for (uint32_t c = threadIdx.x; c < vecs; c += 256) to[c] = to_scaled[c] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) *about = PackedRow{0.f, 0.f, -1, 0.f};
}

// The packed rows of the backward pass, a workgroup to a row.
__global__ __launch_bounds__(256) void cross_entropy_pack_bwd_kernel(
    CrossEntropyArgs p, const float* __restrict__ grad_loss, const float* __restrict__ lse,
    const CrossEntropyPlan* __restrict__ plan, const int32_t* __restrict__ list, uint4* rows, uint4* scaled,
    PackedRow* about) {
  __shared__ float part[2][4];
  const uint32_t vecs = p.k / 8, count = plan->count, all = tiles_of(count, kTileT) * kTileT;
  uint32_t turn = 0;
  for (uint32_t r = blockIdx.x; r < all; r += gridDim.x, turn ^= 1) {
    uint4* const to = rows + (uint64_t)r * vecs;
    uint4* const to_scaled = scaled + (uint64_t)r * vecs;
    if (r >= count) {  // the same for the whole workgroup
      clear_row(vecs, to, to_scaled, about + r);
      continue;
    }
    const uint32_t t = (uint32_t)list[r];
    pack_row(p, grad_loss, lse, t, (int32_t)p.targets[t], plan->grad_top, part[turn], to, to_scaled, about + r);
  }
}

// The plan and the packed rows at once, for tokens up to kPlanned: a workgroup to each,
// which counts the tokens before its own by itself.  One launch less: the loss of
// 509 x 10007 x 1056 takes 32.4 us instead of 37.8, its gradients 67 instead of 74.
constexpr uint32_t kPlanned = 1024;
template <bool kBackward>
__global__ __launch_bounds__(256) void cross_entropy_plan_pack_kernel(CrossEntropyArgs p, const float* __restrict__ grad_loss,
                                                                      const float* __restrict__ lse, PartsRule rule,
                                                                      CrossEntropyPlan* plan, int32_t* list, int32_t* at,
                                                                      uint4* rows, uint4* scaled, PackedRow* about) {
  __shared__ uint32_t sums[4][3];
  __shared__ float part[4];
  const uint32_t vecs = p.k / 8, t = blockIdx.x, tokens = (uint32_t)p.tokens;
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t own = t < tokens ? p.targets[t] : -1;
  const bool has = own >= 0 && own < (int64_t)p.vocab;
  uint32_t before = 0, count = 0, top = 0;
  constexpr uint32_t kEach = kPlanned / 256;
  int64_t v[kEach];
  uint32_t g[kEach];
#pragma unroll
  for (uint32_t i = 0; i < kEach; ++i) {
    const uint32_t o = 256 * i + threadIdx.x;
    v[i] = o < tokens ? p.targets[o] : -1;
    g[i] = kBackward && o < tokens ? __float_as_uint(grad_loss[o]) & 0x7fffffffu : 0u;
  }
#pragma unroll
  for (uint32_t i = 0; i < kEach; ++i) {
    const bool there = v[i] >= 0 && v[i] < (int64_t)p.vocab;
    count += (uint32_t)__popcll(__ballot(there));
    before += (uint32_t)__popcll(__ballot(there && 256 * i + threadIdx.x < t));
    if (there && g[i] < 0x7f800000u) top = g[i] > top ? g[i] : top;
  }
  if (kBackward) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)top, d);
      top = o > top ? o : top;
    }
  }
  if (lane == 0) sums[wave][0] = before, sums[wave][1] = count, sums[wave][2] = top;
  __syncthreads();
  before = count = top = 0;
#pragma unroll
  for (uint32_t w = 0; w < 4; ++w) {
    before += sums[w][0];
    count += sums[w][1];
    top = sums[w][2] > top ? sums[w][2] : top;
  }
  const float grad_top = top ? __uint_as_float(top) : 1.f;
  if (t == 0 && wave == 0) {
    const uint32_t parts = kBackward ? best_parts(rule, count) : 1;
    if (lane == 0) {
      plan->count = count;
      plan->grad_top = grad_top;
      plan->parts = parts;
    }
  }
  if (threadIdx.x == 0 && t < tokens) {
    at[t] = has ? (int32_t)before : -1;
    if (has) list[before] = (int32_t)t;
  }
  if (t >= count && t < tiles_of(count, kTileT) * kTileT) {  // the packed rows past the last one
    if (kBackward)
      clear_row(vecs, rows + (uint64_t)t * vecs, scaled + (uint64_t)t * vecs, about + t);
    else
      for (uint32_t c = threadIdx.x; c < vecs; c += 256) rows[(uint64_t)t * vecs + c] = make_uint4(0, 0, 0, 0);
  }
  if (!has) return;
  uint4* const to = rows + (uint64_t)before * vecs;
  if (kBackward)
    pack_row(p, grad_loss, lse, t, (int32_t)own, grad_top, part, to, scaled + (uint64_t)before * vecs, about + before);
  else
    for (uint32_t c = threadIdx.x; c < vecs; c += 256) to[c] = reinterpret_cast<const uint4*>(p.x)[(uint64_t)t * vecs + c];
}

// A maximum and the sum of 2^(value - maximum); an empty one is (-infinity, 0).
struct TopSum {
  float top, sum;
};
__device__ __forceinline__ TopSum join(TopSum a, TopSum b) {
  const float top = fmaxf(a.top, b.top);
  if (top == -__builtin_inff()) return TopSum{top, a.sum + b.sum};
  return TopSum{top, a.sum * exp2_of(a.top - top) + b.sum * exp2_of(b.top - top)};
}

// The logits' tile: rows i of the vocabulary from v0 (v_end: past the slice),
// columns j of tokens.
// Forward: part[tile of v][token], hit[token].  Backward: P.
struct LogitsArgs {
  CrossEntropyArgs p;
  const CrossEntropyPlan* plan;
  const int32_t* list;  // forward: the packed rows' tokens
  TopSum* part;         // [tiles of v, or shares][pitch]
  float* hit;
  uint64_t pitch;           // of part, tokens
  const uint16_t* rows;     // packed x
  const PackedRow* about;
  uint16_t* probs;          // P of the slice, [tokens rounded up][slice]
  uint32_t v0, slice;       // slice: a multiple of kTileT
};

// acc = the products of w's rows from v0 on and of `tokens` rows x (packed ones
// fill their tile).  Rows from v_end on, and past the tokens, are the tile's first
// again: their results are left out.  k is a multiple of 32: of a last half stage only the
// first k-step counts, and the lanes past its end read its own columns again.
//
// Rows at multiples of 4 KiB lie alike over the memory's channels, and workgroups in
// step with each other would all ask the same ones: of few tokens each begins at a place of its
// own in k (4 x 32000 x 8192: 118 -> 87 us, 1 x 32768 x 2048: 36 -> 30; with rows of
// other lengths it costs up to 3%).
template <class T>
__device__ __forceinline__ void logits_tile(char* ring, const CrossEntropyArgs& p, uint32_t v0, uint32_t v_end,
                                            const uint16_t* x, uint32_t tokens, v4f (&acc)[T::kI][T::kJ]) {
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  typename T::template Source<typename T::I> from_i;
  typename T::template Source<typename T::J> from_j;
  from_i.base = reinterpret_cast<const char*>(p.w + (uint64_t)v0 * p.k);
  from_j.base = reinterpret_cast<const char*>(x);
  from_i.step = from_j.step = 2 * kStageC;
#pragma unroll
  for (uint32_t n = 0; n < T::I::kCopies; ++n) {
    uint32_t row, col;
    T::I::place(wave, threadIdx.x & 63, n, row, col);
    from_i.off[n] = 2 * ((v0 + row < v_end ? row : 0) * p.k + col);
  }
#pragma unroll
  for (uint32_t n = 0; n < T::J::kCopies; ++n) {
    uint32_t row, col;
    T::J::place(wave, threadIdx.x & 63, n, row, col);
    from_j.off[n] = 2 * ((row < tokens ? row : 0) * p.k + col);
  }
  T::multiply(
      ring, tiles_of(p.k, kStageC), p.k / kStageC, p.k % kStageC != 0, from_i, from_j,
      [&](auto& i, auto& j) {
        const uint32_t lane = late_lane();
        uint32_t row, col;
#pragma unroll
        for (uint32_t n = 0; n < T::I::kCopies; ++n) {
          T::I::place(wave, lane, n, row, col);
          i.off[n] -= col < kStageC / 2 ? 0 : kStageC;
        }
#pragma unroll
        for (uint32_t n = 0; n < T::J::kCopies; ++n) {
          T::J::place(wave, lane, n, row, col);
          j.off[n] -= col < kStageC / 2 ? 0 : kStageC;
        }
      },
      acc, T::kStreams && p.k % 2048 == 0 ? blockIdx.x * 5 % (p.k / kStageC) : 0);
}

// The maximum and sum of a tile's column for each token, one per wave and token to
// sums[wave's rows][token]; the targets' logits to hit, in powers of two as the
// maxima are.  target_of(t), t from t0 on: the token's target below v_end, or -1.
// Rows from v_end on are left out.
template <class T, class TargetOf>
__device__ __forceinline__ void column_sums(v4f (&acc)[T::kI][T::kJ], float scale, uint32_t v0, uint32_t v_end, uint32_t t0,
                                            TargetOf target_of, float* hit, TopSum* sums) {
  const uint32_t lane = late_lane(), g = lane >> 4, r = lane & 15;
  const uint32_t wi = T::wave_i(), wj = T::wave_j();
  const float to_log2 = scale * kLog2e;
  const bool ends = v0 + T::kRowsI > v_end;
#pragma unroll
  for (int j = 0; j < T::kJ; ++j) {
    const uint32_t t = t0 + wj + 16 * j + r;
    int32_t target = target_of(t);
    __builtin_amdgcn_sched_barrier(0);  // a block's values at a time: all of them would not fit the registers
    target -= (int32_t)(v0 + wi);       // a target of -1 is below every row
    const bool hits = __ballot(target >= 0 && target < 16 * T::kI) != 0;
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < T::kI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t row = T::row_of(i, g, e);
        float z = acc[i][j][e] * to_log2;
        if (hits && target == (int32_t)row) hit[t] = z;
        if (ends && v0 + wi + row >= v_end) z = -__builtin_inff();
        acc[i][j][e] = z;
        top = fmaxf(top, z);
      }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float from = top == -__builtin_inff() ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < T::kI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += exp2_of(acc[i][j][e] - from);
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (g == 0) sums[wi / (16 * T::kI) * T::kRowsJ + wj + 16 * j + r] = TopSum{top, sum};
  }
}

// Few tokens: bound by w's bytes, which stream past the caches.  Each workgroup takes
// an equal share of w's rows, whatever their number (whole tiles would leave the last
// turn's units idle: 100003 rows in tiles of 128 are one and a half turns), a tile's
// rows at a time, and leaves one sum.  The tokens' rows come from the caches once for
// each tile, so that 64 tokens go with 128 rows (61 x 100003 x 7168: 244 us, 5.9 TB/s;
// with 64 rows 284).  32 tokens go with 64, four workgroups to a compute unit, which
// cover each other's ends (16 x 131072 x 2048: 93 us; two deeper ones took 108 where four took 97).
template <class T, int kPerCu>
__global__ __launch_bounds__(256, kPerCu) void cross_entropy_few_kernel(LogitsArgs a) {
  __shared__ __attribute__((aligned(1024))) char ring[T::kLds];
  const CrossEntropyArgs& p = a.p;
  const uint64_t shares = tiles_of(p.vocab, 16);
  const uint32_t first = (uint32_t)(blockIdx.x * shares / gridDim.x) * 16;
  const uint64_t past = ((uint64_t)blockIdx.x + 1) * shares / gridDim.x * 16;
  const uint32_t end = past < p.vocab ? (uint32_t)past : p.vocab, count = (uint32_t)p.tokens;
  TopSum all{-__builtin_inff(), 0.f};  // of token threadIdx.x
  for (uint32_t v0 = first; v0 < end; v0 += T::kRowsI) {
    v4f acc[T::kI][T::kJ] = {};
    logits_tile<T>(ring, p, v0, end, p.x, count, acc);
    TopSum* const sums = reinterpret_cast<TopSum*>(ring);
    column_sums<T>(
        acc, p.scale, v0, end, 0,
        [&](uint32_t t) -> int32_t {
          const int64_t v = t < count ? p.targets[t] : -1;
          return v >= 0 && v < (int64_t)end ? (int32_t)v : -1;
        },
        a.hit, sums);
    __syncthreads();
    if (threadIdx.x < T::kRowsJ) {
#pragma unroll
      for (int w = 0; w < T::kWI; ++w) all = join(all, sums[w * T::kRowsJ + threadIdx.x]);
    }
    __syncthreads();  // the next tile's copies go there
  }
  if (threadIdx.x < count) a.part[blockIdx.x * a.pitch + threadIdx.x] = all;
}

//
// Bound by the tile loop (matrix units busy 52%): 5734 tokens of 131072 x 2048 in 2.74
// ms, 1.13 PFLOP/s, of the library's products of this shape 1.27 to 1.51, which leave their
// logits in memory; the backward pass's 65536 columns at a time in 1.37 ms, 1.13 PFLOP/s.
template <class T, bool kBackward, int kPerCu>
__global__ __launch_bounds__(256, kPerCu) void cross_entropy_logits_kernel(LogitsArgs a) {
  __shared__ __attribute__((aligned(1024))) char ring[T::kLds];
  const CrossEntropyArgs& p = a.p;
  const uint32_t count = a.plan->count;
  const uint32_t v_end = p.vocab - a.v0 < a.slice ? p.vocab : a.v0 + a.slice;
  const uint32_t tiles_v = tiles_of(v_end - a.v0, T::kRowsI), tiles_t = tiles_of(count, T::kRowsJ);
  const uint64_t tiles = (uint64_t)tiles_v * tiles_t;
  const uint64_t tile = xcd_tile(blockIdx.x, tiles);
  if (tile >= tiles) return;
  // eight tiles of tokens at a time: an XCD's tiles share rows of both operands
  constexpr uint32_t kGroup = 8;
  const uint32_t group = (uint32_t)(tile / ((uint64_t)kGroup * tiles_v));
  const uint32_t in = (uint32_t)(tile - (uint64_t)group * kGroup * tiles_v);
  const uint32_t wide = tiles_t - group * kGroup < kGroup ? tiles_t - group * kGroup : kGroup;
  const uint32_t tile_v = in / wide, tile_t = group * kGroup + in % wide;
  const uint32_t v0 = a.v0 + tile_v * T::kRowsI, t0 = tile_t * T::kRowsJ;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  v4f acc[T::kI][T::kJ] = {};
  logits_tile<T>(ring, p, v0, p.vocab, a.rows + (uint64_t)t0 * p.k, T::kRowsJ, acc);

  if constexpr (!kBackward) {
    column_sums<T>(
        acc, p.scale, v0, v_end, t0,
        [&](uint32_t t) -> int32_t { return t < count ? (int32_t)p.targets[(uint32_t)a.list[t]] : -1; }, a.hit,
        reinterpret_cast<TopSum*>(ring));
  } else {
    // blocks 2 q and 2 q + 1: v = wi + 32 q + 8 g + 0 .. 7; block j: token wj + 16 j + r
    const uint32_t lane = late_lane(), g = lane >> 4, r = lane & 15;
    const uint32_t wi = T::wave_i(), wj = T::wave_j();
    const float to_log2 = p.scale * kLog2e;
    const bool ends = v0 + T::kRowsI > v_end;
    static_assert(T::kPairs && T::kJ % 2 == 0, "32 rows of P at a time");
    const RowBlock<2 * T::kI> block{ring + 1024 * T::kI * wave};
#pragma unroll
    for (int j = 0; j < T::kJ; ++j) {
      const PackedRow about = a.about[t0 + wj + 16 * j + r];
      __builtin_amdgcn_sched_barrier(0);  // a block's values at a time: all of them would not fit the registers
      const int32_t target = about.target - (int32_t)(v0 + wi);
      const bool hits = __ballot(target >= 0 && target < 16 * T::kI) != 0;
      // rows past the last token are zero whatever w holds: grad_w's products take them in
      const uint32_t there = about.target < 0 ? 0u : ~0u;
#pragma unroll
      for (int q = 0; q < T::kI / 2; ++q) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          float d[2];
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const uint32_t row = 32 * q + 8 * g + e + o;
            float v = exp2_of(acc[2 * q + e / 4][j][e % 4 + o] * to_log2 - about.lse2);
            if (hits && target == (int32_t)row) v -= 1.f;
            d[o] = ends && v0 + wi + row >= v_end ? 0.f : v * about.over;
          }
          u[e / 2] = two_bf16(d[0], d[1]) & there;
        }
        block.put(16 * (j & 1) + r, 4 * q + g, make_uint4(u[0], u[1], u[2], u[3]));
      }
      if (j & 1)
        block.drain([&](uint32_t row, uint32_t piece, uint4 v) {
          const uint64_t at = (uint64_t)(t0 + wj + 16 * (j - 1) + row) * a.slice + (v0 - a.v0) + wi + 8 * piece;
          *reinterpret_cast<uint4*>(a.probs + at) = v;
        });
    }
  }
  if constexpr (!kBackward) {
    __syncthreads();
    for (uint32_t j = threadIdx.x; j < T::kRowsJ; j += 256) {
      TopSum s = reinterpret_cast<const TopSum*>(ring)[j];
#pragma unroll
      for (int w = 1; w < T::kWI; ++w) s = join(s, reinterpret_cast<const TopSum*>(ring)[w * T::kRowsJ + j]);
      if (t0 + j < count) a.part[(uint64_t)tile_v * a.pitch + t0 + j] = s;
    }
  }
}

// Joins the tiles: kEach tokens to a workgroup, 256 / kEach lanes to each.
template <uint32_t kEach>
__global__ __launch_bounds__(256) void cross_entropy_join_kernel(CrossEntropyArgs p, const int32_t* __restrict__ at,
                                                                 const TopSum* __restrict__ part, uint64_t pitch,
                                                                 uint32_t tiles, const float* __restrict__ hit,
                                                                 float* __restrict__ loss, float* __restrict__ lse) {
  constexpr uint32_t kShares = 256 / kEach, kAtOnce = 8;
  __shared__ TopSum sums[256];
  const uint32_t j = threadIdx.x % kEach, share = threadIdx.x / kEach;
  const uint64_t t = (uint64_t)blockIdx.x * kEach + j;
  bool has = t < p.tokens;
  uint64_t place = t;
  if (has) {
    if (at) {
      has = at[t] >= 0;
      place = has ? (uint32_t)at[t] : 0;
    } else {
      const int64_t v = p.targets[t];
      has = v >= 0 && v < (int64_t)p.vocab;
    }
  }
  TopSum s{-__builtin_inff(), 0.f};
  if (has) {
    for (uint32_t i0 = share; i0 < tiles; i0 += kShares * kAtOnce) {
      TopSum v[kAtOnce];
#pragma unroll
      for (uint32_t n = 0; n < kAtOnce; ++n) {
        const uint32_t i = i0 + n * kShares;
        v[n] = part[(i < tiles ? i : tiles - 1) * pitch + place];
        if (i >= tiles) v[n] = TopSum{-__builtin_inff(), 0.f};
      }
#pragma unroll
      for (uint32_t n = 0; n < kAtOnce; ++n) s = join(s, v[n]);
    }
  }
  sums[threadIdx.x] = s;
  __syncthreads();
#pragma unroll
  for (uint32_t d = kShares / 2; d >= 1; d >>= 1) {
    if (share < d) sums[threadIdx.x] = join(sums[threadIdx.x], sums[threadIdx.x + kEach * d]);
    __syncthreads();
  }
  if (share == 0 && t < p.tokens) {
    const TopSum all = sums[j];
    // the target's logit is one of those that the maximum was taken from and the sum is one at least: no loss is
    // below zero, and a confident token's keeps nothing of its logit's roundings
    const float log_sum = has ? logf(all.sum) : 0.f;
    lse[t] = has ? all.top * kLn2 + log_sum : 0.f;
    loss[t] = has ? (all.top - hit[place]) * kLn2 + log_sum : 0.f;
  }
}

// grad_x's sums over a slice of the vocabulary: i along k, j the packed tokens.
// 5734 tokens, 2048, 65536 columns: 1.43 ms, 1.08 PFLOP/s, bound by the tile loop.
struct GradRowsArgs {
  CrossEntropyArgs p;
  const CrossEntropyPlan* plan;
  const uint16_t* probs;
  uint32_t v0, slice;
  bool first;     // of the slices
  float one;      // 1: a product takes the sums out of the registers that hold them
  float* sums;    // [parts][pitch][k]
  uint64_t pitch;
};
template <class T>
__device__ __forceinline__ void grad_rows_tile(char* ring, const GradRowsArgs& a, uint32_t group) {
  const CrossEntropyArgs& p = a.p;
  const uint32_t tiles_k = tiles_of(p.k, T::kRowsI), tiles_t = tiles_of(a.plan->count, T::kRowsJ);
  const uint32_t parts = a.plan->parts;
  const uint64_t tiles = (uint64_t)tiles_k * tiles_t * parts;
  const uint64_t tile = xcd_tile(group, tiles);
  if (tile >= tiles) return;
  const uint32_t part = (uint32_t)(tile / ((uint64_t)tiles_k * tiles_t));
  const uint32_t in = (uint32_t)(tile - (uint64_t)part * tiles_k * tiles_t);
  const uint32_t k0 = in % tiles_k * T::kRowsI, t0 = in / tiles_k * T::kRowsJ;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t all = tiles_of(p.vocab - a.v0 < a.slice ? p.vocab - a.v0 : a.slice, kStageC);
  const uint32_t begin = (uint32_t)((uint64_t)all * part / parts), end = (uint32_t)((uint64_t)all * (part + 1) / parts);
  const uint32_t left = p.vocab - a.v0;  // rows of w from the slice on; P is zero past them, any row will do
  typename T::template Source<typename T::I> from_i;
  typename T::template Source<typename T::J> from_j;
  from_i.base = reinterpret_cast<const char*>(p.w + ((uint64_t)a.v0 + begin * kStageC) * p.k + k0);
  from_i.step = 2 * kStageC * (uint64_t)p.k;
  from_j.base = reinterpret_cast<const char*>(a.probs + (uint64_t)t0 * a.slice + begin * kStageC);
  from_j.step = 2 * kStageC;
#pragma unroll
  for (uint32_t n = 0; n < T::I::kCopies; ++n) {
    uint32_t row, col;
    T::I::place(wave, threadIdx.x & 63, n, row, col);
    from_i.off[n] = 2 * (row * p.k + (k0 + col < p.k ? col : 0));
  }
#pragma unroll
  for (uint32_t n = 0; n < T::J::kCopies; ++n) {
    uint32_t row, col;
    T::J::place(wave, threadIdx.x & 63, n, row, col);
    from_j.off[n] = 2 * (row * a.slice + col);
  }
  v4f acc[T::kI][T::kJ] = {};
  T::multiply(
      ring, end - begin, end * kStageC <= left ? end - begin : end - 1 - begin, false, from_i, from_j,
      [&](auto& i, auto&) {
        const uint32_t there = left - (end - 1) * kStageC, lane = late_lane();  // rows of the last stage
        uint32_t row, col;
#pragma unroll
        for (uint32_t n = 0; n < T::I::kCopies; ++n) {
          T::I::place(wave, lane, n, row, col);
          i.off[n] -= 2 * p.k * (row - (row < there ? row : there - 1));
        }
      },
      acc);
  const uint32_t lane = late_lane(), g = lane >> 4, r = lane & 15;
  const uint32_t wi = T::wave_i(), wj = T::wave_j();
  float* const sums = a.sums + (part * a.pitch + t0 + wj) * p.k + k0 + wi;
#pragma unroll
  for (int j = 0; j < T::kJ; ++j)
#pragma unroll
    for (int i = 0; i < T::kI; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      if (k0 + wi + 16 * i >= p.k) continue;  // k is a multiple of 32
      v4f* const at = reinterpret_cast<v4f*>(sums + ((16 * j + r) * p.k + 16 * i + 4 * g));
      v4f v = acc[i][j] * a.one;
      if (!a.first) v += *at;
      *at = v;
    }
}
template <class T, int kPerCu>
__global__ __launch_bounds__(256, kPerCu) void cross_entropy_grad_rows_kernel(GradRowsArgs a) {
  __shared__ __attribute__((aligned(1024))) char ring[T::kLds];
  grad_rows_tile<T>(ring, a, blockIdx.x);
}

// grad_x = the rows' factors times the parts' sums, to the tokens' own rows; zeros for ignored ones.
__global__ __launch_bounds__(256) void cross_entropy_rows_kernel(CrossEntropyArgs p, const PackedRow* __restrict__ about,
                                                                 const int32_t* __restrict__ at,
                                                                 const float* __restrict__ sums,
                                                                 const CrossEntropyPlan* __restrict__ plan,
                                                                 uint64_t pitch, uint16_t* __restrict__ grad_x) {
  const uint32_t vecs = p.k / 8, parts = plan->parts;
  const uint64_t all = p.tokens * vecs, stride = (uint64_t)gridDim.x * 256;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += stride) {
    const uint64_t t = i / vecs, c = i - t * vecs;
    const int32_t row = at[t];
    uint32_t u[4] = {0, 0, 0, 0};
    if (row >= 0) {
      const float by = about[row].factor;
      v4f lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
#pragma unroll 4
      for (uint32_t s = 0; s < parts; ++s) {
        const v4f* from = reinterpret_cast<const v4f*>(sums + (s * pitch + (uint32_t)row) * p.k + 8 * c);
        lo += from[0];
        hi += from[1];
      }
      lo *= by;
      hi *= by;
      u[0] = two_bf16(lo[0], lo[1]);
      u[1] = two_bf16(lo[2], lo[3]);
      u[2] = two_bf16(hi[0], hi[1]);
      u[3] = two_bf16(hi[2], hi[3]);
    }
    reinterpret_cast<uint4*>(grad_x)[i] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// grad_w's rows of a slice: i along k, j the vocabulary.  5734 tokens, 2048, 65536
// columns: 1.29 ms, 1.19 PFLOP/s, where a library product of these layouts does 1.01 to 1.13.
struct GradWeightArgs {
  CrossEntropyArgs p;
  const CrossEntropyPlan* plan;
  const uint16_t* rows;  // scaled
  const uint16_t* probs;
  uint32_t v0, slice;
  uint16_t* grad_w;
};
template <class T>
__device__ __forceinline__ void grad_weight_tile(char* ring, GradWeightArgs a, uint32_t group) {
  static_assert(T::kJ % 2 == 0, "32 rows of the result at a time");
  const CrossEntropyArgs& p = a.p;
  const uint32_t left = p.vocab - a.v0 < a.slice ? p.vocab - a.v0 : a.slice;
  const uint32_t tiles_k = tiles_of(p.k, T::kRowsI), tiles_v = tiles_of(left, T::kRowsJ);
  const uint64_t tiles = (uint64_t)tiles_k * tiles_v;
  const uint64_t tile = xcd_tile(group, tiles);
  if (tile >= tiles) return;
  const uint32_t k0 = (uint32_t)(tile % tiles_k) * T::kRowsI, v0 = (uint32_t)(tile / tiles_k) * T::kRowsJ;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  typename T::template Source<typename T::I> from_i;
  typename T::template Source<typename T::J> from_j;
  from_i.base = reinterpret_cast<const char*>(a.rows + k0);
  from_i.step = 2 * kStageC * (uint64_t)p.k;
  from_j.base = reinterpret_cast<const char*>(a.probs + v0);
  from_j.step = 2 * kStageC * (uint64_t)a.slice;
#pragma unroll
  for (uint32_t n = 0; n < T::I::kCopies; ++n) {
    uint32_t row, col;
    T::I::place(wave, threadIdx.x & 63, n, row, col);
    from_i.off[n] = 2 * (row * p.k + (k0 + col < p.k ? col : 0));
  }
#pragma unroll
  for (uint32_t n = 0; n < T::J::kCopies; ++n) {
    uint32_t row, col;
    T::J::place(wave, threadIdx.x & 63, n, row, col);
    from_j.off[n] = 2 * (row * a.slice + col);
  }
  v4f acc[T::kI][T::kJ] = {};
  const uint32_t stages = tiles_of(a.plan->count, kStageC);  // the packed rows and P fill whole ones
  T::multiply(ring, stages, stages, false, from_i, from_j, [](auto&, auto&) {}, acc);
  const uint32_t lane = late_lane(), g = lane >> 4, r = lane & 15;
  const uint32_t wi = T::wave_i(), wj = T::wave_j();
  const float by = a.plan->grad_top;
  const RowBlock<2 * T::kI> block{ring + 1024 * T::kI * wave};
#pragma unroll
  for (int j = 0; j < T::kJ; ++j) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < T::kI; ++i) {
      const v4f v = acc[i][j] * by;
      *reinterpret_cast<uint2*>(block.at(16 * (j & 1) + r, 2 * i + (g >> 1)) + 8 * (g & 1)) =
          make_uint2(two_bf16(v[0], v[1]), two_bf16(v[2], v[3]));
    }
    if (j & 1)
      block.drain([&](uint32_t row, uint32_t piece, uint4 v) {
        const uint32_t n = v0 + wj + 16 * (j - 1) + row, k = k0 + wi + 8 * piece;
        if (n < left && k < p.k) *reinterpret_cast<uint4*>(a.grad_w + ((uint64_t)a.v0 + n) * p.k + k) = v;
      });
  }
}

template <class T, int kPerCu>
__global__ __launch_bounds__(256, kPerCu) void cross_entropy_grad_weight_kernel(GradWeightArgs a) {
  __shared__ __attribute__((aligned(1024))) char ring[T::kLds];
  grad_weight_tile<T>(ring, a, blockIdx.x);
}

// Both, where tiles of 128 do for both: neither fills the card to its end, and the
// one's tiles run beside the other's (509 x 10007 x 1056: 32 us instead of 21 and 19).
// The first `rows` workgroups, as a rule the longer tiles, do grad_x.
template <class TRows, class TWeight>
__global__ __launch_bounds__(256, 2) void cross_entropy_grads_kernel(GradRowsArgs a, GradWeightArgs b, uint32_t rows) {
  static_assert(TRows::kLds == TWeight::kLds, "one ring for either");
  __shared__ __attribute__((aligned(1024))) char ring[TRows::kLds];
  if (blockIdx.x < rows)
    grad_rows_tile<TRows>(ring, a, blockIdx.x);
  else
    grad_weight_tile<TWeight>(ring, b, blockIdx.x - rows);
}

// grad_w of no tokens.
__global__ __launch_bounds__(256) void cross_entropy_clear_kernel(uint4* out, uint64_t nvec) {
  const uint64_t stride = (uint64_t)gridDim.x * 256;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < nvec; i += stride) out[i] = make_uint4(0, 0, 0, 0);
}

}  // namespace trace_dev

namespace trace_host {

using namespace trace_dev;

namespace {

constexpr uint64_t round_up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

// Tiles: vocabulary x tokens, k x tokens, k x vocabulary.
using Logits256 = Tile<8, 8, 2, 2, false, false, 2>;
using Logits128 = Tile<4, 4, 2, 2, false, false, 2>;
using Few64 = Tile<2, 4, 4, 1, false, false, 3, true>;
using Few32 = Tile<1, 2, 4, 1, false, false, 3, true>;
using GradRows256 = Tile<8, 8, 2, 2, true, false, 2>;
using GradRows128 = Tile<4, 4, 2, 2, true, false, 2>;
using GradWeight256 = Tile<8, 8, 2, 2, true, true, 2>;
using GradWeight128 = Tile<4, 4, 2, 2, true, true, 2>;

constexpr uint64_t tiles_in(uint64_t n, uint64_t m, uint64_t each) { return (n + each - 1) / each * ((m + each - 1) / each); }

constexpr uint64_t kMostTiles = (1u << 24) - 8;  // a launch counts its work-items in 32 bits

// Whether n x m results are done in tiles of 128 rather than 256: they read the
// operands twice as often, and have to be a tenth better for it.
bool small_tiles(uint64_t n, uint64_t m) {
  const uint64_t small = tiles_in(n, m, 128);
  return small <= kMostTiles && 10 * stage_time(small, true) < 9 * stage_time(tiles_in(n, m, 256), false);
}

// Few tokens are not listed: every one is computed, in its own place.
constexpr uint64_t kFew = 64;
constexpr uint32_t kJoinEach = 16;  // listed tokens to a workgroup where their tiles are joined
constexpr uint32_t kFewGroups = 1024;  // workgroups for them, of 64 rows of w at least

// Sums that the forward leaves for each token.
uint32_t logits_parts(uint64_t tokens, uint32_t vocab) {
  if (tokens > kFew) return (uint32_t)tiles_in(vocab, 1, small_tiles(tokens, vocab) ? 128 : 256);
  const uint32_t shares = (vocab + 63) / 64;
  return shares < kFewGroups ? shares : kFewGroups;
}

// Workspace of the forward.
struct ForwardSpace {
  uint64_t pitch, tiles, list, at, rows, part, hit, bytes;
  ForwardSpace(uint64_t tokens, uint32_t vocab, uint32_t k) {
    pitch = tokens > kFew ? round_up(tokens, 16) : tokens;
    tiles = logits_parts(tokens, vocab);
    const uint64_t lists = tokens > kFew ? 4 * pitch : 0;
    list = sizeof(CrossEntropyPlan);
    at = list + lists;
    rows = at + lists;
    hit = rows + (tokens > kFew ? 2 * round_up(tokens, kTileT) * k : 0);
    part = hit + round_up(4 * pitch, 16);
    bytes = part + tiles * pitch * sizeof(TopSum);
  }
};

// Workspace of the backward pass.
struct BackwardSpace {
  uint64_t tall;   // tokens rounded up to whole tiles
  uint32_t slice;  // of the vocabulary
  PartsRule parts;  // of a slice's contraction for grad_x
  uint64_t list, at, about, rows, scaled, probs, sums, bytes;
  BackwardSpace(uint64_t tokens, uint32_t vocab, uint32_t k) {
    tall = round_up(tokens, kTileT);
    // P of a gigabyte, but at least 8192 columns, to fill the card with tiles of grad_w; each
    // slice reads and writes grad_x's sums once
    uint64_t s = (1ull << 29) / tall / kTileT * kTileT;
    if (s < 8192) s = 8192;
    if (s > round_up(vocab, kTileT)) s = round_up(vocab, kTileT);
    slice = (uint32_t)s;
    // as many as all tokens could want, eight stages at least to each; the ones of a
    // call are chosen when the tokens with a target are known
    parts = PartsRule{0, (uint32_t)(s / kStageC), k, false};
    uint64_t best = ~0ull;
    for (const bool small : {false, true})
      for (uint32_t n = 1; n <= 16 && (n == 1 || 8 * n <= parts.stages); ++n) {
        const uint64_t time =
            (small ? 10 : 9) * parts_time(tiles_in(tokens, k, small ? 128 : 256), n, parts.stages, tall * k, small);
        if (time < best && (!small || tiles_in(tokens, k, 128) * 16 <= kMostTiles)) best = time, parts.small = small;
      }
    // fewer tokens fill fewer tiles, and want more parts: up to four turns
    const uint64_t tiles = tiles_in(tokens, k, parts.small ? 128 : 256), turns = (parts.small ? 2048 : 1024) / tiles;
    parts.most = (uint32_t)(turns < 1 ? 1 : (turns > 16 ? 16 : turns));
    if (8 * parts.most > parts.stages) parts.most = parts.stages < 8 ? 1 : parts.stages / 8;
    list = sizeof(CrossEntropyPlan);
    at = list + 4 * tall;
    about = at + 4 * tall;
    rows = about + sizeof(PackedRow) * tall;
    scaled = rows + 2 * tall * k;
    probs = scaled + 2 * tall * k;
    sums = probs + 2 * tall * slice;
    bytes = sums + 4 * (uint64_t)parts.most * tall * k;
  }
};

dim3 vector_grid(uint64_t vecs) {
  const uint64_t n = (vecs + 255) / 256, most = 8192 < kMaxGroups ? 8192 : kMaxGroups;
  return dim3((uint32_t)(n < most ? n : most));
}

uint32_t xcd_grid(uint64_t tiles) { return (uint32_t)((tiles + 7) / 8 * 8); }

}  // namespace

uint64_t cross_entropy_workspace_bytes(uint64_t tokens, uint32_t vocab, uint32_t k) {
  return ForwardSpace(tokens, vocab, k).bytes;
}

uint64_t cross_entropy_bwd_workspace_bytes(uint64_t tokens, uint32_t vocab, uint32_t k) {
  return BackwardSpace(tokens, vocab, k).bytes;
}

hipError_t launch_cross_entropy(const CrossEntropyArgs& p, float* loss, float* lse, hipStream_t stream) {
  const ForwardSpace s(p.tokens, p.vocab, p.k);
  if (tiles_in(p.tokens, p.vocab, 256) > kMostTiles || (p.tokens > kFew && p.tokens / kJoinEach >= kMostTiles))
    return hipErrorInvalidConfiguration;
  char* const at = static_cast<char*>(p.workspace);
  const bool listed = p.tokens > kFew;
  LogitsArgs a{};
  a.p = p;
  a.part = reinterpret_cast<TopSum*>(at + s.part);
  a.hit = reinterpret_cast<float*>(at + s.hit);
  a.pitch = s.pitch;
  a.slice = (uint32_t)round_up(p.vocab, kTileT);
  CrossEntropyPlan* const plan = reinterpret_cast<CrossEntropyPlan*>(at);
  int32_t* const list = reinterpret_cast<int32_t*>(at + s.list);
  int32_t* const places = listed ? reinterpret_cast<int32_t*>(at + s.at) : nullptr;
  if (listed) {
    uint16_t* const rows = reinterpret_cast<uint16_t*>(at + s.rows);
    const uint64_t tall = round_up(p.tokens, kTileT);
    if (p.tokens <= kPlanned) {
      hipLaunchKernelGGL(cross_entropy_plan_pack_kernel<false>, dim3((uint32_t)tall), dim3(256), 0, stream, p,
                         (const float*)nullptr, (const float*)nullptr, PartsRule{}, plan, list, places,
                         reinterpret_cast<uint4*>(rows), (uint4*)nullptr, (PackedRow*)nullptr);
    } else {
      hipLaunchKernelGGL(cross_entropy_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p.targets, (const float*)nullptr,
                         (uint32_t)p.tokens, p.vocab, PartsRule{}, plan, list, places);
      if (hipError_t e = hipGetLastError()) return e;
      hipLaunchKernelGGL(cross_entropy_pack_kernel, vector_grid(tall * (p.k / 8)), dim3(256), 0, stream, p,
                         (const CrossEntropyPlan*)plan, (const int32_t*)list, reinterpret_cast<uint4*>(rows));
    }
    if (hipError_t e = hipGetLastError()) return e;
    a.plan = plan;
    a.list = list;
    a.rows = rows;
  }
  if (!listed) {
    hipLaunchKernelGGL((p.tokens <= 32 ? cross_entropy_few_kernel<Few32, 4> : cross_entropy_few_kernel<Few64, 2>),
                       dim3((uint32_t)s.tiles), dim3(256), 0, stream, a);
  } else {
    const bool small = small_tiles(p.tokens, p.vocab);
    hipLaunchKernelGGL((small ? cross_entropy_logits_kernel<Logits128, false, 2>
                              : cross_entropy_logits_kernel<Logits256, false, 1>),
                       dim3(xcd_grid(tiles_in(p.tokens, p.vocab, small ? 128 : 256))), dim3(256), 0, stream, a);
  }
  if (hipError_t e = hipGetLastError()) return e;
  const auto join = [&](auto each, auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((uint32_t)((p.tokens + each - 1) / each)), dim3(256), 0, stream, p, places,
                       (const TopSum*)a.part, s.pitch, (uint32_t)s.tiles, (const float*)a.hit, loss, lse);
  };
  if (listed)  // neighbouring tokens' parts lie together
    join(kJoinEach, cross_entropy_join_kernel<kJoinEach>);
  else
    join(1u, cross_entropy_join_kernel<1>);
  return hipGetLastError();
}

hipError_t launch_cross_entropy_bwd(const CrossEntropyArgs& p, const float* grad_loss, const float* lse,
                                    uint16_t* grad_x, uint16_t* grad_w, hipStream_t stream) {
  if (p.tokens == 0) {
    const uint64_t vecs = (uint64_t)p.vocab * p.k / 8;
    hipLaunchKernelGGL(cross_entropy_clear_kernel, vector_grid(vecs), dim3(256), 0, stream, reinterpret_cast<uint4*>(grad_w),
                       vecs);
    return hipGetLastError();
  }
  const BackwardSpace s(p.tokens, p.vocab, p.k);
  if (tiles_in(p.tokens, s.slice, 256) > kMostTiles || tiles_in(s.slice, p.k, 256) > kMostTiles ||
      tiles_in(p.tokens, p.k, s.parts.small ? 128 : 256) * s.parts.most > kMostTiles)
    return hipErrorInvalidConfiguration;
  char* const at = static_cast<char*>(p.workspace);
  CrossEntropyPlan* const plan = reinterpret_cast<CrossEntropyPlan*>(at);
  int32_t* const list = reinterpret_cast<int32_t*>(at + s.list);
  int32_t* const places = reinterpret_cast<int32_t*>(at + s.at);
  PackedRow* const about = reinterpret_cast<PackedRow*>(at + s.about);
  uint16_t* const rows = reinterpret_cast<uint16_t*>(at + s.rows);
  uint16_t* const scaled = reinterpret_cast<uint16_t*>(at + s.scaled);
  uint16_t* const probs = reinterpret_cast<uint16_t*>(at + s.probs);
  float* const sums = reinterpret_cast<float*>(at + s.sums);
  if (p.tokens <= kPlanned) {
    hipLaunchKernelGGL(cross_entropy_plan_pack_kernel<true>, dim3((uint32_t)s.tall), dim3(256), 0, stream, p, grad_loss, lse,
                       s.parts, plan, list, places, reinterpret_cast<uint4*>(rows), reinterpret_cast<uint4*>(scaled), about);
  } else {
    hipLaunchKernelGGL(cross_entropy_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p.targets, grad_loss,
                       (uint32_t)p.tokens, p.vocab, s.parts, plan, list, places);
    if (hipError_t e = hipGetLastError()) return e;
    const uint64_t most = 8192 < kMaxGroups ? 8192 : kMaxGroups;
    hipLaunchKernelGGL(cross_entropy_pack_bwd_kernel, dim3((uint32_t)(s.tall < most ? s.tall : most)), dim3(256), 0, stream,
                       p, grad_loss, lse, (const CrossEntropyPlan*)plan, (const int32_t*)list,
                       reinterpret_cast<uint4*>(rows), reinterpret_cast<uint4*>(scaled), about);
  }
  if (hipError_t e = hipGetLastError()) return e;
  for (uint64_t v0 = 0; v0 < p.vocab; v0 += s.slice) {
    const uint64_t cols = p.vocab - v0 < s.slice ? p.vocab - v0 : s.slice;
    LogitsArgs a{};
    a.p = p;
    a.plan = plan;
    a.rows = rows;
    a.about = about;
    a.probs = probs;
    a.v0 = (uint32_t)v0;
    a.slice = s.slice;
    const auto grid = [&](uint64_t n, uint64_t m, uint64_t parts, bool small) {
      return dim3(xcd_grid(tiles_in(n, m, small ? 128 : 256) * parts));
    };
    const bool small = small_tiles(p.tokens, cols);
    hipLaunchKernelGGL((small ? cross_entropy_logits_kernel<Logits128, true, 2>
                              : cross_entropy_logits_kernel<Logits256, true, 1>),
                       grid(p.tokens, cols, 1, small), dim3(256), 0, stream, a);
    if (hipError_t e = hipGetLastError()) return e;
    const GradRowsArgs of_x{p, plan, probs, (uint32_t)v0, s.slice, v0 == 0, 1.f, sums, s.tall};
    const GradWeightArgs of_w{p, plan, scaled, probs, (uint32_t)v0, s.slice, grad_w};
    const bool small_x = s.parts.small, small_w = small_tiles(cols, p.k);
    const dim3 grid_x = grid(p.tokens, p.k, s.parts.most, small_x), grid_w = grid(cols, p.k, 1, small_w);
    if (grad_x && grad_w && small_x && small_w && (uint64_t)grid_x.x + grid_w.x <= kMostTiles) {
      hipLaunchKernelGGL((cross_entropy_grads_kernel<GradRows128, GradWeight128>), dim3(grid_x.x + grid_w.x), dim3(256), 0,
                         stream, of_x, of_w, grid_x.x);
      if (hipError_t e = hipGetLastError()) return e;
      continue;
    }
    if (grad_x) {
      hipLaunchKernelGGL((small_x ? cross_entropy_grad_rows_kernel<GradRows128, 2>
                                  : cross_entropy_grad_rows_kernel<GradRows256, 1>),
                         grid_x, dim3(256), 0, stream, of_x);
      if (hipError_t e = hipGetLastError()) return e;
    }
    if (grad_w) {
      hipLaunchKernelGGL((small_w ? cross_entropy_grad_weight_kernel<GradWeight128, 2>
                                  : cross_entropy_grad_weight_kernel<GradWeight256, 1>),
                         grid_w, dim3(256), 0, stream, of_w);
      if (hipError_t e = hipGetLastError()) return e;
    }
  }
  if (grad_x) {
    hipLaunchKernelGGL(cross_entropy_rows_kernel, vector_grid(p.tokens * (p.k / 8)), dim3(256), 0, stream, p,
                       (const PackedRow*)about, (const int32_t*)places, (const float*)sums,
                       (const CrossEntropyPlan*)plan, s.tall, grad_x);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace trace_host
