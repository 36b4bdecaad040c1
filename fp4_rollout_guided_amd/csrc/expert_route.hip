// libtrace router for gfx950: the experts and weights that expert_sort and
// expert_combine take, the experts' counts and the balance loss, and the
// gradient to the router's logits.
//
//   p[t] = softmax(z[t]);  ids[t] = the topk largest z[t], the lowest index first among equals;
//   weights[t, j] = p[t, ids[t, j]], renormalised over j where asked;
//   counts[e] = pairs with expert e,  counts[experts] = rows routed = N,  probs[e] = sum over t of p[t, e],
//   balance = experts * sum over e of (counts[e] / sum of counts) * (probs[e] / N).
//
// A row of up to 256 experts is held by 16 lanes, so that a wave routes four
// rows and a maximum takes four DPP moves; more experts take the wave's 64
// lanes.  Lanes hold 16 bytes of neighbouring experts at a time, or, where rows are
// not whole vectors, single ones.  The topk rounds each find the largest key and
// then, among the lanes that hold it, the lowest index; lane j keeps round j's, and
// makes its exponential from the key again.
// Probabilities are summed per lane, then in the order of the waves and of the
// workgroups (fp64), counts by integer atomics in LDS: no result depends on the
// order of atomics.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_math.h"
#include "fp4_block.h"
#include "launch.h"
#include "launch_step.h"

namespace trace_dev {

using trace_host::RouteArgs;

constexpr uint32_t kRouteThreads = 1024;
constexpr uint32_t kRouteWaves = kRouteThreads / 64;
constexpr uint32_t kRouteBlocks = 256;  // at most: one to a compute unit

// A logit's place among all floats, the two zeros in one; NaN above all, 0 below all.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  if (z != z) return 0xffffffffu;
  return (int32_t)b < 0 ? ~b : b | 0x80000000u;
}
template <bool kBf16>  // a key's low half may say something else then
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(((int32_t)key < 0 ? key ^ 0x80000000u : ~key) & (kBf16 ? 0xffff0000u : 0xffffffffu));
}
constexpr uint32_t kKeyOfMinusInfinity = 0x007fffffu;

// exp(d), d <= 0: 2^(d log2 e), with what the product's rounding left out (and log2 e
// beyond 24 bits) put back: off by some 2^-23 of itself.  Below -150 it is zero; NaN stays.
__device__ __forceinline__ float exp_of(float d) {
  constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596303e-8f, kLn2 = 0.693147181f;
  d = d < -150.f ? -150.f : d;
  const float t = d * kLog2e;
  const float rest = fmaf(d, kLog2eRest, fmaf(d, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e * kLn2, rest, e);
}

// Reductions over the lanes that hold a row: 16 neighbours, or the wave.
template <int kLanes, class Op>
__device__ __forceinline__ uint32_t over_row(uint32_t v, Op op) {
  v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));   // lanes 1 0 3 2
  v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true));   // lanes 2 3 0 1
  v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true));  // eight lanes mirrored
  v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, true));  // sixteen lanes mirrored
  if (kLanes == 64) {
    v = op(v, (uint32_t)__shfl_xor((int)v, 16));
    v = op(v, (uint32_t)__shfl_xor((int)v, 32));
  }
  return v;
}
template <int kLanes>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  return over_row<kLanes>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int kLanes>
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  return over_row<kLanes>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int kLanes>
__device__ __forceinline__ float row_max(float v) {
  return __uint_as_float(over_row<kLanes>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
  return __uint_as_float(over_row<kLanes>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// Expert i of lane l: kVec neighbours at a time, the lanes' side by side.
template <int kLanes, int kVec>
__device__ __forceinline__ uint32_t expert_of(uint32_t l, int i) {
  return kVec * l + kLanes * kVec * (i / kVec) + i % kVec;
}

// Lane l's logits of a row, -infinity past the last one.  kVec > 1: experts is a
// multiple of it and rows are aligned to kVec logits.
template <bool kBf16, int kLanes, int kPer, int kVec>
__device__ __forceinline__ void load_logits(const void* logits, uint64_t row, uint32_t experts, uint32_t l,
                                            float (&z)[kPer]) {
  constexpr int kDwords = kBf16 ? (kVec + 1) / 2 : kVec;
#pragma unroll
  for (int i = 0; i < kPer; i += kVec) {
    const uint32_t e = expert_of<kLanes, kVec>(l, i);
    const bool in = e < experts;
    const uint64_t at = row * experts + (in ? e : 0);
    if constexpr (kVec == 1) {
      float v;
      if constexpr (kBf16)
        v = __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[at] << 16);
      else
        v = static_cast<const float*>(logits)[at];
      z[i] = in ? v : -__builtin_inff();
    } else {
      uint32_t d[kDwords];
      __builtin_memcpy(d, __builtin_assume_aligned(static_cast<const char*>(logits) + at * (kBf16 ? 2 : 4), 4 * kDwords),
                       4 * kDwords);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float v = kBf16 ? ((j & 1) ? bf16_hi(d[j / 2]) : bf16_lo(d[j / 2])) : __uint_as_float(d[j]);
        z[i + j] = in ? v : -__builtin_inff();
      }
    }
  }
}

// exp(z - top) and their sum; NaN and +infinity make NaNs of the row.
template <int kLanes, int kPer>
__device__ __forceinline__ float row_softmax(float (&z)[kPer], float& top) {
  top = z[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) top = fmaxf(top, z[j]);
  top = row_max<kLanes>(top);
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    z[j] = exp_of(z[j] - top);
    sum += z[j];
  }
  return row_sum<kLanes>(sum);
}

// The sums over all workgroups.
struct RouteTotals {
  int64_t* counts;
  float* probs;
  float* balance;
};
struct RouteLine {  // of a part of the experts: sum of counts * probs, sum of counts, rows routed
  double weighted, pairs, rows;
};
__device__ __forceinline__ float balance_of(uint32_t experts, const RouteLine& all) {
  return all.pairs > 0 ? (float)(experts * all.weighted / (all.pairs * all.rows)) : 0.f;
}
__device__ __forceinline__ RouteLine over_wave(RouteLine v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    v.weighted += __shfl_xor(v.weighted, d);
    v.pairs += __shfl_xor(v.pairs, d);
    v.rows += __shfl_xor(v.rows, d);
  }
  return v;
}

// The workgroups' sums, 16 experts (the rows routed among them) to a workgroup of
// 16 x 16 lanes, whose loads are all under way at once: their latency is all that
// this takes.  The last workgroup to be done joins the others' lines.
constexpr uint32_t kFinishExperts = 16;
constexpr uint32_t kFinishMost = trace_host::kMaxRouted / kFinishExperts + 1;  // workgroups
struct RouteParts {
  RouteLine* lines;  // [kFinishMost]
  uint32_t* done;    // workgroups; zero before
  uint32_t* counts;  // [blocks][experts + 1]
  float* probs;      // [blocks][experts]
};
__global__ __launch_bounds__(256) void expert_route_finish_kernel(RouteParts part, uint32_t blocks, uint32_t experts,
                                                                  RouteTotals out) {
  constexpr uint32_t kShares = 256 / kFinishExperts, kAtOnce = kRouteBlocks / kShares;
  __shared__ double probs_of[256];
  __shared__ double count_of[256];
  __shared__ bool last;
  const uint32_t e = blockIdx.x * kFinishExperts + threadIdx.x % kFinishExperts, share = threadIdx.x / kFinishExperts;
  const uint32_t ec = e <= experts ? e : experts, ep = e < experts ? e : experts - 1;
  uint32_t c[kAtOnce];
  float f[kAtOnce];
#pragma unroll
  for (uint32_t i = 0; i < kAtOnce; ++i) {
    const uint32_t b = share + i * kShares < blocks ? share + i * kShares : blocks - 1;
    c[i] = part.counts[b * (experts + 1) + ec];
    f[i] = part.probs[b * experts + ep];
  }
  double probs = 0, count = 0;
#pragma unroll
  for (uint32_t i = 0; i < kAtOnce; ++i)
    if (share + i * kShares < blocks) count += c[i], probs += f[i];
  probs_of[threadIdx.x] = probs;
  count_of[threadIdx.x] = count;
  __syncthreads();
  if (threadIdx.x < 64) {
    RouteLine line{0, 0, 0};
    if (share == 0 && e <= experts) {
#pragma unroll
      for (uint32_t i = 1; i < kShares; ++i) {
        probs += probs_of[threadIdx.x + i * kFinishExperts];
        count += count_of[threadIdx.x + i * kFinishExperts];
      }
      out.counts[e] = (int64_t)count;
      if (e < experts) {
        out.probs[e] = (float)probs;
        line = RouteLine{count * probs, count, 0};
      } else {
        line.rows = count;
      }
    }
    line = over_wave(line);
    if (threadIdx.x == 0) {
      RouteLine* const to = part.lines + blockIdx.x;
      __hip_atomic_store(&to->weighted, line.weighted, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&to->pairs, line.pairs, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&to->rows, line.rows, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(part.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (last && threadIdx.x < 64) {
    RouteLine all{0, 0, 0};
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += 64) {
      all.weighted += __hip_atomic_load(&part.lines[i].weighted, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      all.pairs += __hip_atomic_load(&part.lines[i].pairs, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      all.rows += __hip_atomic_load(&part.lines[i].rows, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    all = over_wave(all);
    if (threadIdx.x == 0) *out.balance = balance_of(experts, all);
  }
}

// What is compared of expert e's logit: larger first, then the lower index.  A logit
// of 16 bits has room for the index beside it, and each key is there once; one of 32
// bits is a key alone, and the lowest index is looked for among the largest.
template <bool kBf16>
__device__ __forceinline__ uint32_t rank_key(float z, uint32_t e) {
  const uint32_t key = order_key(z);
  return kBf16 ? (key & 0xffff0000u) | (0xffffu - e) : key;
}

// Bound by the arithmetic of the rounds: 16384 rows of 128 in fp32, eight to a row, 9.5
// us (a copy of them takes 2), and the totals 5; 65573 rows of 256 in bf16, six to a row, 32 us
// together.  24 rows of 128: 6.6 us, the latencies of one workgroup.
template <bool kBf16, int kLanes, int kPer, int kVec>
__global__ __launch_bounds__(kRouteThreads) void expert_route_kernel(RouteArgs p, const uint8_t* __restrict__ valid,
                                                                     int64_t* __restrict__ ids,
                                                                     float* __restrict__ weights, RouteParts part,
                                                                     RouteTotals out) {
  constexpr uint32_t kRows = 64 / kLanes, kMost = kLanes * kPer;  // of a wave; experts
  __shared__ uint32_t hist[kMost + 1];
  __shared__ float sums[kRouteWaves][kMost];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % kLanes;
  for (uint32_t e = threadIdx.x; e <= p.experts; e += kRouteThreads) hist[e] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0 && gridDim.x > 1) *part.done = 0;
  __syncthreads();
  float probs[kPer] = {};
  const uint64_t step = (uint64_t)gridDim.x * kRouteWaves * kRows;
  for (uint64_t row0 = ((uint64_t)blockIdx.x * kRouteWaves + wave) * kRows; row0 < p.tokens; row0 += step) {
    const uint64_t row = row0 + lane / kLanes;
    const bool there = row < p.tokens;
    const uint64_t from = there ? row : p.tokens - 1;
    float z[kPer];
    load_logits<kBf16, kLanes, kPer, kVec>(p.logits, from, p.experts, l, z);
    const bool wanted = there && (!valid || valid[from] != 0);
    uint32_t key[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t e = expert_of<kLanes, kVec>(l, j);
      key[j] = e < p.experts ? rank_key<kBf16>(z[j], e) : 0u;
    }
    float top;
    const float sum = row_softmax<kLanes, kPer>(z, top);
    // lane l keeps the pairs l, l + kLanes, ... until all are known
    constexpr uint32_t kKept = (trace_host::kMaxRouted < 64 ? trace_host::kMaxRouted : 64) / kLanes;
    int32_t kept_id[kKept];
    float kept_e[kKept], chosen = 0.f;
    bool some = false;
#pragma unroll
    for (uint32_t k = 0; k < kKept; ++k) {
      kept_id[k] = -1;
      uint32_t kept_key = 0;
      const uint32_t end = p.topk > kLanes * k ? (p.topk - kLanes * k < kLanes ? p.topk - kLanes * k : kLanes) : 0;
      for (uint32_t j = 0; j < end; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < kPer; ++i) best = key[i] > best ? key[i] : best;
        best = row_max<kLanes>(best);
        uint32_t at;
        if constexpr (kBf16) {
          at = 0xffffu - (best & 0xffffu);
#pragma unroll
          for (int i = 0; i < kPer; ++i) key[i] = key[i] == best ? 0u : key[i];
          best &= 0xffff0000u;
        } else {
          uint32_t mine = 0xffffffffu;
#pragma unroll
          for (int i = kPer - 1; i >= 0; --i) mine = key[i] == best ? expert_of<kLanes, kVec>(l, i) : mine;
          at = row_min<kLanes>(mine);
#pragma unroll
          for (int i = 0; i < kPer; ++i) key[i] = at == expert_of<kLanes, kVec>(l, i) ? 0u : key[i];
        }
        const bool found = best > kKeyOfMinusInfinity && wanted;
        some |= found;
        kept_id[k] = l == j && found ? (int32_t)at : kept_id[k];
        kept_key = l == j ? best : kept_key;
      }
      if (kept_id[k] >= 0) atomicAdd(&hist[kept_id[k]], 1u);
      kept_e[k] = kept_id[k] >= 0 ? exp_of(logit_of<kBf16>(kept_key) - top) : 0.f;
      chosen += kept_e[k];
    }
    const float by = p.renormalize ? row_sum<kLanes>(chosen) : sum;
    if (there) {
#pragma unroll
      for (uint32_t k = 0; k < kKept; ++k) {
        const uint32_t j = l + kLanes * k;
        if (j < p.topk) {
          ids[row * p.topk + j] = kept_id[k];
          weights[row * p.topk + j] = kept_id[k] >= 0 ? kept_e[k] / by : 0.f;
        }
      }
    }
    if (some) {
      const float each = 1.f / sum;
#pragma unroll
      for (int j = 0; j < kPer; ++j) probs[j] += z[j] * each;
      if (l == 0) atomicAdd(&hist[p.experts], 1u);
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (kLanes == 16) {
      probs[j] += __shfl_xor(probs[j], 16);
      probs[j] += __shfl_xor(probs[j], 32);
    }
    if (lane < kLanes) sums[wave][expert_of<kLanes, kVec>(l, j)] = probs[j];
  }
  __syncthreads();
  if (gridDim.x > 1) {
    for (uint32_t e = threadIdx.x; e <= p.experts; e += kRouteThreads) {
      part.counts[blockIdx.x * (p.experts + 1) + e] = hist[e];
      if (e < p.experts) {
        float v = sums[0][e];
#pragma unroll
        for (uint32_t w = 1; w < kRouteWaves; ++w) v += sums[w][e];
        part.probs[blockIdx.x * p.experts + e] = v;
      }
    }
    return;
  }
  // few rows: the only workgroup finishes by itself
  __shared__ RouteLine lines[kRouteWaves];
  RouteLine line{0, 0, 0};
  for (uint32_t e = threadIdx.x; e <= p.experts; e += kRouteThreads) {
    const uint32_t count = hist[e];
    out.counts[e] = count;
    if (e < p.experts) {
      float v = sums[0][e];
#pragma unroll
      for (uint32_t w = 1; w < kRouteWaves; ++w) v += sums[w][e];
      out.probs[e] = v;
      line.weighted += (double)count * v;
      line.pairs += count;
    } else {
      line.rows = count;
    }
  }
  line = over_wave(line);
  if (lane == 0) lines[wave] = line;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (uint32_t w = 1; w < kRouteWaves; ++w) {
      line.weighted += lines[w].weighted;
      line.pairs += lines[w].pairs;
      line.rows += lines[w].rows;
    }
    *out.balance = balance_of(p.experts, line);
  }
}

// The gradient to the logits.  With s = sum over j of weights[j] grad_weights[j],
//   renormalised: dz[ids[j]] += weights[j] (grad_weights[j] - s)   (the softmax of the chosen logits alone)
//   otherwise:    dz[e] -= p[e] s,  dz[ids[j]] += weights[j] grad_weights[j]
//   balance:      dz[e] += p[e] (c[e] - sum of p c),  c[e] = grad_balance experts counts[e] / (sum of counts * N).
// Rows whose ids are all negative get zeros.
// What the chosen experts add goes to their lanes by way of LDS, which is zero but
// there (each lane looking through its experts for each of them was a third of the
// arithmetic).  65573 rows of 256 in bf16, six to a row: 17 us, 4.2 TB/s, bound by
// arithmetic; 16384 rows of 128 in fp32: 6.6 us.
template <bool kBf16, int kLanes, int kPer, int kVec>
__global__ __launch_bounds__(256) void expert_route_bwd_kernel(RouteArgs p, const float* __restrict__ grad_weights,
                                                               const float* __restrict__ grad_balance,
                                                               const int64_t* __restrict__ ids,
                                                               const float* __restrict__ weights,
                                                               const int64_t* __restrict__ counts, void* grad_logits) {
  constexpr uint32_t kRows = 64 / kLanes, kMost = kLanes * kPer;
  __shared__ __attribute__((aligned(16))) float added[4 * kRows * kMost];
  __shared__ __attribute__((aligned(16))) float slopes[kMost];
  __shared__ double lines[4];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % kLanes;
  float* const to = added + (wave * kRows + lane / kLanes) * kMost;  // of this lane's row
  for (uint32_t i = threadIdx.x; i < 4 * kRows * kMost; i += 256) added[i] = 0.f;
  float c[kPer] = {};
  if (grad_balance) {
    double own[(kMost + 255) / 256], pairs = 0;
#pragma unroll
    for (uint32_t i = 0; i < (kMost + 255) / 256; ++i) {
      const uint32_t e = threadIdx.x + 256 * i;
      own[i] = e < p.experts ? (double)counts[e] : 0.0;
      pairs += own[i];
    }
    const double rows = (double)counts[p.experts];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) pairs += __shfl_xor(pairs, d);
    if (lane == 0) lines[wave] = pairs;
    __syncthreads();
    pairs = lines[0] + lines[1] + lines[2] + lines[3];
    const double each = pairs > 0 && rows > 0 ? (double)*grad_balance * p.experts / (pairs * rows) : 0.0;
#pragma unroll
    for (uint32_t i = 0; i < (kMost + 255) / 256; ++i)
      if (threadIdx.x + 256 * i < kMost) slopes[threadIdx.x + 256 * i] = (float)(each * own[i]);
  }
  __syncthreads();
  if (grad_balance) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) c[j] = slopes[expert_of<kLanes, kVec>(l, j)];
  }
  const uint64_t step = (uint64_t)gridDim.x * 4 * kRows;
  for (uint64_t row0 = ((uint64_t)blockIdx.x * 4 + wave) * kRows; row0 < p.tokens; row0 += step) {
    const uint64_t row = row0 + lane / kLanes;
    const bool there = row < p.tokens;
    const uint64_t from = there ? row : p.tokens - 1;
    // lane l holds pairs l, l + kLanes, ...
    constexpr uint32_t kKept = 64 / kLanes;
    int64_t id[kKept];
    float w[kKept], g[kKept];
    float z[kPer], dz[kPer], top;
    load_logits<kBf16, kLanes, kPer, kVec>(p.logits, from, p.experts, l, z);
    uint32_t some = 0;
#pragma unroll
    for (uint32_t i = 0; i < kKept; ++i) {
      const uint32_t j = l + kLanes * i;
      id[i] = -1, w[i] = 0.f, g[i] = 0.f;
      if (j < p.topk) {
        id[i] = ids[from * p.topk + j];
        if (grad_weights) {
          w[i] = weights[from * p.topk + j];
          g[i] = grad_weights[from * p.topk + j];
        }
      }
      some |= (uint32_t)(id[i] >= 0);
    }
    const bool wanted = row_max<kLanes>(some) != 0;  // whichever of its pairs stands
    const float each = 1.f / row_softmax<kLanes, kPer>(z, top);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      z[j] *= each;
      dot += z[j] * c[j];
    }
    dot = row_sum<kLanes>(dot);
    if (grad_weights) {
      float s = 0.f;
#pragma unroll
      for (uint32_t i = 0; i < kKept; ++i)
        if (id[i] >= 0) s += w[i] * g[i];
      s = row_sum<kLanes>(s);
      const auto to_chosen = [&](auto put) {
#pragma unroll
        for (uint32_t i = 0; i < kKept; ++i)
          if (l + kLanes * i < p.topk && id[i] >= 0 && id[i] < (int64_t)p.experts) put(to + id[i], i);
        // one wave's accesses of LDS are done in their order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      };
      to_chosen([&](float* at, uint32_t i) { unsafeAtomicAdd(at, w[i] * (p.renormalize ? g[i] - s : g[i])); });
      const float less = p.renormalize ? dot : dot + s;
#pragma unroll
      for (int i = 0; i < kPer; ++i) dz[i] = z[i] * (c[i] - less) + to[expert_of<kLanes, kVec>(l, i)];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      to_chosen([&](float* at, uint32_t) { *at = 0.f; });
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) dz[j] = z[j] * (c[j] - dot);
    }
    if (!there) continue;
#pragma unroll
    for (int i = 0; i < kPer; i += kVec) {
      const uint32_t e = expert_of<kLanes, kVec>(l, i);
      if (e >= p.experts) continue;
      const uint64_t at = row * p.experts + e;
      if constexpr (kVec == 1) {
        const float v = wanted ? dz[i] : 0.f;
        if constexpr (kBf16) {
          const __bf16 h = (__bf16)v;
          __builtin_memcpy(static_cast<uint16_t*>(grad_logits) + at, &h, 2);
        } else {
          static_cast<float*>(grad_logits)[at] = v;
        }
      } else {
        constexpr int kDwords = kBf16 ? kVec / 2 : kVec;
        uint32_t d[kDwords];
#pragma unroll
        for (int j = 0; j < kDwords; ++j) {
          if constexpr (kBf16) {
            const bf16x2 two = __builtin_convertvector(
                (f32x2){wanted ? dz[i + 2 * j] : 0.f, wanted ? dz[i + 2 * j + 1] : 0.f}, bf16x2);
            __builtin_memcpy(&d[j], &two, 4);
          } else {
            d[j] = __float_as_uint(wanted ? dz[i + j] : 0.f);
          }
        }
        __builtin_memcpy(__builtin_assume_aligned(static_cast<char*>(grad_logits) + at * (kBf16 ? 2 : 4), 4 * kDwords), d,
                         4 * kDwords);
      }
    }
  }
}

}  // namespace trace_dev

namespace trace_host {

using namespace trace_dev;

namespace {

uint32_t route_blocks(uint64_t tokens, uint32_t experts) {
  const uint64_t rows = kRouteWaves * (experts <= 256 ? 4u : 1u);  // of a workgroup's turn
  const uint64_t blocks = (tokens + rows - 1) / rows;
  const uint64_t most = kRouteBlocks < kMaxGroups ? kRouteBlocks : kMaxGroups;
  return (uint32_t)(blocks < 1 ? 1 : (blocks < most ? blocks : most));
}

// Kernels by the number of experts, and vectors of 16 bytes (8 bytes for up to 64
// experts in bf16) where rows are whole ones: the gradients of 65573 rows of 256 in
// bf16 take 22.7 us one by one and 20.3 so.
template <bool kBf16, int kLanes, int kPer, class Run>
void by_vectors(bool vectors, const Run& run) {
  constexpr int kVec = kBf16 && kPer >= 8 ? 8 : 4;
  constexpr std::integral_constant<bool, kBf16> bf16;
  constexpr std::integral_constant<int, kLanes> lanes;
  constexpr std::integral_constant<int, kPer> per;
  if (vectors)
    run(bf16, lanes, per, std::integral_constant<int, kVec>());
  else
    run(bf16, lanes, per, std::integral_constant<int, 1>());
}
template <bool kBf16, class Run>
void by_experts(uint32_t experts, uintptr_t where, const Run& run) {
  const uint32_t vec = kBf16 && experts > 64 ? 8 : 4;
  const bool vectors = experts % vec == 0 && where % (vec * (kBf16 ? 2 : 4)) == 0;
  if (experts <= 64)
    by_vectors<kBf16, 16, 4>(vectors, run);
  else if (experts <= 128)
    by_vectors<kBf16, 16, 8>(vectors, run);
  else if (experts <= 256)
    by_vectors<kBf16, 16, 16>(vectors, run);
  else if (experts <= 512)
    by_vectors<kBf16, 64, 8>(vectors, run);
  else
    by_vectors<kBf16, 64, 16>(vectors, run);
}
template <class Run>
void by_kind(const RouteArgs& p, uintptr_t where, const Run& run) {
  if (p.bf16)
    by_experts<true>(p.experts, where, run);
  else
    by_experts<false>(p.experts, where, run);
}

}  // namespace

uint64_t route_workspace_bytes(uint64_t tokens, uint32_t experts) {
  return kFinishMost * sizeof(RouteLine) + 16 + (uint64_t)route_blocks(tokens, experts) * (2 * experts + 1) * 4;
}

hipError_t launch_route(const RouteArgs& p, const uint8_t* valid, void* workspace, int64_t* ids, float* weights,
                        int64_t* counts, float* probs, float* balance, hipStream_t stream) {
  const uint32_t blocks = route_blocks(p.tokens, p.experts);
  RouteParts part;
  part.lines = static_cast<RouteLine*>(workspace);
  part.done = reinterpret_cast<uint32_t*>(part.lines + kFinishMost);
  part.counts = part.done + 4;
  part.probs = reinterpret_cast<float*>(part.counts + (uint64_t)blocks * (p.experts + 1));
  const RouteTotals out{counts, probs, balance};
  by_kind(p, (uintptr_t)p.logits, [&](auto bf16, auto lanes, auto per, auto vec) {
    hipLaunchKernelGGL((expert_route_kernel<decltype(bf16)::value, decltype(lanes)::value, decltype(per)::value,
                                            decltype(vec)::value>),
                       dim3(blocks), dim3(kRouteThreads), 0, stream, p, valid, ids, weights, part, out);
  });
  if (hipError_t e = hipGetLastError()) return e;
  if (blocks == 1) return hipSuccess;
  hipLaunchKernelGGL(expert_route_finish_kernel, dim3(p.experts / kFinishExperts + 1), dim3(256), 0, stream, part, blocks,
                     p.experts, out);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteArgs& p, const float* grad_weights, const float* grad_balance,
                            const int64_t* ids, const float* weights, const int64_t* counts, void* grad_logits,
                            hipStream_t stream) {
  const uint64_t rows = 4 * (p.experts <= 256 ? 4u : 1u);
  const uint64_t blocks = (p.tokens + rows - 1) / rows;
  const uint64_t most = 2048 < kMaxGroups ? 2048 : kMaxGroups;
  const uint32_t grid = (uint32_t)(blocks < most ? blocks : most);
  by_kind(p, (uintptr_t)p.logits | (uintptr_t)grad_logits, [&](auto bf16, auto lanes, auto per, auto vec) {
    hipLaunchKernelGGL((expert_route_bwd_kernel<decltype(bf16)::value, decltype(lanes)::value, decltype(per)::value,
                                                decltype(vec)::value>),
                       dim3(grid), dim3(256), 0, stream, p, grad_weights, grad_balance, ids, weights, counts, grad_logits);
  });
  return hipGetLastError();
}

}  // namespace trace_host
