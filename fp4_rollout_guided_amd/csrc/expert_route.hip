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
// not whole vectors, single ones.  The topk rounds each find
// the largest key and then, among the lanes that hold it, the lowest index.
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
constexpr uint32_t kKeyOfMinusInfinity = 0x007fffffu;

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

// exp(z - top) and their sum's reciprocal's operand; NaN and +infinity make NaNs of the row.
template <int kLanes, int kPer>
__device__ __forceinline__ float row_softmax(float (&z)[kPer]) {
  float top = z[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) top = fmaxf(top, z[j]);
  top = row_max<kLanes>(top);
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    z[j] = expf(z[j] - top);
    sum += z[j];
  }
  return row_sum<kLanes>(sum);
}

// The sums over all workgroups, by one workgroup.
struct RouteTotals {
  int64_t* counts;
  float* probs;
  float* balance;
};
__device__ __forceinline__ void finish_route(const uint32_t* part_counts, const float* part_probs, uint32_t blocks,
                                             uint32_t experts, const RouteTotals& out) {
  // part_counts: [blocks][experts + 1], part_probs: [blocks][experts]
  __shared__ double probs_of[kRouteThreads];
  __shared__ double pairs_of[kRouteThreads];
  __shared__ double lines[kRouteWaves][3];
  uint32_t wide = 1;  // lanes to an expert: a power of two
  while (wide * 2 * (experts + 1) <= kRouteThreads) wide *= 2;
  const uint32_t per = kRouteThreads / wide;  // experts at a time, the rows routed among them
  double weighted = 0, pairs = 0;
  for (uint32_t e0 = 0; e0 <= experts; e0 += per) {
    const uint32_t e = e0 + threadIdx.x % per, share = threadIdx.x / per;
    double probs = 0, count = 0;
    constexpr uint32_t kAtOnce = 16;  // loads under way: their latency is all that this takes
    const uint32_t ec = e <= experts ? e : experts, ep = e < experts ? e : experts - 1;
    for (uint32_t b0 = share; b0 < blocks; b0 += wide * kAtOnce) {
      uint32_t c[kAtOnce];
      float f[kAtOnce];
#pragma unroll
      for (uint32_t i = 0; i < kAtOnce; ++i) {
        const uint32_t b = b0 + i * wide < blocks ? b0 + i * wide : blocks - 1;
        c[i] = part_counts[b * (experts + 1) + ec];
        f[i] = part_probs[b * experts + ep];
      }
#pragma unroll
      for (uint32_t i = 0; i < kAtOnce; ++i)
        if (b0 + i * wide < blocks) count += c[i], probs += f[i];
    }
    __syncthreads();
    probs_of[threadIdx.x] = probs;
    pairs_of[threadIdx.x] = count;
    __syncthreads();
    if (share == 0 && e <= experts) {
      for (uint32_t i = 1; i < wide; ++i) {
        probs += probs_of[threadIdx.x + i * per];
        count += pairs_of[threadIdx.x + i * per];
      }
      out.counts[e] = (int64_t)count;
      if (e < experts) {
        out.probs[e] = (float)probs;
        weighted += count * probs;
        pairs += count;
      } else {
        lines[0][2] = count;
      }
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    weighted += __shfl_xor(weighted, d);
    pairs += __shfl_xor(pairs, d);
  }
  const uint32_t wave = threadIdx.x / 64;
  if (threadIdx.x % 64 == 0) {
    lines[wave][0] = weighted;
    lines[wave][1] = pairs;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (uint32_t w = 1; w < kRouteWaves; ++w) weighted += lines[w][0], pairs += lines[w][1];
    const double rows = lines[0][2];
    *out.balance = pairs > 0 ? (float)(experts * weighted / (pairs * rows)) : 0.f;
  }
}

template <bool kBf16, int kLanes, int kPer, int kVec>
__global__ __launch_bounds__(kRouteThreads) void expert_route_kernel(RouteArgs p, const uint8_t* __restrict__ valid,
                                                                     int64_t* __restrict__ ids,
                                                                     float* __restrict__ weights, uint32_t* part_counts,
                                                                     float* part_probs, RouteTotals out) {
  constexpr uint32_t kRows = 64 / kLanes, kMost = kLanes * kPer;  // of a wave; experts
  __shared__ uint32_t hist[kMost + 1];
  __shared__ float sums[kRouteWaves][kMost];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % kLanes;
  for (uint32_t e = threadIdx.x; e <= p.experts; e += kRouteThreads) hist[e] = 0;
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
    for (int j = 0; j < kPer; ++j) key[j] = expert_of<kLanes, kVec>(l, j) < p.experts ? order_key(z[j]) : 0u;
    const float sum = row_softmax<kLanes, kPer>(z);
    // lane l keeps the pairs l, l + kLanes, ... until all are known
    constexpr uint32_t kKept = (trace_host::kMaxRouted < 64 ? trace_host::kMaxRouted : 64) / kLanes;
    int32_t kept_id[kKept];
    float kept_e[kKept], chosen = 0.f;
    bool some = false;
#pragma unroll
    for (uint32_t i = 0; i < kKept; ++i) kept_id[i] = -1, kept_e[i] = 0.f;
    for (uint32_t j = 0; j < p.topk; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) best = key[i] > best ? key[i] : best;
      best = row_max<kLanes>(best);
      uint32_t at = 0xffffffffu;
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i) at = key[i] == best ? expert_of<kLanes, kVec>(l, i) : at;
      at = row_min<kLanes>(at);
      const bool found = best > kKeyOfMinusInfinity && wanted;
      float e = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const bool here = at == expert_of<kLanes, kVec>(l, i);
        e = here ? z[i] : e;
        key[i] = here ? 0u : key[i];
      }
      // the chosen exponential is in one lane: the others add zeros
      e = found ? e : 0.f;
      e = row_sum<kLanes>(e);
      chosen += e;
      some |= found;
#pragma unroll
      for (uint32_t i = 0; i < kKept; ++i) {
        const bool mine = j == l + kLanes * i;
        kept_id[i] = mine && found ? (int32_t)at : kept_id[i];
        kept_e[i] = mine && found ? e : kept_e[i];
      }
      if (l == 0 && found) atomicAdd(&hist[at], 1u);
    }
    const float by = p.renormalize ? chosen : sum;
    if (there) {
#pragma unroll
      for (uint32_t i = 0; i < kKept; ++i) {
        const uint32_t j = l + kLanes * i;
        if (j < p.topk) {
          ids[row * p.topk + j] = kept_id[i];
          weights[row * p.topk + j] = kept_id[i] >= 0 ? kept_e[i] / by : 0.f;
        }
      }
    }
    if (some) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) probs[j] += z[j] / sum;
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
  part_counts += (uint64_t)blockIdx.x * (p.experts + 1);
  part_probs += (uint64_t)blockIdx.x * p.experts;
  for (uint32_t e = threadIdx.x; e <= p.experts; e += kRouteThreads) {
    part_counts[e] = hist[e];
    if (e < p.experts) {
      float v = sums[0][e];
      for (uint32_t w = 1; w < kRouteWaves; ++w) v += sums[w][e];
      part_probs[e] = v;
    }
  }
  if (gridDim.x == 1) {  // few rows: the only workgroup finishes by itself
    __threadfence_block();
    __syncthreads();
    finish_route(part_counts, part_probs, 1, p.experts, out);
  }
}

__global__ __launch_bounds__(kRouteThreads) void expert_route_finish_kernel(const uint32_t* part_counts,
                                                                            const float* part_probs, uint32_t blocks,
                                                                            uint32_t experts, RouteTotals out) {
  finish_route(part_counts, part_probs, blocks, experts, out);
}

// The gradient to the logits.  With s = sum over j of weights[j] grad_weights[j],
//   renormalised: dz[ids[j]] += weights[j] (grad_weights[j] - s)   (the softmax of the chosen logits alone)
//   otherwise:    dz[e] -= p[e] s,  dz[ids[j]] += weights[j] grad_weights[j]
//   balance:      dz[e] += p[e] (c[e] - sum of p c),  c[e] = grad_balance experts counts[e] / (sum of counts * N).
// Rows without an expert (ids[t, 0] < 0) get zeros.
template <bool kBf16, int kLanes, int kPer, int kVec>
__global__ __launch_bounds__(256) void expert_route_bwd_kernel(RouteArgs p, const float* __restrict__ grad_weights,
                                                               const float* __restrict__ grad_balance,
                                                               const int64_t* __restrict__ ids,
                                                               const float* __restrict__ weights,
                                                               const int64_t* __restrict__ counts, void* grad_logits) {
  constexpr uint32_t kRows = 64 / kLanes;
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % kLanes;
  float c[kPer] = {};
  if (grad_balance) {
    double pairs = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t e = expert_of<kLanes, kVec>(l, j);
      if (e < p.experts) pairs += (double)counts[e];
    }
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) pairs += __shfl_xor(pairs, d);
    const double rows = (double)counts[p.experts];
    const double each = pairs > 0 && rows > 0 ? (double)*grad_balance * p.experts / (pairs * rows) : 0.0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t e = expert_of<kLanes, kVec>(l, j);
      if (e < p.experts) c[j] = (float)(each * (double)counts[e]);
    }
  }
  const uint64_t step = (uint64_t)gridDim.x * 4 * kRows;
  for (uint64_t row0 = ((uint64_t)blockIdx.x * 4 + wave) * kRows; row0 < p.tokens; row0 += step) {
    const uint64_t row = row0 + lane / kLanes;
    const bool there = row < p.tokens;
    const uint64_t from = there ? row : p.tokens - 1;
    float z[kPer], dz[kPer];
    load_logits<kBf16, kLanes, kPer, kVec>(p.logits, from, p.experts, l, z);
    const bool wanted = ids[from * p.topk] >= 0;
    const float sum = row_softmax<kLanes, kPer>(z);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      z[j] /= sum;
      dot += z[j] * c[j];
    }
    dot = row_sum<kLanes>(dot);
#pragma unroll
    for (int j = 0; j < kPer; ++j) dz[j] = z[j] * (c[j] - dot);
    if (grad_weights) {
      // lane l holds pairs l, l + kLanes, ..., loaded at once
      constexpr uint32_t kKept = 64 / kLanes;
      int32_t id[kKept];
      float w[kKept], g[kKept], s = 0.f;
#pragma unroll
      for (uint32_t i = 0; i < kKept; ++i) {
        const uint32_t j = l + kLanes * i;
        id[i] = -1, w[i] = 0.f, g[i] = 0.f;
        if (j < p.topk) {
          id[i] = (int32_t)ids[from * p.topk + j];
          w[i] = weights[from * p.topk + j];
          g[i] = grad_weights[from * p.topk + j];
        }
        if (id[i] >= 0) s += w[i] * g[i];
      }
      s = row_sum<kLanes>(s);
#pragma unroll
      for (uint32_t i = 0; i < kKept; ++i) w[i] *= p.renormalize ? g[i] - s : g[i];
#pragma unroll
      for (int i = 0; i < kPer; ++i) dz[i] -= p.renormalize ? 0.f : z[i] * s;
#pragma unroll
      for (uint32_t k = 0; k < kKept; ++k) {
        const uint32_t end = p.topk > kLanes * k ? (p.topk - kLanes * k < kLanes ? p.topk - kLanes * k : kLanes) : 0;
        for (uint32_t j = 0; j < end; ++j) {
          const int32_t at = __shfl(id[k], (int)j, kLanes);
          const float d = __shfl(w[k], (int)j, kLanes);
#pragma unroll
          for (int i = 0; i < kPer; ++i) dz[i] += at == (int32_t)expert_of<kLanes, kVec>(l, i) ? d : 0.f;
        }
      }
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
  return (uint32_t)(blocks < most ? blocks : most);
}

// Kernels by the number of experts, and vectors of 16 bytes (8 bytes for up to 64
// experts in bf16) where rows are whole ones: 65573 rows of 256 in bf16, their
// gradients, 59 us one by one and 40 so.
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
  return (uint64_t)route_blocks(tokens, experts) * (2 * experts + 1) * 4;
}

hipError_t launch_route(const RouteArgs& p, const uint8_t* valid, void* workspace, int64_t* ids, float* weights,
                        int64_t* counts, float* probs, float* balance, hipStream_t stream) {
  const uint32_t blocks = route_blocks(p.tokens, p.experts);
  uint32_t* const part_counts = static_cast<uint32_t*>(workspace);
  float* const part_probs = reinterpret_cast<float*>(part_counts + (uint64_t)blocks * (p.experts + 1));
  const RouteTotals out{counts, probs, balance};
  if (blocks) {
    by_kind(p, (uintptr_t)p.logits, [&](auto bf16, auto lanes, auto per, auto vec) {
      hipLaunchKernelGGL((expert_route_kernel<decltype(bf16)::value, decltype(lanes)::value, decltype(per)::value,
                                              decltype(vec)::value>),
                         dim3(blocks), dim3(kRouteThreads), 0, stream, p, valid, ids, weights, part_counts, part_probs, out);
    });
    if (hipError_t e = hipGetLastError()) return e;
    if (blocks == 1) return hipSuccess;
  }
  hipLaunchKernelGGL(expert_route_finish_kernel, dim3(1), dim3(kRouteThreads), 0, stream, part_counts, part_probs,
                     blocks, p.experts, out);
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
