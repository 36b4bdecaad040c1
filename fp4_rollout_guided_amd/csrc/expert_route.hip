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
// lanes.  Lane l holds experts l, l + 16, ... (loads of neighbouring lanes are
// neighbours, whatever the row's alignment).  The topk rounds each find
// the largest key and then, among the lanes that hold it, the lowest index.
// Probabilities are summed per lane, then in the order of the waves and of the
// workgroups (fp64), counts by integer atomics in LDS: no result depends on the
// order of atomics.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"
#include "launch.h"
#include "launch_step.h"

namespace trace_dev {

using trace_host::RouteArgs;

constexpr uint32_t kRouteThreads = 1024;
constexpr uint32_t kRouteWaves = kRouteThreads / 64;
constexpr uint32_t kRouteBlocks = 256;  // at most: one to a compute unit

// A logit's place among all floats; NaN above all, 0 below all.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z);
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

// Lane l's logits of a row: experts l + kLanes j; -infinity past the last one.
template <bool kBf16, int kLanes, int kPer>
__device__ __forceinline__ void load_logits(const void* logits, uint64_t row, uint32_t experts, uint32_t l,
                                            float (&z)[kPer]) {
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint32_t e = l + kLanes * j;
    z[j] = -__builtin_inff();
    if (e < experts) {
      if (kBf16)
        z[j] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[row * experts + e] << 16);
      else
        z[j] = static_cast<const float*>(logits)[row * experts + e];
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
    if (e <= experts) {
#pragma unroll 8
      for (uint32_t b = share; b < blocks; b += wide) {
        count += part_counts[(uint64_t)b * (experts + 1) + e];
        if (e < experts) probs += part_probs[(uint64_t)b * experts + e];
      }
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

template <bool kBf16, int kLanes, int kPer>
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
    load_logits<kBf16, kLanes, kPer>(p.logits, from, p.experts, l, z);
    const bool wanted = there && (!valid || valid[from] != 0);
    uint32_t key[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) key[j] = l + kLanes * j < p.experts ? order_key(z[j]) : 0u;
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
      for (int i = kPer - 1; i >= 0; --i) at = key[i] == best ? l + kLanes * i : at;
      at = row_min<kLanes>(at);
      const bool found = best > kKeyOfMinusInfinity && wanted;
      float e = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const bool here = at == l + kLanes * i;
        e = here ? z[i] : e;
        key[i] = here ? 0u : key[i];
      }
      // the chosen exponential is in one lane: the others add zeros
      e = found ? e : 0.f;
      e = row_sum<kLanes>(at % kLanes == l ? e : 0.f);
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
    if (lane < kLanes) sums[wave][l + kLanes * j] = probs[j];
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
template <bool kBf16, int kLanes, int kPer>
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
      const uint32_t e = l + kLanes * j;
      if (e < p.experts) pairs += (double)counts[e];
    }
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) pairs += __shfl_xor(pairs, d);
    const double rows = (double)counts[p.experts];
    const double each = pairs > 0 && rows > 0 ? (double)*grad_balance * p.experts / (pairs * rows) : 0.0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t e = l + kLanes * j;
      if (e < p.experts) c[j] = (float)(each * (double)counts[e]);
    }
  }
  const uint64_t step = (uint64_t)gridDim.x * 4 * kRows;
  for (uint64_t row0 = ((uint64_t)blockIdx.x * 4 + wave) * kRows; row0 < p.tokens; row0 += step) {
    const uint64_t row = row0 + lane / kLanes;
    const bool there = row < p.tokens;
    const uint64_t from = there ? row : p.tokens - 1;
    float z[kPer], dz[kPer];
    load_logits<kBf16, kLanes, kPer>(p.logits, from, p.experts, l, z);
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
      // pairs kLanes at a time, one to a lane; their products' sum first
      float s = 0.f;
      for (uint32_t j = l; j < p.topk; j += kLanes)
        if (ids[from * p.topk + j] >= 0) s += weights[from * p.topk + j] * grad_weights[from * p.topk + j];
      s = row_sum<kLanes>(s);
#pragma unroll
      for (int i = 0; i < kPer; ++i) dz[i] -= p.renormalize ? 0.f : z[i] * s;
      for (uint32_t j = 0; j < p.topk; ++j) {
        const int64_t id = ids[from * p.topk + j];
        if (id < 0) continue;
        const float w = weights[from * p.topk + j], g = grad_weights[from * p.topk + j];
        const float d = w * (p.renormalize ? g - s : g);
#pragma unroll
        for (int i = 0; i < kPer; ++i) dz[i] += id == (int64_t)(l + kLanes * i) ? d : 0.f;
      }
    }
    if (!there) continue;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t e = l + kLanes * j;
      if (e >= p.experts) continue;
      const float v = wanted ? dz[j] : 0.f;
      if (kBf16) {
        const __bf16 h = (__bf16)v;
        __builtin_memcpy(static_cast<uint16_t*>(grad_logits) + row * p.experts + e, &h, 2);
      } else {
        static_cast<float*>(grad_logits)[row * p.experts + e] = v;
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

template <bool kBf16, class Run>
void by_experts(uint32_t experts, const Run& run) {
  if (experts <= 64)
    run(std::integral_constant<int, 16>(), std::integral_constant<int, 4>());
  else if (experts <= 128)
    run(std::integral_constant<int, 16>(), std::integral_constant<int, 8>());
  else if (experts <= 256)
    run(std::integral_constant<int, 16>(), std::integral_constant<int, 16>());
  else if (experts <= 512)
    run(std::integral_constant<int, 64>(), std::integral_constant<int, 8>());
  else
    run(std::integral_constant<int, 64>(), std::integral_constant<int, 16>());
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
    const auto run = [&](auto bf16) {
      constexpr bool kB = decltype(bf16)::value;
      by_experts<kB>(p.experts, [&](auto lanes, auto per) {
        hipLaunchKernelGGL((expert_route_kernel<kB, decltype(lanes)::value, decltype(per)::value>), dim3(blocks),
                           dim3(kRouteThreads), 0, stream, p, valid, ids, weights, part_counts, part_probs, out);
      });
    };
    if (p.bf16)
      run(std::true_type());
    else
      run(std::false_type());
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
  const auto run = [&](auto bf16) {
    constexpr bool kB = decltype(bf16)::value;
    by_experts<kB>(p.experts, [&](auto lanes, auto per) {
      hipLaunchKernelGGL((expert_route_bwd_kernel<kB, decltype(lanes)::value, decltype(per)::value>), dim3(grid),
                         dim3(256), 0, stream, p, grad_weights, grad_balance, ids, weights, counts, grad_logits);
    });
  };
  if (p.bf16)
    run(std::true_type());
  else
    run(std::false_type());
  return hipGetLastError();
}

}  // namespace trace_host
