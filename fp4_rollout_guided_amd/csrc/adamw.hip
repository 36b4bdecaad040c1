// libtrace optimiser step for gfx950: AdamW over many tensors at once.
//
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2,
//   p <- p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// in fp32, every operation rounded by itself, in this order, so that any other
// program that does the same gets the same bits.
//
// States in 8 bits are MXFP8 records of m and of sqrt(v) (the root has half of
// v's range of exponents, and the step divides by it): E4M3 codes under one E8M0
// byte per 32 elements, the smallest power of two that leaves no element past
// 448.  Rounding to nearest would hold them still: with b2 = 0.999 a root moves
// by 0.05% a step at most downwards, and codes lie 6 to 12% apart.  They are
// rounded to either neighbour with the probability that keeps the mean, by random
// bits from the caller's seed and the element's place.  Parameters in bf16
// are rounded likewise where a seed is given, or to nearest.  It is the root whose mean is
// kept: v, its square, gains the roundings' variance on every step, and under steady
// gradients settles 5% above their mean square with b2 = 0.999, 4% with 0.99, 2.6% with 0.95
// (8192 elements simulated), which makes steps 1 to 2.5% shorter.
//
// Bound by memory: each element's bytes once in, once out, 16 bytes per lane of
// an fp32 tensor.  A workgroup owns 4096 consecutive elements of one tensor and
// loads all of them before the first arithmetic.  94 million elements with fp32 states
// and bf16 gradients and copies: 0.45 ms, 5.8 TB/s.  With 8-bit states and bf16 parameters the
// arithmetic counts (two records, random bits, exact root and quotient): 0.23 to 0.26 ms between
// cards, 4.2 to 3.7 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_math.h"
#include "fp4_block.h"
#include "launch.h"
#include "launch_step.h"

namespace trace_dev {

using trace_host::AdamwScalars;
using trace_host::AdamwTensor;
using trace_host::mix_bits;

constexpr uint32_t kAdamThreads = 256;
constexpr uint32_t kAdamChunk = 4096;
// A launch's tensors are kernel arguments, 4 KiB at most: without the addresses of
// scales a wave's lanes' number of them.
struct AdamwPlain {
  explicit AdamwPlain(const AdamwTensor& t) : param(t.param), grad(t.grad), avg(t.avg), sq(t.sq), copy(t.copy), n(t.n) {}
  AdamwPlain() = default;
  void* param;
  const void* grad;
  void* avg;
  void* sq;
  uint16_t* copy;
  uint64_t n;
  static constexpr uint8_t *avg_scales = nullptr, *sq_scales = nullptr;
};
template <bool kMx8>
struct AdamwBatch {
  static constexpr uint32_t kMost = kMx8 ? 48 : 64;
  using Tensor = std::conditional_t<kMx8, AdamwTensor, AdamwPlain>;
  Tensor t[kMost];
  uint64_t place[kMost];  // of its first element among all tensors' elements, each tensor filled up to 32
  uint32_t first[kMost];  // the tensor's first workgroup
  uint32_t count;
};
static_assert(sizeof(AdamwBatch<true>) + sizeof(AdamwScalars) + 16 <= 4096, "kernel arguments");
static_assert(sizeof(AdamwBatch<false>) + sizeof(AdamwScalars) + 16 <= 4096, "kernel arguments");

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// kPer consecutive elements of a tensor in fp32 or bf16, raw, at element i of
// `from`; kWhole: all of them exist, otherwise the first `left` do.
template <bool kBf16, bool kNT, int kPer>
struct Elements {
  static constexpr int kDwords = kBf16 ? kPer / 2 : kPer;
  uint32_t raw[kDwords];
  template <bool kWhole>
  __device__ __forceinline__ void load(const void* from, uint32_t i, uint32_t left) {
    if constexpr (kWhole) {
      if constexpr (kDwords == 2) {
        const u32x2* at = reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(from) + i);
        const u32x2 v = kNT ? __builtin_nontemporal_load(at) : *at;
        raw[0] = v[0], raw[1] = v[1];
      } else {
#pragma unroll
        for (int d = 0; d < kDwords; d += 4) {
          const uint4 v = load_vec<kNT>(
              reinterpret_cast<const uint4*>(static_cast<const char*>(from) + (uint64_t)i * (kBf16 ? 2 : 4)) + d / 4);
          raw[d] = v.x, raw[d + 1] = v.y, raw[d + 2] = v.z, raw[d + 3] = v.w;
        }
      }
    } else {
#pragma unroll
      for (int d = 0; d < kDwords; ++d) raw[d] = 0;
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j) {
        if (j >= left) continue;
        if constexpr (kBf16)
          raw[j >> 1] |= (uint32_t)static_cast<const uint16_t*>(from)[i + j] << (16 * (j & 1));
        else
          raw[j] = static_cast<const uint32_t*>(from)[i + j];
      }
    }
  }
  __device__ __forceinline__ void values(float (&v)[kPer]) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if constexpr (kBf16)
        v[j] = (j & 1) ? bf16_hi(raw[j >> 1]) : bf16_lo(raw[j >> 1]);
      else
        v[j] = __uint_as_float(raw[j]);
    }
  }
  template <bool kWhole>
  __device__ __forceinline__ void store(void* to, uint32_t i, uint32_t left) const {
    if constexpr (kWhole) {
      if constexpr (kDwords == 2) {
        u32x2* at = reinterpret_cast<u32x2*>(static_cast<uint16_t*>(to) + i);
        const u32x2 v = {raw[0], raw[1]};
        if (kNT)
          __builtin_nontemporal_store(v, at);
        else
          *at = v;
      } else {
#pragma unroll
        for (int d = 0; d < kDwords; d += 4)
          store_vec<kNT>(reinterpret_cast<uint4*>(static_cast<char*>(to) + (uint64_t)i * (kBf16 ? 2 : 4)) + d / 4,
                         make_uint4(raw[d], raw[d + 1], raw[d + 2], raw[d + 3]));
      }
    } else {
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j) {
        if (j >= left) continue;
        if constexpr (kBf16)
          static_cast<uint16_t*>(to)[i + j] = (uint16_t)(raw[j >> 1] >> (16 * (j & 1)));
        else
          static_cast<uint32_t*>(to)[i + j] = raw[j];
      }
    }
  }
};

// Eight code bytes likewise.
template <bool kWhole, bool kNT>
__device__ __forceinline__ u32x2 load_codes(const void* from, uint32_t i, uint32_t left) {
  u32x2 v = {0, 0};
  if constexpr (kWhole) {
    const u32x2* at = reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(from) + i);
    return kNT ? __builtin_nontemporal_load(at) : *at;
  }
#pragma unroll
  for (uint32_t j = 0; j < 8; ++j)
    if (j < left) v[j >> 2] |= (uint32_t)static_cast<const uint8_t*>(from)[i + j] << (8 * (j & 3));
  return v;
}
template <bool kWhole, bool kNT>
__device__ __forceinline__ void store_codes(void* to, uint32_t i, uint32_t left, u32x2 v) {
  if constexpr (kWhole) {
    u32x2* at = reinterpret_cast<u32x2*>(static_cast<uint8_t*>(to) + i);
    if (kNT)
      __builtin_nontemporal_store(v, at);
    else
      *at = v;
    return;
  }
#pragma unroll
  for (uint32_t j = 0; j < 8; ++j)
    if (j < left) static_cast<uint8_t*>(to)[i + j] = (uint8_t)(v[j >> 2] >> (8 * (j & 3)));
}

// 2^(b - 127), b in 0 .. 254, and NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : (b == 255 ? 0x7fc00000u : b << 23));
}

__device__ __forceinline__ void decode_codes(u32x2 c, uint32_t scale, float (&v)[8]) {
  const float s = e8m0_value(scale);
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    v[4 * d + 0] = __builtin_amdgcn_cvt_f32_fp8((int)c[d], 0) * s;
    v[4 * d + 1] = __builtin_amdgcn_cvt_f32_fp8((int)c[d], 1) * s;
    v[4 * d + 2] = __builtin_amdgcn_cvt_f32_fp8((int)c[d], 2) * s;
    v[4 * d + 3] = __builtin_amdgcn_cvt_f32_fp8((int)c[d], 3) * s;
  }
}

// The largest of the values of lanes 4 i .. 4 i + 3, in all of them.
__device__ __forceinline__ uint32_t max_of_four(uint32_t v) {
  const auto with = [&](uint32_t o) { v = v > o ? v : o; };
  with((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));  // lanes 1 0 3 2
  with((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true));  // lanes 2 3 0 1
  return v;
}

// A block's E8M0 byte and this lane's codes; u(j): 16 random bits.  A block with
// an infinity or NaN gets byte 255.  Below 2^-6 the codes' steps are all 2^-9:
// with 2^-6 added the same bits of the sum count them.
template <class Bits>
__device__ __forceinline__ uint32_t encode_codes(const float (&v)[8], const Bits& u, u32x2& codes) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t a = __float_as_uint(v[j]) & 0x7fffffffu;
    top = a > top ? a : top;
  }
  top = max_of_four(top);
  // the smallest e with top <= 448 * 2^e, 448 = 1.75 * 2^8; subnormal tops: -127
  const int e8 = (int)((top + 0x1fffffu) >> 23) - 8;  // carries where the fraction passes 0.75
  const bool bad = top >= 0x7f800000u;
  const uint32_t byte = bad ? 255u : (uint32_t)(e8 > 0 ? e8 : 0);
  const float inv = __uint_as_float(bad ? 0x00400000u : (254u - byte) << 23);
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    uint32_t all = 0;
#pragma unroll
    for (int j = 3; j >= 0; --j) {
      const float z = fabsf(v[4 * d + j]) * inv;
      const bool low = z < 0x1p-6f;
      const float y = low ? z + 0x1p-6f : z;
      const uint32_t c = ((__float_as_uint(y) + (u(4 * d + j) << 4)) >> 20) - (low ? 121u << 3 : 120u << 3);
      all = all << 8 | c;
    }
    uint32_t signs = 0;
#pragma unroll
    for (int j = 3; j >= 0; --j) signs = signs >> 8 | (__float_as_uint(v[4 * d + 3 - j]) & 0x80000000u);
    codes[d] = (bad ? 0x7f7f7f7fu : all) | signs;
  }
  return byte;
}

// p to one of its neighbours in bf16 by 16 random bits; to nearest without.
__device__ __forceinline__ uint32_t bf16_random(float p, uint32_t u) {
  const uint32_t b = __float_as_uint(p);
  return (b + ((b & 0x7f800000u) == 0x7f800000u ? 0u : u)) >> 16;
}
__device__ __forceinline__ uint32_t bf16_nearest(float p) {
  const uint32_t b = __float_as_uint(p);
  return p != p ? (b >> 16 | 0x40u) : bf16_rne_bits(p);
}

// One workgroup's elements; kWhole: all of its chunk exist.
template <bool kParamBf16, bool kGradBf16, bool kMx8, bool kNT, bool kWhole>
__device__ __forceinline__ void adamw_chunk(const typename AdamwBatch<kMx8>::Tensor& all, uint64_t chunk,
                                            uint64_t first_place, const AdamwScalars& s, float gs, bool random) {
  constexpr int kPer = kMx8 ? 8 : 4;  // to a lane: a block of 32 is four lanes
  constexpr uint32_t kRounds = kAdamChunk / (kAdamThreads * kPer);
  // the chunk's own tensors: places within it take 32 bits
  char* const param = static_cast<char*>(all.param) + chunk * (kParamBf16 ? 2 : 4);
  const char* const grad = static_cast<const char*>(all.grad) + chunk * (kGradBf16 ? 2 : 4);
  char* const avg = static_cast<char*>(all.avg) + chunk * (kMx8 ? 1 : 4);
  char* const sq = static_cast<char*>(all.sq) + chunk * (kMx8 ? 1 : 4);
  uint8_t* const avg_scales = all.avg_scales + chunk / 32;
  uint8_t* const sq_scales = all.sq_scales + chunk / 32;
  uint16_t* const copy = all.copy ? all.copy + chunk : nullptr;
  const uint32_t n = kWhole ? kAdamChunk : (uint32_t)(all.n - chunk);
  Elements<kParamBf16, kNT, kPer> p[kRounds];
  Elements<kGradBf16, kNT, kPer> g[kRounds];
  Elements<false, kNT, kPer> m[kRounds], v[kRounds];
  u32x2 mc[kRounds], rc[kRounds];
  uint32_t ms[kRounds], rs[kRounds];
  const auto left_of = [&](uint32_t i) -> uint32_t {
    return kWhole ? kPer : (i >= n ? 0u : (n - i < kPer ? n - i : (uint32_t)kPer));
  };
#pragma unroll
  for (uint32_t k = 0; k < kRounds; ++k) {
    const uint32_t i = (k * kAdamThreads + threadIdx.x) * kPer, left = left_of(i);
    if (!kWhole && left == 0) continue;
    p[k].template load<kWhole>(param, i, left);
    g[k].template load<kWhole>(grad, i, left);
    if constexpr (kMx8) {
      mc[k] = load_codes<kWhole, kNT>(avg, i, left);
      rc[k] = load_codes<kWhole, kNT>(sq, i, left);
      ms[k] = avg_scales[i / 32];
      rs[k] = sq_scales[i / 32];
    } else {
      m[k].template load<kWhole>(avg, i, left);
      v[k].template load<kWhole>(sq, i, left);
    }
  }
#pragma unroll
  for (uint32_t k = 0; k < kRounds; ++k) {
    const uint32_t i = (k * kAdamThreads + threadIdx.x) * kPer, left = left_of(i);
    // a block's lanes stay together: those past the end hold zeros
    if (!kWhole && i / 32 * 32 >= n) continue;
    float pv[kPer] = {}, gv[kPer] = {}, mv[kPer] = {}, vv[kPer] = {}, rv[kPer];
    if (kWhole || left) {
      p[k].values(pv);
      g[k].values(gv);
      if constexpr (kMx8) {
        decode_codes(mc[k], ms[k], mv);
        decode_codes(rc[k], rs[k], rv);
#pragma unroll
        for (int j = 0; j < kPer; ++j) vv[j] = rv[j] * rv[j];
      } else {
        m[k].values(mv);
        v[k].values(vv);
      }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float gj = gv[j] * gs;
      mv[j] = mv[j] * s.beta1 + gj * s.rest1;
      vv[j] = vv[j] * s.beta2 + (gj * gj) * s.rest2;
      rv[j] = sqrtf(vv[j]);
      pv[j] = pv[j] * s.decay - (mv[j] / (rv[j] * s.root + s.eps)) * s.rate;
      if (kMx8 && !kWhole && (uint32_t)j >= left) mv[j] = rv[j] = 0.f;  // the block's other elements alone choose its scale
    }
    uint32_t bits[kPer] = {};
    if (kMx8 || (kParamBf16 && random)) {
      const uint64_t place = first_place + chunk;  // of the chunk, a multiple of 32
      const uint32_t low = (uint32_t)place + i;
      const uint32_t key = mix_bits(s.key + (uint32_t)((place + i) >> 32));
#pragma unroll
      for (int j = 0; j < kPer; ++j) bits[j] = mix_bits(mix_bits(low + j) + key);
    }
    if (kWhole || left) {
      Elements<kParamBf16, kNT, kPer> out;
      if constexpr (kParamBf16) {
        uint32_t h[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) h[j] = random ? bf16_random(pv[j], mix_bits(bits[j]) >> 16) : bf16_nearest(pv[j]);
#pragma unroll
        for (int j = 0; j < kPer; j += 2) out.raw[j / 2] = h[j] | h[j + 1] << 16;
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) out.raw[j] = __float_as_uint(pv[j]);
        if (copy) {
          Elements<true, kNT, kPer> c;
#pragma unroll
          for (int j = 0; j < kPer; j += 2) c.raw[j / 2] = bf16_nearest(pv[j]) | bf16_nearest(pv[j + 1]) << 16;
          c.template store<kWhole>(copy, i, left);
        }
      }
      out.template store<kWhole>(param, i, left);
    }
    if constexpr (kMx8) {
      u32x2 codes;
      uint32_t byte = encode_codes(mv, [&](int j) { return bits[j] & 0xffffu; }, codes);
      if (kWhole || left) store_codes<kWhole, kNT>(avg, i, left, codes);
      if ((threadIdx.x & 3) == 0) avg_scales[i / 32] = (uint8_t)byte;
      byte = encode_codes(rv, [&](int j) { return bits[j] >> 16; }, codes);
      if (kWhole || left) store_codes<kWhole, kNT>(sq, i, left, codes);
      if ((threadIdx.x & 3) == 0) sq_scales[i / 32] = (uint8_t)byte;
    } else if (kWhole || left) {
      Elements<false, kNT, kPer> o;
#pragma unroll
      for (int j = 0; j < kPer; ++j) o.raw[j] = __float_as_uint(mv[j]);
      o.template store<kWhole>(avg, i, left);
#pragma unroll
      for (int j = 0; j < kPer; ++j) o.raw[j] = __float_as_uint(vv[j]);
      o.template store<kWhole>(sq, i, left);
    }
  }
}

template <bool kParamBf16, bool kGradBf16, bool kMx8, bool kNT>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(AdamwBatch<kMx8> batch, AdamwScalars s,
                                                             const float* __restrict__ grad_scale, bool random) {
  // the tensor of this workgroup: the last one that starts at or before it
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t hit = __ballot(lane < batch.count && batch.first[lane < batch.count ? lane : 0] <= blockIdx.x);
  const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(63 - __builtin_clzll(hit)));
  const uint64_t chunk = (uint64_t)(blockIdx.x - batch.first[at]) * kAdamChunk;
  const float gs = grad_scale ? *grad_scale : 1.f;
  if (chunk + kAdamChunk <= batch.t[at].n)
    adamw_chunk<kParamBf16, kGradBf16, kMx8, kNT, true>(batch.t[at], chunk, batch.place[at], s, gs, random);
  else
    adamw_chunk<kParamBf16, kGradBf16, kMx8, kNT, false>(batch.t[at], chunk, batch.place[at], s, gs, random);
}

}  // namespace trace_dev

namespace trace_host {

using namespace trace_dev;

namespace {

template <bool kParamBf16, bool kGradBf16, bool kMx8>
hipError_t run_adamw(const AdamwTensor* tensors, uint32_t count, bool nt, const AdamwScalars& s, const float* grad_scale,
                     bool random, hipStream_t stream) {
  constexpr uint32_t kMostGroups = 0xffffffffu / kAdamThreads;  // a launch counts its work-items in 32 bits
  using Batch = AdamwBatch<kMx8>;
  Batch b;
  b.count = 0;
  uint64_t groups = 0, place = 0;
  const auto flush = [&]() -> hipError_t {
    if (b.count == 0) return hipSuccess;
    hipLaunchKernelGGL((nt ? adamw_kernel<kParamBf16, kGradBf16, kMx8, true> : adamw_kernel<kParamBf16, kGradBf16, kMx8, false>),
                       dim3((uint32_t)groups), dim3(kAdamThreads), 0, stream, b, s, grad_scale, random);
    b.count = 0;
    groups = 0;
    return hipGetLastError();
  };
  for (uint32_t i = 0; i < count; ++i) {
    const AdamwTensor& t = tensors[i];
    if (t.n == 0) continue;
    const uint64_t need = (t.n + kAdamChunk - 1) / kAdamChunk;
    if (b.count == Batch::kMost || groups + need > kMostGroups)
      if (hipError_t e = flush()) return e;
    b.t[b.count] = typename Batch::Tensor(t);
    b.first[b.count] = (uint32_t)groups;
    b.place[b.count] = place;
    ++b.count;
    groups += need;
    place += (t.n + 31) / 32 * 32;
  }
  return flush();
}

}  // namespace

hipError_t launch_adamw(const AdamwTensor* tensors, uint32_t count, const AdamwTypes& types, const AdamwScalars& s,
                        const float* grad_scale, hipStream_t stream) {
  const uint64_t each = (types.param_bf16 ? 4 : 8) + (types.grad_bf16 ? 2 : 4) + (types.mx8 ? 4 : 16);
  uint64_t all = 0;
  for (uint32_t i = 0; i < count; ++i) all += tensors[i].n;
  const bool nt = past_cache(all * each);
  const auto of = [&](auto pb, auto gb) {
    constexpr bool kP = decltype(pb)::value, kG = decltype(gb)::value;
    return types.mx8 ? run_adamw<kP, kG, true>(tensors, count, nt, s, grad_scale, types.random, stream)
                     : run_adamw<kP, kG, false>(tensors, count, nt, s, grad_scale, types.random, stream);
  };
  constexpr std::integral_constant<bool, true> yes;
  constexpr std::integral_constant<bool, false> no;
  return types.param_bf16 ? (types.grad_bf16 ? of(yes, yes) : of(yes, no)) : (types.grad_bf16 ? of(no, yes) : of(no, no));
}

}  // namespace trace_host
