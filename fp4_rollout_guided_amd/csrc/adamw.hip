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
// are rounded likewise where a seed is given, or to nearest.
//
// Bound by memory: each element's bytes once in, once out, 16 bytes per lane of
// an fp32 tensor.  A workgroup owns 4096 consecutive elements of one tensor and
// loads all of them before the first arithmetic.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"
#include "fp4_block.h"
#include "launch.h"
#include "launch_step.h"

namespace trace_dev {

using trace_host::AdamwScalars;
using trace_host::AdamwTensor;

constexpr uint32_t kAdamThreads = 256;
constexpr uint32_t kAdamRounds = 4;
constexpr uint32_t kAdamChunk = kAdamThreads * 4 * kAdamRounds;
// Tensors of a launch: their descriptors are kernel arguments, 4 KiB at most.
constexpr uint32_t kAdamTensors = 48;

struct AdamwBatch {
  AdamwTensor t[kAdamTensors];
  uint32_t first[kAdamTensors];  // the tensor's first workgroup
  uint64_t place[kAdamTensors];  // of its first element among all tensors' elements, each tensor filled up to 32
  uint32_t count;
};
static_assert(sizeof(AdamwBatch) + sizeof(AdamwScalars) + 16 <= 4096, "kernel arguments");

// A 32-bit integer to another one, each bit of which depends on all of its
// bits: shifts and products with odd numbers, the fractions of the square roots
// of two and three.
__host__ __device__ inline uint32_t mix_bits(uint32_t h) {
  h ^= h >> 16;
  h *= 0x6a09e667u;
  h ^= h >> 15;
  h *= 0xbb67ae85u;
  return h ^ (h >> 16);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Four consecutive elements at element i, of which `left` exist.
template <bool kBf16, bool kNT>
struct Four {
  uint32_t raw[kBf16 ? 2 : 4];
  __device__ __forceinline__ void load(const void* from, uint64_t i, uint32_t left) {
    if (left >= 4) {
      if constexpr (kBf16) {
        const u32x2* at = reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(from) + i);
        const u32x2 v = kNT ? __builtin_nontemporal_load(at) : *at;
        raw[0] = v[0], raw[1] = v[1];
      } else {
        const uint4 v = load_vec<kNT>(reinterpret_cast<const uint4*>(static_cast<const uint32_t*>(from) + i));
        raw[0] = v.x, raw[1] = v.y, raw[2] = v.z, raw[3] = v.w;
      }
      return;
    }
#pragma unroll
    for (uint32_t j = 0; j < (kBf16 ? 2 : 4); ++j) raw[j] = 0;
#pragma unroll
    for (uint32_t j = 0; j < 3; ++j) {
      if (j >= left) continue;
      if constexpr (kBf16)
        raw[j >> 1] |= (uint32_t)static_cast<const uint16_t*>(from)[i + j] << (16 * (j & 1));
      else
        raw[j] = static_cast<const uint32_t*>(from)[i + j];
    }
  }
  __device__ __forceinline__ void values(float (&v)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kBf16)
        v[j] = (j & 1) ? bf16_hi(raw[j >> 1]) : bf16_lo(raw[j >> 1]);
      else
        v[j] = __uint_as_float(raw[j]);
    }
  }
  __device__ __forceinline__ void store(void* to, uint64_t i, uint32_t left) const {
    if (left >= 4) {
      if constexpr (kBf16) {
        u32x2* at = reinterpret_cast<u32x2*>(static_cast<uint16_t*>(to) + i);
        const u32x2 v = {raw[0], raw[1]};
        if (kNT)
          __builtin_nontemporal_store(v, at);
        else
          *at = v;
      } else {
        store_vec<kNT>(reinterpret_cast<uint4*>(static_cast<uint32_t*>(to) + i),
                       make_uint4(raw[0], raw[1], raw[2], raw[3]));
      }
      return;
    }
#pragma unroll
    for (uint32_t j = 0; j < 3; ++j) {
      if (j >= left) continue;
      if constexpr (kBf16)
        static_cast<uint16_t*>(to)[i + j] = (uint16_t)(raw[j >> 1] >> (16 * (j & 1)));
      else
        static_cast<uint32_t*>(to)[i + j] = raw[j];
    }
  }
};

// Four code bytes likewise.
template <bool kNT>
__device__ __forceinline__ uint32_t load_codes(const void* from, uint64_t i, uint32_t left) {
  if (left >= 4) {
    const uint32_t* at = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(from) + i);
    return kNT ? __builtin_nontemporal_load(at) : *at;
  }
  uint32_t v = 0;
  for (uint32_t j = 0; j < left; ++j) v |= (uint32_t)static_cast<const uint8_t*>(from)[i + j] << (8 * j);
  return v;
}
template <bool kNT>
__device__ __forceinline__ void store_codes(void* to, uint64_t i, uint32_t left, uint32_t v) {
  if (left >= 4) {
    uint32_t* at = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(to) + i);
    if (kNT)
      __builtin_nontemporal_store(v, at);
    else
      *at = v;
    return;
  }
  for (uint32_t j = 0; j < left; ++j) static_cast<uint8_t*>(to)[i + j] = (uint8_t)(v >> (8 * j));
}

// 2^(b - 127), b in 0 .. 254, and NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : (b == 255 ? 0x7fc00000u : b << 23));
}

__device__ __forceinline__ void decode_codes(uint32_t c, uint32_t scale, float (&v)[4]) {
  const float s = e8m0_value(scale);
  v[0] = __builtin_amdgcn_cvt_f32_fp8((int)c, 0) * s;
  v[1] = __builtin_amdgcn_cvt_f32_fp8((int)c, 1) * s;
  v[2] = __builtin_amdgcn_cvt_f32_fp8((int)c, 2) * s;
  v[3] = __builtin_amdgcn_cvt_f32_fp8((int)c, 3) * s;
}

// The larger of the values of lanes 8 i .. 8 i + 7, in all of them.
__device__ __forceinline__ uint32_t max_of_eight(uint32_t v) {
  const auto with = [&](uint32_t o) { v = v > o ? v : o; };
  with((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));   // lanes 1 0 3 2
  with((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true));   // lanes 2 3 0 1
  with((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true));  // eight lanes mirrored
  return v;
}

// A block's E8M0 byte and its elements' codes; u: 16 random bits each.  A block
// with an infinity or NaN gets byte 255.
__device__ __forceinline__ uint32_t encode_codes(const float (&v)[4], const uint32_t (&u)[4], uint32_t& codes) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = __float_as_uint(v[j]) & 0x7fffffffu;
    top = a > top ? a : top;
  }
  top = max_of_eight(top);
  // the smallest e with top <= 448 * 2^e, 448 = 1.75 * 2^8; subnormal tops: -127
  const int e8 = (int)(top >> 23) + ((top & 0x7fffffu) > 0x600000u ? 1 : 0) - 8;
  const uint32_t byte = top >= 0x7f800000u ? 255u : (uint32_t)(e8 > 0 ? e8 : 0);
  const float inv = __uint_as_float(byte >= 254 ? 0x00400000u : (254u - byte) << 23);
  codes = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float z = fabsf(v[j]) * inv;
    uint32_t c;
    if (z < 0x1p-6f)
      c = (uint32_t)floorf(z * 512.f + (float)u[j] * 0x1p-16f);
    else
      c = ((__float_as_uint(z) + (u[j] << 4)) >> 20) - (120u << 3);
    c = byte == 255u ? 0x7fu : c;
    codes |= (c | (__float_as_uint(v[j]) >> 31 << 7)) << (8 * j);
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

template <bool kParamBf16, bool kGradBf16, bool kMx8, bool kNT>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(AdamwBatch batch, AdamwScalars s,
                                                             const float* __restrict__ grad_scale, bool random) {
  // the tensor of this workgroup: the last one that starts at or before it
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t hit = __ballot(lane < batch.count && batch.first[lane < batch.count ? lane : 0] <= blockIdx.x);
  const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(63 - __builtin_clzll(hit)));
  const AdamwTensor t = batch.t[at];
  const uint64_t chunk = (uint64_t)(blockIdx.x - batch.first[at]) * kAdamChunk;
  const float gs = grad_scale ? *grad_scale : 1.f;
  Four<kParamBf16, kNT> p[kAdamRounds];
  Four<kGradBf16, kNT> g[kAdamRounds];
  Four<false, kNT> m[kAdamRounds], v[kAdamRounds];
  uint32_t mc[kAdamRounds], rc[kAdamRounds], ms[kAdamRounds], rs[kAdamRounds];
#pragma unroll
  for (uint32_t k = 0; k < kAdamRounds; ++k) {
    const uint64_t i = chunk + (k * kAdamThreads + threadIdx.x) * 4;
    if (i >= t.n) continue;
    const uint32_t left = t.n - i < 4 ? (uint32_t)(t.n - i) : 4u;
    p[k].load(t.param, i, left);
    g[k].load(t.grad, i, left);
    if constexpr (kMx8) {
      mc[k] = load_codes<kNT>(t.avg, i, left);
      rc[k] = load_codes<kNT>(t.sq, i, left);
      ms[k] = t.avg_scales[i / 32];
      rs[k] = t.sq_scales[i / 32];
    } else {
      m[k].load(t.avg, i, left);
      v[k].load(t.sq, i, left);
    }
  }
#pragma unroll
  for (uint32_t k = 0; k < kAdamRounds; ++k) {
    const uint64_t i = chunk + (k * kAdamThreads + threadIdx.x) * 4;
    // a block's eight lanes stay together: those past the end hold zeros
    if (i / 32 * 32 >= t.n) continue;
    const uint32_t left = i >= t.n ? 0u : (t.n - i < 4 ? (uint32_t)(t.n - i) : 4u);
    float pv[4] = {0, 0, 0, 0}, gv[4] = {0, 0, 0, 0}, mv[4] = {0, 0, 0, 0}, vv[4] = {0, 0, 0, 0}, rv[4];
    if (left) {
      p[k].values(pv);
      g[k].values(gv);
      if constexpr (kMx8) {
        decode_codes(mc[k], ms[k], mv);
        decode_codes(rc[k], rs[k], rv);
#pragma unroll
        for (int j = 0; j < 4; ++j) vv[j] = rv[j] * rv[j];
      } else {
        m[k].values(mv);
        v[k].values(vv);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float gj = gv[j] * gs;
      mv[j] = mv[j] * s.beta1 + gj * s.rest1;
      vv[j] = vv[j] * s.beta2 + (gj * gj) * s.rest2;
      rv[j] = sqrtf(vv[j]);
      pv[j] = pv[j] * s.decay - (mv[j] / (rv[j] * s.root + s.eps)) * s.rate;
      if (kMx8 && (uint32_t)j >= left) mv[j] = rv[j] = 0.f;  // the block's other elements alone choose its scale
    }
    uint32_t bits[4] = {0, 0, 0, 0};
    if (kMx8 || (kParamBf16 && random)) {
      const uint64_t place = batch.place[at] + i;
      const uint32_t key = mix_bits(s.key + (uint32_t)(place >> 32));
#pragma unroll
      for (int j = 0; j < 4; ++j) bits[j] = mix_bits(mix_bits((uint32_t)place + j) + key);  // place is a multiple of 4
    }
    if (left) {
      Four<kParamBf16, kNT> out;
      if constexpr (kParamBf16) {
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = random ? bf16_random(pv[j], mix_bits(bits[j]) >> 16) : bf16_nearest(pv[j]);
        out.raw[0] = h[0] | h[1] << 16, out.raw[1] = h[2] | h[3] << 16;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) out.raw[j] = __float_as_uint(pv[j]);
        if (t.copy) {
          Four<true, kNT> c;
          c.raw[0] = bf16_nearest(pv[0]) | bf16_nearest(pv[1]) << 16;
          c.raw[1] = bf16_nearest(pv[2]) | bf16_nearest(pv[3]) << 16;
          c.store(t.copy, i, left);
        }
      }
      out.store(t.param, i, left);
    }
    if constexpr (kMx8) {
      uint32_t lo[4], hi[4], codes;
#pragma unroll
      for (int j = 0; j < 4; ++j) lo[j] = bits[j] & 0xffffu, hi[j] = bits[j] >> 16;
      uint32_t byte = encode_codes(mv, lo, codes);
      if (left) store_codes<kNT>(t.avg, i, left, codes);
      if ((i & 31) == 0) t.avg_scales[i / 32] = (uint8_t)byte;
      byte = encode_codes(rv, hi, codes);
      if (left) store_codes<kNT>(t.sq, i, left, codes);
      if ((i & 31) == 0) t.sq_scales[i / 32] = (uint8_t)byte;
    } else if (left) {
      Four<false, kNT> o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o.raw[j] = __float_as_uint(mv[j]);
      o.store(t.avg, i, left);
#pragma unroll
      for (int j = 0; j < 4; ++j) o.raw[j] = __float_as_uint(vv[j]);
      o.store(t.sq, i, left);
    }
  }
}

}  // namespace trace_dev

namespace trace_host {

using namespace trace_dev;

hipError_t launch_adamw(const AdamwTensor* tensors, uint32_t count, const AdamwTypes& types, const AdamwScalars& s,
                        const float* grad_scale, hipStream_t stream) {
  const uint64_t each = (types.param_bf16 ? 4 : 8) + (types.grad_bf16 ? 2 : 4) + (types.mx8 ? 4 : 16);
  uint64_t all = 0;
  for (uint32_t i = 0; i < count; ++i) all += tensors[i].n;
  const bool nt = past_cache(all * each);
  constexpr uint32_t kMostGroups = 0xffffffffu / kAdamThreads;  // a launch counts its work-items in 32 bits
  const auto kernel = [&](auto pb, auto gb, auto mx) {
    constexpr bool kP = decltype(pb)::value, kG = decltype(gb)::value, kM = decltype(mx)::value;
    return nt ? adamw_kernel<kP, kG, kM, true> : adamw_kernel<kP, kG, kM, false>;
  };
  constexpr std::integral_constant<bool, true> yes;
  constexpr std::integral_constant<bool, false> no;
  const auto of = [&](auto pb, auto gb) { return types.mx8 ? kernel(pb, gb, yes) : kernel(pb, gb, no); };
  const auto run = types.param_bf16 ? (types.grad_bf16 ? of(yes, yes) : of(yes, no))
                                    : (types.grad_bf16 ? of(no, yes) : of(no, no));
  AdamwBatch b;
  b.count = 0;
  uint64_t groups = 0, place = 0;
  const auto flush = [&]() -> hipError_t {
    if (b.count == 0) return hipSuccess;
    hipLaunchKernelGGL(run, dim3((uint32_t)groups), dim3(kAdamThreads), 0, stream, b, s, grad_scale, types.random);
    b.count = 0;
    groups = 0;
    return hipGetLastError();
  };
  for (uint32_t i = 0; i < count; ++i) {
    const AdamwTensor& t = tensors[i];
    if (t.n == 0) continue;
    const uint64_t need = (t.n + kAdamChunk - 1) / kAdamChunk;
    if (b.count == kAdamTensors || groups + need > kMostGroups)
      if (hipError_t e = flush()) return e;
    b.t[b.count] = t;
    b.first[b.count] = (uint32_t)groups;
    b.place[b.count] = place;
    ++b.count;
    groups += need;
    place += (t.n + 31) / 32 * 32;
  }
  return flush();
}

}  // namespace trace_host
