// Internal host-side launchers of the vocabulary loss, the router and the
// optimiser step (not part of the C ABI).  Arguments have been validated by
// api_step.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace trace_host {

// Softmax cross entropy of x W^T over the vocabulary.
struct CrossEntropyArgs {
  const uint16_t* x;       // [tokens, k]
  const uint16_t* w;       // [vocab, k]
  const int64_t* targets;  // [tokens]; outside [0, vocab): ignored
  uint64_t tokens;
  uint32_t vocab, k;
  float scale;
  void* workspace;
};
uint64_t cross_entropy_workspace_bytes(uint64_t tokens, uint32_t vocab, uint32_t k);
uint64_t cross_entropy_bwd_workspace_bytes(uint64_t tokens, uint32_t vocab, uint32_t k);
hipError_t launch_cross_entropy(const CrossEntropyArgs& p, float* loss, float* lse, hipStream_t stream);
// grad_x or grad_w may be nullptr.
hipError_t launch_cross_entropy_bwd(const CrossEntropyArgs& p, const float* grad_loss, const float* lse,
                                    uint16_t* grad_x, uint16_t* grad_w, hipStream_t stream);

// The router.
constexpr uint32_t kMaxRouted = 1024;  // experts
struct RouteArgs {
  const void* logits;  // [tokens, experts] in bf16 or fp32
  bool bf16;
  uint64_t tokens;
  uint32_t experts, topk;
  bool renormalize;
};
uint64_t route_workspace_bytes(uint64_t tokens, uint32_t experts);
// valid: [tokens], 0 for rows left out, or nullptr.
hipError_t launch_route(const RouteArgs& p, const uint8_t* valid, void* workspace, int64_t* ids, float* weights,
                        int64_t* counts, float* probs, float* balance, hipStream_t stream);
// grad_weights or grad_balance may be nullptr: zeros.
hipError_t launch_route_bwd(const RouteArgs& p, const float* grad_weights, const float* grad_balance,
                            const int64_t* ids, const float* weights, const int64_t* counts, void* grad_logits,
                            hipStream_t stream);

// The optimiser step.

// A 32-bit integer to another one, each bit of which depends on all of its
// bits: shifts and products with odd numbers, the fractions of the square roots
// of two and three.  The seed's on the host, each element's place on the GPU.
__host__ __device__ inline uint32_t mix_bits(uint32_t h) {
  h ^= h >> 16;
  h *= 0x6a09e667u;
  h ^= h >> 15;
  h *= 0xbb67ae85u;
  return h ^ (h >> 16);
}
struct AdamwTensor {
  void* param;
  const void* grad;
  void* avg;            // fp32, or E4M3 codes
  void* sq;             // fp32, or E4M3 codes of the root
  uint8_t* avg_scales;  // nullptr with fp32 states
  uint8_t* sq_scales;
  uint16_t* copy;       // nullptr: none
  uint64_t n;
};
struct AdamwScalars {
  float beta1, rest1, beta2, rest2, eps, decay, rate, root;
  uint32_t key;
};
struct AdamwTypes {
  bool param_bf16, grad_bf16, mx8, random;
};
hipError_t launch_adamw(const AdamwTensor* tensors, uint32_t count, const AdamwTypes& types, const AdamwScalars& s,
                        const float* grad_scale, hipStream_t stream);

}  // namespace trace_host
