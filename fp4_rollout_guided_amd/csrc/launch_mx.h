// Internal host-side launchers of the microscaled products and of the routed
// rows (not part of the C ABI).  Arguments have been validated by
// api_mx_product.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace trace_host {

// Element format of the activations' codes; the weights' is E2M1.
enum MxFormat { kE2M1 = 0, kE4M3 = 1 };

// One product y = A W^T, or one per group of packed rows.
struct MxProductArgs {
  const uint16_t* x;         // [rows, k] in bf16, where mx_product_rounds; else nullptr
  const uint8_t* a_codes;    // [src_rows, k]
  const uint8_t* a_scales;   // [src_rows, k / 32]
  const int64_t* row_index;  // row r reads source row row_index[r]; nullptr: row r (src_rows == rows)
  uint64_t src_rows;
  uint64_t rows;
  const int64_t* offsets;  // [groups + 1], or nullptr for one group of all rows
  uint32_t groups;
  const uint8_t* w_codes;   // [groups, n, k]
  const uint8_t* w_scales;  // [groups, n, k / 32]
  uint32_t n, k;
  void* y;   // [rows, n] in bf16, or
  bool f32;  // in fp32 (grouped products)
  bool stream_out = false;  // y is past the last-level cache: the launcher's
  bool plan_only = false;   // check the grid, launch nothing
};

// The gradients: grad_y W (to the activations) or grad_y^T A (to the weights).
struct MxGradArgs {
  const uint16_t* grad_y;  // [rows, n]
  uint64_t rows;
  const int64_t* offsets;  // as above
  uint32_t groups;
  const uint8_t* q_codes;   // the other factor: W [groups, n, k], or A [src_rows, k]
  const uint8_t* q_scales;
  const int64_t* row_index;  // of A's rows, or nullptr
  uint64_t src_rows;
  uint32_t n, k;
  const uint8_t* mask;  // clip mask of the gradient's own tensor, or nullptr
  void* grad;           // [rows, k], or [groups, n, k], in bf16, or
  bool f32;             // in fp32 (grouped, to the activations)
  float* partial;       // workspace of the split contraction, or nullptr
  bool stream_out = false;  // grad is past the last-level cache: the launcher's
};

// Sizes in 32-element blocks; mask may be nullptr.  used: nullptr, or where
// the device has how many rows of row_blocks blocks are wanted.
hipError_t launch_mx_quantize(MxFormat fmt, const uint16_t* x, uint64_t nblocks, uint8_t* scales, uint8_t* codes,
                              uint8_t* mask, const int64_t* used, uint32_t row_blocks, hipStream_t stream);
// Whether a product of so many rows takes bf16 activations as they are.
bool mx_product_rounds(uint64_t rows, uint64_t k, bool grouped);
hipError_t launch_mx_product(MxFormat fmt, const MxProductArgs& p, hipStream_t stream);

hipError_t launch_mx_grad_input(const MxGradArgs& p, hipStream_t stream);
// Parts of the contraction over the rows that are summed in a workspace of
// parts * n * k fp32 words; 1: no workspace.
uint32_t mx_grad_weight_parts(uint64_t rows, uint32_t groups, uint32_t n, uint32_t k);
hipError_t launch_mx_grad_weight(MxFormat fmt, const MxGradArgs& p, hipStream_t stream);

// Routed rows.
constexpr uint32_t kMaxExperts = 1024;
constexpr uint32_t kMaxTopk = 64;
uint64_t expert_sort_workspace_words(uint64_t pairs, uint32_t experts);
hipError_t launch_expert_sort(const int64_t* ids, uint64_t pairs, uint32_t topk, uint32_t experts, uint32_t* workspace,
                              int64_t* offsets, int64_t* row_index, int64_t* slot, hipStream_t stream);
hipError_t launch_expert_dispatch(const uint16_t* x, uint64_t tokens, uint64_t cols, const int64_t* row_index,
                                  uint64_t rows, uint16_t* out, hipStream_t stream);
// y: bf16, or fp32 where f32.
hipError_t launch_expert_combine(const void* y, bool f32, uint64_t rows, uint64_t cols, const int64_t* slot,
                                 const float* weights, uint64_t tokens, uint32_t topk, uint16_t* out,
                                 hipStream_t stream);
// clear: rows of grad_y that no slot names become zeros.
hipError_t launch_expert_combine_bwd(const uint16_t* grad_out, const uint16_t* y, uint64_t rows, uint64_t cols,
                                     const int64_t* slot, const float* weights, uint64_t tokens, uint32_t topk,
                                     bool clear, uint16_t* grad_y, float* grad_weights, hipStream_t stream);

}  // namespace trace_host
