// C ABI of the microscaled products and the routed rows: argument validation
// and dispatch to the HIP launchers, as in api.cpp.
#include "trace.h"

#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "launch_mx.h"

using namespace trace_api;
using trace_host::kE2M1;
using trace_host::kE4M3;
using trace_host::MxFormat;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxDim = (int64_t)1 << 24;
constexpr int64_t kMaxProductGroups = 4096;

// Sizes of a product: rows x k times (groups of) n x k.
trace_status product_sizes(int64_t src_rows, int64_t rows, int64_t groups, int64_t n, int64_t k) {
  if (rows < 0 || rows >= kMaxRows || src_rows < 0 || src_rows >= kMaxRows) return TRACE_E_SHAPE;
  if (n < 0 || n >= kMaxDim || n % 16 != 0 || k < 0 || k >= kMaxDim || k % 32 != 0) return TRACE_E_SHAPE;
  if (groups < 1 || groups > kMaxProductGroups) return TRACE_E_SHAPE;
  return TRACE_OK;
}

// offsets and groups of one weight (NULL, 0) or of one per group; *groups_out
// is the number of weights.
trace_status product_groups(const int64_t* offsets, int64_t groups, int64_t* groups_out) {
  if (!offsets) {
    *groups_out = 1;
    return groups == 0 ? TRACE_OK : TRACE_E_NULL;
  }
  if (!aligned(offsets, 8)) return TRACE_E_ALIGN;
  *groups_out = groups;
  return TRACE_OK;
}

// A launcher's answer; a grid past the hardware's limit is the sizes' fault.
trace_status launch_status(hipError_t e) { return e == hipErrorInvalidConfiguration ? TRACE_E_SHAPE : hip_status(e); }

uint64_t code_bytes(MxFormat fmt, uint64_t elements) { return fmt == kE2M1 ? elements / 2 : elements; }

size_t linear_workspace(MxFormat fmt, int64_t src_rows, int64_t rows, int64_t groups, int64_t k) {
  uint64_t n = 0;
  if (mx_site_size(src_rows, k, &n) != TRACE_OK || product_sizes(src_rows, rows, groups == 0 ? 1 : groups, 0, k) != TRACE_OK)
    return 0;
  if (trace_host::mx_product_rounds((uint64_t)rows, (uint64_t)k, groups > 0)) return 0;
  return (size_t)(code_bytes(fmt, n) + (n / 32 + 15) / 16 * 16);
}

trace_status quantize(MxFormat fmt, const uint16_t* x, int64_t rows, int64_t cols, uint8_t* scales, uint8_t* codes,
                      uint8_t* mask, void* stream) {
  uint64_t n = 0;
  if (trace_status st = mx_site_size(rows, cols, &n)) return st;
  if (n == 0) return TRACE_OK;
  if (!x || !scales || !codes) return TRACE_E_NULL;
  if (!aligned(x, 16) || !aligned(codes, 16) || (mask && !aligned(mask, 2))) return TRACE_E_ALIGN;
  const Range outs[3] = {rng(scales, n / 32), rng(codes, code_bytes(fmt, n)), rng(mask, mask ? n / 8 : 0)};
  const Range ins[1] = {rng(x, 2 * n)};
  if (trace_status st = check_alias(outs, 3, ins, 1)) return st;
  return hip_status(trace_host::launch_mx_quantize(fmt, x, n / 32, scales, codes, mask, nullptr, 0,
                                                   static_cast<hipStream_t>(stream)));
}

// x: bf16 activations to round first (workspace takes their record), or NULL
// where a_scales and a_codes hold it.
trace_status product(MxFormat fmt, const uint16_t* x, void* workspace, size_t workspace_bytes,
                     const uint8_t* a_scales, const uint8_t* a_codes, int64_t src_rows, const int64_t* row_index,
                     int64_t rows, const int64_t* offsets, int64_t groups, const uint8_t* w_scales,
                     const uint8_t* w_codes, int64_t n, int64_t k, bool linear, void* y, bool f32, void* stream) {
  int64_t weights = 0;
  if (trace_status st = product_groups(offsets, groups, &weights)) return st;
  if (trace_status st = product_sizes(src_rows, rows, weights, n, k)) return st;
  if (row_index && !offsets) return TRACE_E_NULL;
  if (!row_index && rows > 0 && src_rows != rows) return TRACE_E_SHAPE;  // no rows need no index
  uint64_t na = 0;
  if (trace_status st = mx_site_size(src_rows, k, &na)) return st;
  const size_t need = linear ? linear_workspace(fmt, src_rows, rows, groups, k) : 0;
  if (rows == 0 || n == 0) return TRACE_OK;
  const uint64_t nw = (uint64_t)weights * (uint64_t)n * (uint64_t)k, ny = (uint64_t)rows * (uint64_t)n;
  if (!y || (nw > 0 && (!w_scales || !w_codes))) return TRACE_E_NULL;
  if (na > 0 && (linear ? !x || (need > 0 && !workspace) : !a_scales || !a_codes)) return TRACE_E_NULL;
  if (linear && workspace_bytes < need) return TRACE_E_SHAPE;
  if (!aligned(x, 16) || !aligned(workspace, 16) || !aligned(a_codes, 16) || !aligned(w_codes, 16) || !aligned(y, 16) ||
      !aligned(row_index, 8))
    return TRACE_E_ALIGN;
  const Range outs[2] = {rng(y, (f32 ? 4 : 2) * ny), rng(workspace, need)};
  const Range ins[7] = {rng(x, x ? 2 * na : 0),
                        rng(a_scales, a_scales ? na / 32 : 0),
                        rng(a_codes, a_codes ? code_bytes(fmt, na) : 0),
                        rng(w_scales, nw / 32),
                        rng(w_codes, nw / 2),
                        rng(row_index, row_index ? 8 * (uint64_t)rows : 0),
                        rng(offsets, offsets ? 8 * ((uint64_t)weights + 1) : 0)};
  if (trace_status st = check_alias(outs, 2, ins, 7)) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* const codes = static_cast<uint8_t*>(workspace);  // of the rounded activations, where need > 0
  uint8_t* const scales = need > 0 ? codes + code_bytes(fmt, na) : nullptr;
  const bool rounds = linear && trace_host::mx_product_rounds((uint64_t)rows, (uint64_t)k, groups > 0);
  trace_host::MxProductArgs p{rounds ? x : nullptr, need > 0 ? codes : a_codes, need > 0 ? scales : a_scales, row_index,
                              (uint64_t)src_rows, (uint64_t)rows, offsets, (uint32_t)weights, w_codes, w_scales,
                              (uint32_t)n, (uint32_t)k, y, f32};
  if (need > 0) {
    p.plan_only = true;  // sizes that are refused are refused before anything is enqueued
    if (trace_status st = launch_status(trace_host::launch_mx_product(fmt, p, s))) return st;
    p.plan_only = false;
    const int64_t* used = offsets && !row_index ? offsets + groups : nullptr;  // rows behind the last group are not read
    if (trace_status st = hip_status(trace_host::launch_mx_quantize(fmt, x, na / 32, scales, codes, nullptr, used,
                                                                    (uint32_t)(k / 32), s)))
      return st;
  }
  return launch_status(trace_host::launch_mx_product(fmt, p, s));
}

trace_status grad_input(const uint16_t* grad_y, int64_t rows, const int64_t* offsets, int64_t groups,
                        const uint8_t* w_scales, const uint8_t* w_codes, int64_t n, int64_t k, const uint8_t* mask,
                        void* grad_x, bool f32, void* stream) {
  int64_t weights = 0;
  if (trace_status st = product_groups(offsets, groups, &weights)) return st;
  if (trace_status st = product_sizes(rows, rows, weights, n, k)) return st;
  if (rows == 0 || k == 0) return TRACE_OK;
  const uint64_t nw = (uint64_t)weights * (uint64_t)n * (uint64_t)k;
  const uint64_t ny = (uint64_t)rows * (uint64_t)n, nx = (uint64_t)rows * (uint64_t)k;
  if (!grad_x || (n > 0 && (!grad_y || !w_scales || !w_codes))) return TRACE_E_NULL;
  if (!aligned(grad_y, 16) || !aligned(w_codes, 16) || !aligned(grad_x, 16) || !aligned(mask, 2)) return TRACE_E_ALIGN;
  const Range outs[1] = {rng(grad_x, (f32 ? 4 : 2) * nx)};
  const Range ins[5] = {rng(grad_y, 2 * ny), rng(w_scales, nw / 32), rng(w_codes, nw / 2),
                        rng(mask, mask ? nx / 8 : 0), rng(offsets, offsets ? 8 * ((uint64_t)weights + 1) : 0)};
  if (trace_status st = check_alias(outs, 1, ins, 5)) return st;
  const trace_host::MxGradArgs p{grad_y, (uint64_t)rows, offsets, (uint32_t)weights, w_codes, w_scales, nullptr,
                                 (uint64_t)rows, (uint32_t)n, (uint32_t)k, mask, grad_x, f32, nullptr};
  return launch_status(trace_host::launch_mx_grad_input(p, static_cast<hipStream_t>(stream)));
}

size_t grad_weight_workspace(int64_t rows, int64_t groups, int64_t n, int64_t k) {
  const int64_t weights = groups == 0 ? 1 : groups;
  if (product_sizes(rows, rows, weights, n, k) != TRACE_OK) return 0;
  const uint64_t parts = trace_host::mx_grad_weight_parts((uint64_t)rows, groups == 0 ? 0u : (uint32_t)groups,
                                                          (uint32_t)n, (uint32_t)k);
  return parts > 1 ? (size_t)(parts * (uint64_t)n * (uint64_t)k * sizeof(float)) : 0;
}

trace_status grad_weight(MxFormat fmt, const uint16_t* grad_y, int64_t rows, const int64_t* offsets, int64_t groups,
                         const uint8_t* a_scales, const uint8_t* a_codes, int64_t src_rows, const int64_t* row_index,
                         int64_t n, int64_t k, const uint8_t* mask, uint16_t* grad_w, void* workspace,
                         size_t workspace_bytes, void* stream) {
  int64_t weights = 0;
  if (trace_status st = product_groups(offsets, groups, &weights)) return st;
  if (trace_status st = product_sizes(src_rows, rows, weights, n, k)) return st;
  if (row_index && !offsets) return TRACE_E_NULL;
  if (!row_index && rows > 0 && src_rows != rows) return TRACE_E_SHAPE;  // no rows need no index
  uint64_t na = 0;
  if (trace_status st = mx_site_size(src_rows, k, &na)) return st;
  const uint64_t nw = (uint64_t)weights * (uint64_t)n * (uint64_t)k, ny = (uint64_t)rows * (uint64_t)n;
  if (nw == 0) return TRACE_OK;
  const size_t need = grad_weight_workspace(rows, groups, n, k);
  if (!grad_w || (rows > 0 && !grad_y) || (need > 0 && !workspace)) return TRACE_E_NULL;
  if (na > 0 && rows > 0 && (!a_scales || !a_codes)) return TRACE_E_NULL;
  if (workspace_bytes < need) return TRACE_E_SHAPE;
  if (!aligned(grad_y, 16) || !aligned(a_codes, 16) || !aligned(grad_w, 16) || !aligned(mask, 2) ||
      !aligned(workspace, 16) || !aligned(row_index, 8))
    return TRACE_E_ALIGN;
  const Range outs[2] = {rng(grad_w, 2 * nw), rng(workspace, need)};
  const Range ins[6] = {rng(grad_y, 2 * ny), rng(a_scales, a_scales ? na / 32 : 0),
                        rng(a_codes, a_codes ? code_bytes(fmt, na) : 0), rng(mask, mask ? nw / 8 : 0),
                        rng(row_index, row_index ? 8 * (uint64_t)rows : 0),
                        rng(offsets, offsets ? 8 * ((uint64_t)weights + 1) : 0)};
  if (trace_status st = check_alias(outs, 2, ins, 6)) return st;
  const trace_host::MxGradArgs p{grad_y, (uint64_t)rows, offsets, (uint32_t)weights, a_codes, a_scales, row_index,
                                 (uint64_t)src_rows, (uint32_t)n, (uint32_t)k, mask, grad_w, false,
                                 static_cast<float*>(workspace)};
  return launch_status(trace_host::launch_mx_grad_weight(fmt, p, static_cast<hipStream_t>(stream)));
}

}  // namespace

static_assert(TRACE_MAX_EXPERTS == trace_host::kMaxExperts, "expert limits differ");
static_assert(TRACE_MAX_TOPK == trace_host::kMaxTopk, "top-k limits differ");

extern "C" {

trace_status trace_mx_quantize(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* scales, uint8_t* codes,
                               uint8_t* mask, void* stream) {
  return quantize(kE2M1, x, rows, cols, scales, codes, mask, stream);
}

trace_status trace_mx8_quantize(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* scales, uint8_t* codes,
                                uint8_t* mask, void* stream) {
  return quantize(kE4M3, x, rows, cols, scales, codes, mask, stream);
}

trace_status trace_mx_matmul(const uint8_t* a_scales, const uint8_t* a_codes, int64_t rows, const uint8_t* w_scales,
                             const uint8_t* w_codes, int64_t n, int64_t k, uint16_t* y, void* stream) {
  return product(kE2M1, nullptr, nullptr, 0, a_scales, a_codes, rows, nullptr, rows, nullptr, 0, w_scales, w_codes, n,
                 k, false, y, false, stream);
}

trace_status trace_mx8_matmul(const uint8_t* a_scales, const uint8_t* a_codes, int64_t rows, const uint8_t* w_scales,
                              const uint8_t* w_codes, int64_t n, int64_t k, uint16_t* y, void* stream) {
  return product(kE4M3, nullptr, nullptr, 0, a_scales, a_codes, rows, nullptr, rows, nullptr, 0, w_scales, w_codes, n,
                 k, false, y, false, stream);
}

trace_status trace_grouped_mx_matmul(const uint8_t* a_scales, const uint8_t* a_codes, int64_t src_rows,
                                     const int64_t* row_index, int64_t rows, const int64_t* offsets, int64_t groups,
                                     const uint8_t* w_scales, const uint8_t* w_codes, int64_t n, int64_t k, uint16_t* y,
                                     void* stream) {
  if (!offsets) return TRACE_E_NULL;
  return product(kE2M1, nullptr, nullptr, 0, a_scales, a_codes, src_rows, row_index, rows, offsets, groups, w_scales,
                 w_codes, n, k, false, y, false, stream);
}

trace_status trace_grouped_mx8_matmul(const uint8_t* a_scales, const uint8_t* a_codes, int64_t src_rows,
                                      const int64_t* row_index, int64_t rows, const int64_t* offsets, int64_t groups,
                                      const uint8_t* w_scales, const uint8_t* w_codes, int64_t n, int64_t k,
                                      uint16_t* y, void* stream) {
  if (!offsets) return TRACE_E_NULL;
  return product(kE4M3, nullptr, nullptr, 0, a_scales, a_codes, src_rows, row_index, rows, offsets, groups, w_scales,
                 w_codes, n, k, false, y, false, stream);
}

size_t trace_mx_linear_workspace_bytes(int64_t src_rows, int64_t rows, int64_t groups, int64_t k) {
  return linear_workspace(kE2M1, src_rows, rows, groups, k);
}

size_t trace_mx8_linear_workspace_bytes(int64_t src_rows, int64_t rows, int64_t groups, int64_t k) {
  return linear_workspace(kE4M3, src_rows, rows, groups, k);
}

trace_status trace_mx_linear(const uint16_t* x, int64_t src_rows, const int64_t* row_index, int64_t rows,
                             const int64_t* offsets, int64_t groups, const uint8_t* w_scales, const uint8_t* w_codes,
                             int64_t n, int64_t k, void* workspace, size_t workspace_bytes, uint16_t* y,
                             void* stream) {
  return product(kE2M1, x, workspace, workspace_bytes, nullptr, nullptr, src_rows, row_index, rows, offsets, groups,
                 w_scales, w_codes, n, k, true, y, false, stream);
}

trace_status trace_mx8_linear(const uint16_t* x, int64_t src_rows, const int64_t* row_index, int64_t rows,
                              const int64_t* offsets, int64_t groups, const uint8_t* w_scales, const uint8_t* w_codes,
                              int64_t n, int64_t k, void* workspace, size_t workspace_bytes, uint16_t* y,
                              void* stream) {
  return product(kE4M3, x, workspace, workspace_bytes, nullptr, nullptr, src_rows, row_index, rows, offsets, groups,
                 w_scales, w_codes, n, k, true, y, false, stream);
}

trace_status trace_grouped_mx_matmul_f32(const uint8_t* a_scales, const uint8_t* a_codes, int64_t src_rows,
                                         const int64_t* row_index, int64_t rows, const int64_t* offsets,
                                         int64_t groups, const uint8_t* w_scales, const uint8_t* w_codes, int64_t n,
                                         int64_t k, float* y, void* stream) {
  if (!offsets) return TRACE_E_NULL;
  return product(kE2M1, nullptr, nullptr, 0, a_scales, a_codes, src_rows, row_index, rows, offsets, groups, w_scales,
                 w_codes, n, k, false, y, true, stream);
}

trace_status trace_grouped_mx_linear_f32(const uint16_t* x, int64_t src_rows, const int64_t* row_index, int64_t rows,
                                         const int64_t* offsets, int64_t groups, const uint8_t* w_scales,
                                         const uint8_t* w_codes, int64_t n, int64_t k, void* workspace,
                                         size_t workspace_bytes, float* y, void* stream) {
  if (!offsets) return TRACE_E_NULL;
  return product(kE2M1, x, workspace, workspace_bytes, nullptr, nullptr, src_rows, row_index, rows, offsets, groups,
                 w_scales, w_codes, n, k, true, y, true, stream);
}

trace_status trace_grouped_mx8_matmul_f32(const uint8_t* a_scales, const uint8_t* a_codes, int64_t src_rows,
                                          const int64_t* row_index, int64_t rows, const int64_t* offsets,
                                          int64_t groups, const uint8_t* w_scales, const uint8_t* w_codes, int64_t n,
                                          int64_t k, float* y, void* stream) {
  if (!offsets) return TRACE_E_NULL;
  return product(kE4M3, nullptr, nullptr, 0, a_scales, a_codes, src_rows, row_index, rows, offsets, groups, w_scales,
                 w_codes, n, k, false, y, true, stream);
}

trace_status trace_grouped_mx8_linear_f32(const uint16_t* x, int64_t src_rows, const int64_t* row_index, int64_t rows,
                                          const int64_t* offsets, int64_t groups, const uint8_t* w_scales,
                                          const uint8_t* w_codes, int64_t n, int64_t k, void* workspace,
                                          size_t workspace_bytes, float* y, void* stream) {
  if (!offsets) return TRACE_E_NULL;
  return product(kE4M3, x, workspace, workspace_bytes, nullptr, nullptr, src_rows, row_index, rows, offsets, groups,
                 w_scales, w_codes, n, k, true, y, true, stream);
}

trace_status trace_mx_matmul_bwd_input(const uint16_t* grad_y, int64_t rows, const int64_t* offsets, int64_t groups,
                                       const uint8_t* w_scales, const uint8_t* w_codes, int64_t n, int64_t k,
                                       const uint8_t* mask, uint16_t* grad_x, void* stream) {
  return grad_input(grad_y, rows, offsets, groups, w_scales, w_codes, n, k, mask, grad_x, false, stream);
}

trace_status trace_grouped_mx_matmul_bwd_input_f32(const uint16_t* grad_y, int64_t rows, const int64_t* offsets,
                                                   int64_t groups, const uint8_t* w_scales, const uint8_t* w_codes,
                                                   int64_t n, int64_t k, const uint8_t* mask, float* grad_x,
                                                   void* stream) {
  if (!offsets) return TRACE_E_NULL;
  return grad_input(grad_y, rows, offsets, groups, w_scales, w_codes, n, k, mask, grad_x, true, stream);
}

size_t trace_mx_matmul_bwd_weight_workspace_bytes(int64_t rows, int64_t groups, int64_t n, int64_t k) {
  return grad_weight_workspace(rows, groups, n, k);
}

trace_status trace_mx_matmul_bwd_weight(const uint16_t* grad_y, int64_t rows, const int64_t* offsets, int64_t groups,
                                        const uint8_t* a_scales, const uint8_t* a_codes, int64_t src_rows,
                                        const int64_t* row_index, int64_t n, int64_t k, const uint8_t* mask,
                                        uint16_t* grad_w, void* workspace, size_t workspace_bytes, void* stream) {
  return grad_weight(kE2M1, grad_y, rows, offsets, groups, a_scales, a_codes, src_rows, row_index, n, k, mask, grad_w,
                     workspace, workspace_bytes, stream);
}

trace_status trace_mx8_matmul_bwd_weight(const uint16_t* grad_y, int64_t rows, const int64_t* offsets, int64_t groups,
                                         const uint8_t* a_scales, const uint8_t* a_codes, int64_t src_rows,
                                         const int64_t* row_index, int64_t n, int64_t k, const uint8_t* mask,
                                         uint16_t* grad_w, void* workspace, size_t workspace_bytes, void* stream) {
  return grad_weight(kE4M3, grad_y, rows, offsets, groups, a_scales, a_codes, src_rows, row_index, n, k, mask, grad_w,
                     workspace, workspace_bytes, stream);
}

// ---------------------------------------------------------------------------
// routed rows
// ---------------------------------------------------------------------------

static bool sort_sizes(int64_t tokens, int64_t topk, int64_t experts) {
  return tokens >= 0 && topk >= 1 && topk <= TRACE_MAX_TOPK && experts >= 1 && experts <= TRACE_MAX_EXPERTS &&
         tokens < kMaxRows && tokens * topk < kMaxRows;
}

size_t trace_expert_sort_workspace_bytes(int64_t tokens, int64_t topk, int64_t experts) {
  if (!sort_sizes(tokens, topk, experts)) return 0;
  return (size_t)trace_host::expert_sort_workspace_words((uint64_t)(tokens * topk), (uint32_t)experts) * sizeof(uint32_t);
}

trace_status trace_expert_sort(const int64_t* ids, int64_t tokens, int64_t topk, int64_t experts, void* workspace,
                               size_t workspace_bytes, int64_t* offsets, int64_t* row_index, int64_t* slot,
                               void* stream) {
  if (!sort_sizes(tokens, topk, experts)) return TRACE_E_SHAPE;
  const uint64_t pairs = (uint64_t)(tokens * topk);
  const size_t need = trace_expert_sort_workspace_bytes(tokens, topk, experts);
  if (!offsets || (pairs > 0 && (!ids || !row_index || !slot)) || (need > 0 && !workspace)) return TRACE_E_NULL;
  if (workspace_bytes < need) return TRACE_E_SHAPE;
  if (!aligned(ids, 8) || !aligned(offsets, 8) || !aligned(row_index, 8) || !aligned(slot, 8) || !aligned(workspace, 4))
    return TRACE_E_ALIGN;
  const Range outs[4] = {rng(offsets, 8 * ((uint64_t)experts + 1)), rng(row_index, 8 * pairs), rng(slot, 8 * pairs),
                         rng(workspace, need)};
  const Range ins[1] = {rng(ids, 8 * pairs)};
  if (trace_status st = check_alias(outs, 4, ins, 1)) return st;
  return hip_status(trace_host::launch_expert_sort(ids, pairs, (uint32_t)topk, (uint32_t)experts,
                                                   static_cast<uint32_t*>(workspace), offsets, row_index, slot,
                                                   static_cast<hipStream_t>(stream)));
}

trace_status trace_expert_dispatch(const uint16_t* x, int64_t tokens, int64_t cols, const int64_t* row_index,
                                   int64_t rows, uint16_t* out, void* stream) {
  uint64_t nx = 0, n = 0;
  if (trace_status st = site_size(tokens, cols, &nx)) return st;
  if (trace_status st = site_size(rows, cols, &n)) return st;
  if (cols >= kMaxDim) return TRACE_E_SHAPE;
  if (n == 0) return TRACE_OK;
  if (!row_index || !out || (nx > 0 && !x)) return TRACE_E_NULL;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(row_index, 8)) return TRACE_E_ALIGN;
  const Range outs[1] = {rng(out, 2 * n)};
  const Range ins[2] = {rng(x, 2 * nx), rng(row_index, 8 * (uint64_t)rows)};
  if (trace_status st = check_alias(outs, 1, ins, 2)) return st;
  return hip_status(trace_host::launch_expert_dispatch(x, (uint64_t)tokens, (uint64_t)cols, row_index, (uint64_t)rows,
                                                       out, static_cast<hipStream_t>(stream)));
}

static trace_status combine(const void* y, bool f32, int64_t rows, int64_t cols, const int64_t* slot, const float* weights,
                            int64_t tokens, int64_t topk, uint16_t* out, void* stream) {
  uint64_t ny = 0, n = 0;
  if (trace_status st = site_size(rows, cols, &ny)) return st;
  if (trace_status st = site_size(tokens, cols, &n)) return st;
  if (!sort_sizes(tokens, topk, 1) || cols >= kMaxDim) return TRACE_E_SHAPE;
  if (n == 0) return TRACE_OK;
  if (!slot || !out || (ny > 0 && !y)) return TRACE_E_NULL;
  if (!aligned(y, 16) || !aligned(out, 16) || !aligned(slot, 8) || !aligned(weights, 4)) return TRACE_E_ALIGN;
  const uint64_t pairs = (uint64_t)(tokens * topk);
  const Range outs[1] = {rng(out, 2 * n)};
  const Range ins[3] = {rng(y, (f32 ? 4 : 2) * ny), rng(slot, 8 * pairs), rng(weights, weights ? 4 * pairs : 0)};
  if (trace_status st = check_alias(outs, 1, ins, 3)) return st;
  return hip_status(trace_host::launch_expert_combine(y, f32, (uint64_t)rows, (uint64_t)cols, slot, weights,
                                                      (uint64_t)tokens, (uint32_t)topk, out,
                                                      static_cast<hipStream_t>(stream)));
}

trace_status trace_expert_combine(const uint16_t* y, int64_t rows, int64_t cols, const int64_t* slot,
                                  const float* weights, int64_t tokens, int64_t topk, uint16_t* out, void* stream) {
  return combine(y, false, rows, cols, slot, weights, tokens, topk, out, stream);
}

trace_status trace_expert_combine_f32(const float* y, int64_t rows, int64_t cols, const int64_t* slot,
                                      const float* weights, int64_t tokens, int64_t topk, uint16_t* out,
                                      void* stream) {
  return combine(y, true, rows, cols, slot, weights, tokens, topk, out, stream);
}

trace_status trace_expert_combine_bwd(const uint16_t* grad_out, const uint16_t* y, int64_t rows, int64_t cols,
                                      const int64_t* slot, const float* weights, int64_t tokens, int64_t topk,
                                      const int64_t* offsets, int64_t groups, uint16_t* grad_y, float* grad_weights,
                                      void* stream) {
  uint64_t ny = 0, n = 0;
  if (trace_status st = site_size(rows, cols, &ny)) return st;
  if (trace_status st = site_size(tokens, cols, &n)) return st;
  if (!sort_sizes(tokens, topk, 1) || cols >= kMaxDim || rows >= kMaxRows) return TRACE_E_SHAPE;
  int64_t count = 0;
  if (trace_status st = product_groups(offsets, groups, &count)) return st;
  if (offsets && (groups < 1 || groups > kMaxProductGroups)) return TRACE_E_SHAPE;
  const uint64_t pairs = (uint64_t)(tokens * topk);
  if (pairs == 0 && (ny == 0 || !offsets)) return TRACE_OK;
  if (pairs > 0 && (!slot || !grad_weights || (n > 0 && !grad_out))) return TRACE_E_NULL;
  if (ny > 0 && (!y || !grad_y)) return TRACE_E_NULL;
  if (!aligned(grad_out, 16) || !aligned(y, 16) || !aligned(grad_y, 16) || !aligned(slot, 8) || !aligned(weights, 4) ||
      !aligned(grad_weights, 4))
    return TRACE_E_ALIGN;
  const Range outs[2] = {rng(grad_y, 2 * ny), rng(grad_weights, 4 * pairs)};
  const Range ins[5] = {rng(grad_out, 2 * n), rng(y, 2 * ny), rng(slot, 8 * pairs), rng(weights, weights ? 4 * pairs : 0),
                        rng(offsets, offsets ? 8 * ((uint64_t)groups + 1) : 0)};
  if (trace_status st = check_alias(outs, 2, ins, 5)) return st;
  return hip_status(trace_host::launch_expert_combine_bwd(grad_out, y, (uint64_t)rows, (uint64_t)cols, slot, weights,
                                                          (uint64_t)tokens, (uint32_t)topk, offsets != nullptr, grad_y,
                                                          grad_weights, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
