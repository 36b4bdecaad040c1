// C ABI of the vocabulary loss, the router and the optimiser step: argument
// validation and dispatch to the HIP launchers, as in api.cpp.
#include "trace.h"

#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>
#include <new>

#include "api_checks.h"
#include "launch_step.h"

using namespace trace_api;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxDim = (int64_t)1 << 20;  // a tile's rows are addressed in 32 bits

trace_status launch_status(hipError_t e) { return e == hipErrorInvalidConfiguration ? TRACE_E_SHAPE : hip_status(e); }

// ---------------------------------------------------------------------------
// the vocabulary loss
// ---------------------------------------------------------------------------

trace_status loss_sizes(int64_t tokens, int64_t vocab, int64_t k) {
  if (tokens < 0 || tokens >= kMaxRows || vocab < 1 || vocab >= kMaxRows - 256) return TRACE_E_SHAPE;
  return k < 32 || k >= kMaxDim || k % 32 != 0 ? TRACE_E_SHAPE : TRACE_OK;
}

trace_host::CrossEntropyArgs loss_args(const uint16_t* x, const uint16_t* w, const int64_t* targets, int64_t tokens,
                                       int64_t vocab, int64_t k, float scale, void* workspace) {
  return {x, w, targets, (uint64_t)tokens, (uint32_t)vocab, (uint32_t)k, scale, workspace};
}

// ---------------------------------------------------------------------------
// the router
// ---------------------------------------------------------------------------

trace_status route_sizes(int64_t tokens, int64_t experts, int64_t topk) {
  if (experts < 1 || experts > trace_host::kMaxRouted || topk < 1 || topk > 64 || topk > experts) return TRACE_E_SHAPE;
  return tokens < 0 || tokens >= kMaxRows / topk ? TRACE_E_SHAPE : TRACE_OK;
}

trace_status route(const void* logits, bool bf16, const uint8_t* valid, int64_t tokens, int64_t experts, int64_t topk,
                   int renormalize, void* workspace, size_t workspace_bytes, int64_t* ids, float* weights,
                   int64_t* counts, float* probs, float* balance, void* stream) {
  if (trace_status st = route_sizes(tokens, experts, topk)) return st;
  const uint64_t need = trace_host::route_workspace_bytes((uint64_t)tokens, (uint32_t)experts);
  const uint64_t pairs = (uint64_t)(tokens * topk), e = (uint64_t)experts;
  if (!counts || !probs || !balance || (tokens > 0 && (!logits || !ids || !weights)) || (need > 0 && !workspace))
    return TRACE_E_NULL;
  if (workspace_bytes < need) return TRACE_E_SHAPE;
  if (!aligned(logits, bf16 ? 2 : 4) || !aligned(ids, 8) || !aligned(weights, 4) || !aligned(counts, 8) ||
      !aligned(probs, 4) || !aligned(balance, 4) || !aligned(workspace, 16))
    return TRACE_E_ALIGN;
  const Range outs[6] = {rng(ids, 8 * pairs), rng(weights, 4 * pairs), rng(counts, 8 * (e + 1)),
                         rng(probs, 4 * e),   rng(balance, 4),         rng(workspace, need)};
  const Range ins[2] = {rng(logits, (bf16 ? 2 : 4) * (uint64_t)tokens * e), rng(valid, valid ? (uint64_t)tokens : 0)};
  if (trace_status st = check_alias(outs, 6, ins, 2)) return st;
  const trace_host::RouteArgs p{logits, bf16, (uint64_t)tokens, (uint32_t)experts, (uint32_t)topk, renormalize != 0};
  return launch_status(trace_host::launch_route(p, valid, workspace, ids, weights, counts, probs, balance,
                                                static_cast<hipStream_t>(stream)));
}

trace_status route_bwd(const float* grad_weights, const float* grad_balance, const void* logits, bool bf16,
                       const int64_t* ids, const float* weights, const int64_t* counts, int64_t tokens,
                       int64_t experts, int64_t topk, int renormalize, void* grad_logits, void* stream) {
  if (trace_status st = route_sizes(tokens, experts, topk)) return st;
  if (tokens == 0) return TRACE_OK;
  if (!logits || !ids || !weights || !counts || !grad_logits) return TRACE_E_NULL;
  const uint64_t pairs = (uint64_t)(tokens * topk), e = (uint64_t)experts, each = bf16 ? 2 : 4;
  if (!aligned(logits, each) || !aligned(grad_logits, each) || !aligned(ids, 8) || !aligned(weights, 4) ||
      !aligned(counts, 8) || !aligned(grad_weights, 4) || !aligned(grad_balance, 4))
    return TRACE_E_ALIGN;
  const Range outs[1] = {rng(grad_logits, each * (uint64_t)tokens * e)};
  const Range ins[6] = {rng(logits, each * (uint64_t)tokens * e),
                        rng(ids, 8 * pairs),
                        rng(weights, 4 * pairs),
                        rng(counts, 8 * (e + 1)),
                        rng(grad_weights, grad_weights ? 4 * pairs : 0),
                        rng(grad_balance, grad_balance ? 4 : 0)};
  if (trace_status st = check_alias(outs, 1, ins, 6, 0, 0)) return st;  // in place of the logits: each row is read first
  const trace_host::RouteArgs p{logits, bf16, (uint64_t)tokens, (uint32_t)experts, (uint32_t)topk, renormalize != 0};
  return launch_status(trace_host::launch_route_bwd(p, grad_weights, grad_balance, ids, weights, counts, grad_logits,
                                                    static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------------------
// the optimiser step
// ---------------------------------------------------------------------------

constexpr int32_t kMaxTensors = 1 << 20;

struct Span {
  uintptr_t lo, hi;
  bool written;
};

// Whether something that is written overlaps anything else.  `runs` runs of
// `each` spans (the tensors' params, their grads, ...), in ascending order as a rule
// where the tensors are parts of larger ones.
bool spans_clash(Span* s, size_t runs, size_t each) {
  const auto before = [](const Span& a, const Span& b) { return a.lo < b.lo; };
  for (size_t r = 0; r < runs; ++r) {
    Span* const run = s + r * each;
    if (!std::is_sorted(run, run + each, before)) std::sort(run, run + each, before);
  }
  uintptr_t any = 0, written = 0;  // how far what came before reaches
  size_t at[8] = {};
  for (;;) {
    size_t best = runs;
    for (size_t r = 0; r < runs; ++r)
      if (at[r] < each && (best == runs || s[r * each + at[r]].lo < s[best * each + at[best]].lo)) best = r;
    if (best == runs) return false;
    const Span& x = s[best * each + at[best]++];
    if (x.hi == x.lo) continue;
    if (x.lo < written || (x.written && x.lo < any)) return true;
    any = std::max(any, x.hi);
    if (x.written) written = std::max(written, x.hi);
  }
}

trace_status adamw(const trace_adamw_tensor* tensors, int32_t count, const trace_adamw_options* o,
                   const float* grad_scale, void* stream) {
  if (count < 0 || count > kMaxTensors) return TRACE_E_SHAPE;
  if (!o || (count > 0 && !tensors)) return TRACE_E_NULL;
  if (o->step < 1 || !(o->beta1 >= 0 && o->beta1 < 1) || !(o->beta2 >= 0 && o->beta2 < 1) || !(o->eps >= 0) ||
      !isfinite(o->eps) || !isfinite(o->lr) || !isfinite(o->weight_decay))
    return TRACE_E_SHAPE;
  const bool mx8 = o->states_mx8 != 0;
  const uint64_t param = o->param_bf16 ? 2 : 4, grad = o->grad_bf16 ? 2 : 4, state = mx8 ? 1 : 4;
  if (!aligned(grad_scale, 4)) return TRACE_E_ALIGN;
  uint64_t all = 0;
  for (int32_t i = 0; i < count; ++i) {
    const trace_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > ((int64_t)1 << 48)) return TRACE_E_SHAPE;
    if (t.n == 0) continue;
    all += (uint64_t)t.n;
    if (all > (1ull << 48)) return TRACE_E_SHAPE;
    if (!t.param || !t.grad || !t.avg || !t.sq || (mx8 && (!t.avg_scales || !t.sq_scales))) return TRACE_E_NULL;
    if (t.copy && o->param_bf16) return TRACE_E_SHAPE;
    if (!aligned(t.param, 16) || !aligned(t.grad, 16) || !aligned(t.avg, mx8 ? 8 : 16) ||
        !aligned(t.sq, mx8 ? 8 : 16) || !aligned(t.copy, 16))
      return TRACE_E_ALIGN;
  }
  if (all == 0) return TRACE_OK;
  constexpr size_t kRuns = 7;
  Span few[kRuns * 16];
  const size_t each = (size_t)count;
  Span* const spans = each > 16 ? new (std::nothrow) Span[kRuns * each] : few;
  if (!spans) return hip_status(hipErrorOutOfMemory);
  for (size_t i = 0; i < each; ++i) {
    const trace_adamw_tensor& t = tensors[i];
    const uint64_t e = (uint64_t)t.n;
    const auto put = [&](size_t run, const void* p, uint64_t bytes, bool written) {
      spans[run * each + i] = Span{(uintptr_t)p, p ? (uintptr_t)p + bytes : 0, written};
    };
    put(0, t.param, param * e, true);
    put(1, t.grad, grad * e, false);
    put(2, t.avg, state * e, true);
    put(3, t.sq, state * e, true);
    put(4, t.copy, 2 * e, true);
    put(5, mx8 ? t.avg_scales : nullptr, (e + 31) / 32, true);
    put(6, mx8 ? t.sq_scales : nullptr, (e + 31) / 32, true);
  }
  bool clash = spans_clash(spans, mx8 ? kRuns : kRuns - 2, each);
  const uintptr_t scale_at = (uintptr_t)grad_scale;
  for (size_t i = 0; grad_scale && i < kRuns * each; ++i)
    clash |= spans[i].written && spans[i].lo < scale_at + 4 && scale_at < spans[i].hi;
  if (spans != few) delete[] spans;
  if (clash) return TRACE_E_ALIAS;
  const double rest1 = 1 - pow(o->beta1, (double)o->step), rest2 = 1 - pow(o->beta2, (double)o->step);
  trace_host::AdamwScalars s{};
  s.beta1 = (float)o->beta1;
  s.rest1 = (float)(1 - o->beta1);
  s.beta2 = (float)o->beta2;
  s.rest2 = (float)(1 - o->beta2);
  s.eps = (float)o->eps;
  s.decay = (float)(1 - o->lr * o->weight_decay);
  s.rate = (float)(o->lr / rest1);
  s.root = (float)(1 / sqrt(rest2));
  s.key = trace_host::mix_bits(trace_host::mix_bits((uint32_t)o->seed) + (uint32_t)(o->seed >> 32));
  const trace_host::AdamwTypes types{o->param_bf16 != 0, o->grad_bf16 != 0, mx8, o->randomly != 0};
  static_assert(sizeof(trace_host::AdamwTensor) == sizeof(trace_adamw_tensor), "the same layout");
  return launch_status(trace_host::launch_adamw(reinterpret_cast<const trace_host::AdamwTensor*>(tensors),
                                                (uint32_t)count, types, s, grad_scale,
                                                static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int trace_step_revision(void) { return TRACE_STEP_REVISION; }

size_t trace_linear_cross_entropy_workspace_bytes(int64_t tokens, int64_t vocab, int64_t k) {
  if (loss_sizes(tokens, vocab, k) != TRACE_OK || tokens == 0) return 0;
  return (size_t)trace_host::cross_entropy_workspace_bytes((uint64_t)tokens, (uint32_t)vocab, (uint32_t)k);
}

trace_status trace_linear_cross_entropy(const uint16_t* x, const uint16_t* w, const int64_t* targets, int64_t tokens,
                                        int64_t vocab, int64_t k, float scale, void* workspace,
                                        size_t workspace_bytes, float* loss, float* lse, void* stream) {
  if (trace_status st = loss_sizes(tokens, vocab, k)) return st;
  if (tokens == 0) return TRACE_OK;
  const size_t need = trace_linear_cross_entropy_workspace_bytes(tokens, vocab, k);
  if (!x || !w || !targets || !workspace || !loss || !lse) return TRACE_E_NULL;
  if (workspace_bytes < need) return TRACE_E_SHAPE;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(targets, 8) || !aligned(workspace, 16) || !aligned(loss, 4) ||
      !aligned(lse, 4))
    return TRACE_E_ALIGN;
  const uint64_t t = (uint64_t)tokens;
  const Range outs[3] = {rng(loss, 4 * t), rng(lse, 4 * t), rng(workspace, need)};
  const Range ins[3] = {rng(x, 2 * t * (uint64_t)k), rng(w, 2 * (uint64_t)vocab * (uint64_t)k), rng(targets, 8 * t)};
  if (trace_status st = check_alias(outs, 3, ins, 3)) return st;
  return launch_status(trace_host::launch_cross_entropy(loss_args(x, w, targets, tokens, vocab, k, scale, workspace),
                                                        loss, lse, static_cast<hipStream_t>(stream)));
}

size_t trace_linear_cross_entropy_bwd_workspace_bytes(int64_t tokens, int64_t vocab, int64_t k) {
  if (loss_sizes(tokens, vocab, k) != TRACE_OK || tokens == 0) return 0;
  return (size_t)trace_host::cross_entropy_bwd_workspace_bytes((uint64_t)tokens, (uint32_t)vocab, (uint32_t)k);
}

trace_status trace_linear_cross_entropy_bwd(const float* grad_loss, const uint16_t* x, const uint16_t* w,
                                            const int64_t* targets, const float* lse, int64_t tokens, int64_t vocab,
                                            int64_t k, float scale, void* workspace, size_t workspace_bytes,
                                            uint16_t* grad_x, uint16_t* grad_w, void* stream) {
  if (trace_status st = loss_sizes(tokens, vocab, k)) return st;
  if (tokens == 0 && !grad_w) return TRACE_OK;
  const size_t need = trace_linear_cross_entropy_bwd_workspace_bytes(tokens, vocab, k);
  if (tokens > 0 && (!grad_loss || !x || !w || !targets || !lse || !workspace)) return TRACE_E_NULL;
  if (!grad_x && !grad_w) return TRACE_OK;
  if (workspace_bytes < need) return TRACE_E_SHAPE;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(targets, 8) || !aligned(workspace, 16) ||
      !aligned(grad_loss, 4) || !aligned(lse, 4) || !aligned(grad_x, 16) || !aligned(grad_w, 16))
    return TRACE_E_ALIGN;
  const uint64_t t = (uint64_t)tokens, nx = t * (uint64_t)k, nw = (uint64_t)vocab * (uint64_t)k;
  const Range outs[3] = {rng(grad_x, grad_x ? 2 * nx : 0), rng(grad_w, grad_w ? 2 * nw : 0), rng(workspace, need)};
  const Range ins[5] = {rng(grad_loss, 4 * t), rng(x, 2 * nx), rng(w, t ? 2 * nw : 0), rng(targets, 8 * t),
                        rng(lse, 4 * t)};
  if (trace_status st = check_alias(outs, 3, ins, 5)) return st;
  return launch_status(trace_host::launch_cross_entropy_bwd(
      loss_args(x, w, targets, tokens, vocab, k, scale, workspace), grad_loss, lse, grad_x, grad_w,
      static_cast<hipStream_t>(stream)));
}

size_t trace_expert_route_workspace_bytes(int64_t tokens, int64_t experts) {
  if (route_sizes(tokens, experts, 1) != TRACE_OK) return 0;
  return (size_t)trace_host::route_workspace_bytes((uint64_t)tokens, (uint32_t)experts);
}

trace_status trace_expert_route(const uint16_t* logits, const uint8_t* valid, int64_t tokens, int64_t experts,
                                int64_t topk, int renormalize, void* workspace, size_t workspace_bytes, int64_t* ids,
                                float* weights, int64_t* counts, float* probs, float* balance, void* stream) {
  return route(logits, true, valid, tokens, experts, topk, renormalize, workspace, workspace_bytes, ids, weights,
               counts, probs, balance, stream);
}

trace_status trace_expert_route_f32(const float* logits, const uint8_t* valid, int64_t tokens, int64_t experts,
                                    int64_t topk, int renormalize, void* workspace, size_t workspace_bytes,
                                    int64_t* ids, float* weights, int64_t* counts, float* probs, float* balance,
                                    void* stream) {
  return route(logits, false, valid, tokens, experts, topk, renormalize, workspace, workspace_bytes, ids, weights,
               counts, probs, balance, stream);
}

trace_status trace_expert_route_bwd(const float* grad_weights, const float* grad_balance, const uint16_t* logits,
                                    const int64_t* ids, const float* weights, const int64_t* counts, int64_t tokens,
                                    int64_t experts, int64_t topk, int renormalize, uint16_t* grad_logits,
                                    void* stream) {
  return route_bwd(grad_weights, grad_balance, logits, true, ids, weights, counts, tokens, experts, topk, renormalize,
                   grad_logits, stream);
}

trace_status trace_expert_route_bwd_f32(const float* grad_weights, const float* grad_balance, const float* logits,
                                        const int64_t* ids, const float* weights, const int64_t* counts,
                                        int64_t tokens, int64_t experts, int64_t topk, int renormalize,
                                        float* grad_logits, void* stream) {
  return route_bwd(grad_weights, grad_balance, logits, false, ids, weights, counts, tokens, experts, topk, renormalize,
                   grad_logits, stream);
}

trace_status trace_adamw_step(const trace_adamw_tensor* tensors, int32_t count, const trace_adamw_options* options,
                              const float* grad_scale, void* stream) {
  return adamw(tensors, count, options, grad_scale, stream);
}

}  // extern "C"
