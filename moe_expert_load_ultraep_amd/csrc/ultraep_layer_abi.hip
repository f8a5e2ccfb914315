// C ABI of the steps around the experts: argument checks and launches.  See
// include/ultraep_layer.h for the contract of every entry point.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "ultraep_internal.h"
#include "ultraep_layer.h"

namespace {

using ultraep::aligned;
using ultraep::from_hip;

constexpr int64_t kMaxRows = int64_t{1} << 31;
constexpr int32_t kMaxGluWidth = 1 << 22;

bool bad_type(int32_t t) { return t != ULTRAEP_TYPE_F32 && t != ULTRAEP_TYPE_BF16; }
bool bad_flag(int32_t f) { return f != 0 && f != 1; }
bool half_given(const void* a, const void* b) { return (a == nullptr) != (b == nullptr); }

// Shared checks of both directions of the routing.
int route_checks(const ultraep_ctx* ctx, const ultraep::RouteArgs& a, int32_t type, int32_t score, int32_t renorm,
                 const int32_t* idx, const float* w) {
  if (!ctx || a.tokens < 0 || (a.tokens > 0 && (!a.logits || !idx || !w))) return ULTRAEP_EINVAL;
  if (a.k < 1 || a.k > a.E || a.k > ULTRAEP_MAX_TOPK || bad_type(type) || bad_flag(renorm) ||
      (score != ULTRAEP_ROUTE_SOFTMAX && score != ULTRAEP_ROUTE_SIGMOID) || !std::isfinite(a.scale))
    return ULTRAEP_EINVAL;
  if (a.groups < 1 || a.E % a.groups != 0 || a.topk_groups < 1 || a.topk_groups > a.groups || a.group_top < 1 ||
      a.group_top > 2)
    return ULTRAEP_EINVAL;
  if (a.groups > ULTRAEP_MAX_ROUTE_GROUPS || a.tokens >= kMaxRows || !aligned(a.logits, a.bf16 ? 2 : 4) ||
      !aligned(a.bias, 4) || !aligned(idx, 4) || !aligned(w, 4))
    return ULTRAEP_EUNSUPPORTED;
  return ULTRAEP_OK;
}

// Shared checks of both directions of the norm.
int norm_checks(int64_t rows, int32_t H, int32_t stream_type, int32_t weight_type) {
  if (rows < 0 || H <= 0 || bad_type(stream_type) || bad_type(weight_type)) return ULTRAEP_EINVAL;
  if (H % 8 != 0 || H > ULTRAEP_MAX_NORM_WIDTH || rows >= kMaxRows) return ULTRAEP_EUNSUPPORTED;
  return ULTRAEP_OK;
}

// Shared by both directions of the gated activation (back: grad is wanted; W: columns
// of the results).
int glu(const ultraep_ctx* ctx, const void* plan, const uint16_t* h, const uint16_t* grad, bool back, int32_t F,
        int32_t activation, int32_t p_begin, int32_t p_end, uint8_t* q, uint8_t* q_scale, uint8_t* qt, uint8_t* qt_scale,
        int64_t capacity_rows, int64_t capacity_blocks, void* stream) {
  if (!ctx || !plan || F <= 0 || capacity_rows < 0 || p_begin < 0 || p_end < p_begin || p_end > ctx->sh.P) return ULTRAEP_EINVAL;
  if (activation != ULTRAEP_GLU_SILU && activation != ULTRAEP_GLU_GELU) return ULTRAEP_EINVAL;
  const bool idle = capacity_rows == 0 || p_begin == p_end;  // nothing is read or written, buffers need no address
  if (!idle && (!h || (back && !grad) || half_given(q, q_scale) || half_given(qt, qt_scale) || (!q && !qt))) return ULTRAEP_EINVAL;
  if (qt && capacity_blocks < capacity_rows / ULTRAEP_QUANT_BLOCK + (p_end - p_begin)) return ULTRAEP_EINVAL;
  if (F % 8 != 0 || F > kMaxGluWidth || capacity_rows >= kMaxRows || !aligned(plan, 4) || !aligned(h, 16) ||
      !aligned(grad, 16) || !aligned(q, 16) || !aligned(q_scale, 4) || !aligned(qt, 16))
    return ULTRAEP_EUNSUPPORTED;
  const int32_t* off = static_cast<const int32_t*>(plan) + ctx->sh.lay.off[ULTRAEP_PLAN_PHYS_OFF] + p_begin;
  return from_hip(ultraep::launch_glu_quant(off, p_end - p_begin, h, grad, F, activation == ULTRAEP_GLU_GELU, q, q_scale, qt,
                                            qt_scale, capacity_rows, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int ultraep_route(const ultraep_ctx* ctx, const void* logits, int32_t logits_type, int64_t tokens,
                  int32_t k, int32_t score, const float* bias, int32_t groups, int32_t topk_groups,
                  int32_t group_top, int32_t renormalize, float scale, int32_t* topk_idx,
                  float* topk_w, void* stream) {
  const ultraep::RouteArgs a{logits, logits_type == ULTRAEP_TYPE_BF16, tokens, ctx ? ctx->sh.E : 0, k,
                             score == ULTRAEP_ROUTE_SIGMOID, bias, groups, topk_groups, group_top, renormalize == 1, scale};
  const int st = route_checks(ctx, a, logits_type, score, renormalize, topk_idx, topk_w);
  if (st != ULTRAEP_OK) return st;
  return from_hip(ultraep::launch_route(a, topk_idx, topk_w, static_cast<hipStream_t>(stream)));
}

int ultraep_route_backward(const ultraep_ctx* ctx, const void* logits, int32_t logits_type,
                           int64_t tokens, int32_t k, int32_t score, int32_t renormalize, float scale,
                           const int32_t* topk_idx, const float* grad_topk_w, void* grad_logits,
                           void* stream) {
  const ultraep::RouteArgs a{logits, logits_type == ULTRAEP_TYPE_BF16, tokens, ctx ? ctx->sh.E : 0, k,
                             score == ULTRAEP_ROUTE_SIGMOID, nullptr, 1, 1, 1, renormalize == 1, scale};
  const int st = route_checks(ctx, a, logits_type, score, renormalize, topk_idx, grad_topk_w);
  if (st != ULTRAEP_OK) return st;
  if (tokens > 0 && !grad_logits) return ULTRAEP_EINVAL;
  if (!aligned(grad_logits, a.bf16 ? 2 : 4)) return ULTRAEP_EUNSUPPORTED;
  return from_hip(ultraep::launch_route_backward(a, topk_idx, grad_topk_w, grad_logits, static_cast<hipStream_t>(stream)));
}

int ultraep_residual_norm(const ultraep_ctx* ctx, const uint16_t* x, const void* residual,
                          int32_t residual_type, const void* weight, int32_t weight_type, float eps,
                          int64_t rows, int32_t H, void* h, uint16_t* y, uint8_t* q, uint8_t* q_scale,
                          float* rstd, void* stream) {
  const int st = norm_checks(rows, H, residual_type, weight_type);
  if (!ctx || st == ULTRAEP_EINVAL) return ULTRAEP_EINVAL;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return ULTRAEP_EINVAL;
  if (rows > 0 && (!x || !weight || (h && !residual) || half_given(q, q_scale) || (!h && !y && !q && !rstd))) return ULTRAEP_EINVAL;
  if (st != ULTRAEP_OK || !aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(h, 16) ||
      !aligned(y, 16) || !aligned(q, 16) || !aligned(q_scale, 4) || !aligned(rstd, 4))
    return ULTRAEP_EUNSUPPORTED;
  return from_hip(ultraep::launch_norm({rows, H, weight, weight_type == ULTRAEP_TYPE_BF16}, x, residual,
                                       residual_type == ULTRAEP_TYPE_BF16, eps, h, y, q, q_scale, rstd,
                                       static_cast<hipStream_t>(stream)));
}

int ultraep_residual_norm_workspace_bytes(int64_t rows, int32_t H, size_t* out) {
  if (!out) return ULTRAEP_EINVAL;
  const int st = norm_checks(rows, H, ULTRAEP_TYPE_F32, ULTRAEP_TYPE_F32);
  if (st != ULTRAEP_OK) return st;
  *out = ultraep::norm_workspace_bytes(rows, H);
  return ULTRAEP_OK;
}

int ultraep_residual_norm_backward(const ultraep_ctx* ctx, const uint16_t* grad_y, const void* h,
                                   int32_t h_type, const void* weight, int32_t weight_type,
                                   const float* rstd, const void* grad_in, int64_t rows, int32_t H,
                                   void* grad_h, uint16_t* grad_x, float* grad_weight,
                                   int32_t accumulate, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  const int st = norm_checks(rows, H, h_type, weight_type);
  if (!ctx || st == ULTRAEP_EINVAL) return ULTRAEP_EINVAL;
  if (bad_flag(accumulate) || (grad_x && h_type == ULTRAEP_TYPE_BF16)) return ULTRAEP_EINVAL;
  if (rows > 0 && (!grad_y || !h || !weight || !rstd || !grad_h || (grad_weight && !workspace))) return ULTRAEP_EINVAL;
  if (st != ULTRAEP_OK || !aligned(grad_y, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(rstd, 4) ||
      !aligned(grad_in, 16) || !aligned(grad_h, 16) || !aligned(grad_x, 16) || !aligned(grad_weight, 16) ||
      (grad_weight && !aligned(workspace, 16)))
    return ULTRAEP_EUNSUPPORTED;
  if (grad_weight && rows > 0 && workspace_bytes < ultraep::norm_workspace_bytes(rows, H)) return ULTRAEP_EWORKSPACE;
  return from_hip(ultraep::launch_norm_backward({rows, H, weight, weight_type == ULTRAEP_TYPE_BF16}, grad_y, h,
                                                h_type == ULTRAEP_TYPE_BF16, rstd, grad_in, grad_h, grad_x, grad_weight,
                                                accumulate != 0, static_cast<float*>(workspace),
                                                static_cast<hipStream_t>(stream)));
}

int ultraep_glu_quant(const ultraep_ctx* ctx, const void* plan, const uint16_t* h, int32_t F,
                      int32_t activation, int32_t p_begin, int32_t p_end, uint8_t* q,
                      uint8_t* q_scale, uint8_t* qt, uint8_t* qt_scale, int64_t capacity_rows,
                      int64_t capacity_blocks, void* stream) {
  return glu(ctx, plan, h, nullptr, false, F, activation, p_begin, p_end, q, q_scale, qt, qt_scale, capacity_rows,
             capacity_blocks, stream);
}

int ultraep_glu_quant_backward(const ultraep_ctx* ctx, const void* plan, const uint16_t* h,
                               const uint16_t* grad, int32_t F, int32_t activation, int32_t p_begin,
                               int32_t p_end, uint8_t* q, uint8_t* q_scale, uint8_t* qt,
                               uint8_t* qt_scale, int64_t capacity_rows, int64_t capacity_blocks,
                               void* stream) {
  return glu(ctx, plan, h, grad, true, F, activation, p_begin, p_end, q, q_scale, qt, qt_scale, capacity_rows,
             capacity_blocks, stream);
}

}  // extern "C"
