// C ABI of the experts' steps: argument checks and launches.  See
// include/ultraep_experts.h for the contract of every entry point.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ultraep_experts.h"
#include "ultraep_internal.h"

namespace {

using ultraep::aligned;
using ultraep::from_hip;

constexpr int32_t kMaxWidth = 1 << 20;        // N and K of the products
constexpr int32_t kMaxRowWidth = 1 << 24;     // H of the quantiser
constexpr int64_t kMaxRows = int64_t{1} << 31;

constexpr int64_t kMaxTiles = 1 << 23;        // workgroups of a product

bool too_many_tiles(int64_t rows, int32_t groups, int32_t width) {
  return (rows / 256 + groups) * ((width + 255) / 256) > kMaxTiles;
}

bool bad_range(const ultraep_ctx* ctx, int32_t p_begin, int32_t p_end) {
  return p_begin < 0 || p_end < p_begin || p_end > ctx->sh.P;
}

const int32_t* segment(const ultraep_ctx* ctx, const void* plan, int32_t p_begin) {
  return static_cast<const int32_t*>(plan) + ctx->sh.lay.off[ULTRAEP_PLAN_PHYS_OFF] + p_begin;
}

bool half_given(const void* a, const void* b) { return (a == nullptr) != (b == nullptr); }

// No rows, or no experts to have any: nothing is read or written, and the
// buffers, having no elements, need no address.
bool idle(int64_t rows, int32_t p_begin, int32_t p_end) { return rows == 0 || p_begin == p_end; }

}  // namespace

extern "C" {

int ultraep_permute_quant(const ultraep_ctx* ctx, const void* plan, const int32_t* inv, int32_t k,
                          const uint16_t* hidden, int64_t hidden_rows, int32_t H, int32_t p_begin,
                          int32_t p_end, uint8_t* q, uint8_t* q_scale, uint8_t* qt,
                          uint8_t* qt_scale, int64_t capacity_rows, int64_t capacity_blocks,
                          void* stream) {
  if (!ctx || !plan || (!hidden && hidden_rows > 0)) return ULTRAEP_EINVAL;
  if (!idle(capacity_rows, p_begin, p_end) && (half_given(q, q_scale) || half_given(qt, qt_scale) || (!q && !qt)))
    return ULTRAEP_EINVAL;
  if (H <= 0 || hidden_rows < 0 || capacity_rows < 0 || bad_range(ctx, p_begin, p_end)) return ULTRAEP_EINVAL;
  if (inv && (k < 1 || k > ULTRAEP_MAX_TOPK)) return ULTRAEP_EINVAL;
  if (qt && capacity_blocks < capacity_rows / ULTRAEP_QUANT_BLOCK + (p_end - p_begin)) return ULTRAEP_EINVAL;
  if (H % 8 != 0 || H > kMaxRowWidth || capacity_rows >= kMaxRows || !aligned(plan, 4) || !aligned(inv, 4) ||
      !aligned(hidden, 16) || !aligned(q, 16) || !aligned(q_scale, 4) || !aligned(qt, 16))
    return ULTRAEP_EUNSUPPORTED;
  return from_hip(ultraep::launch_permute_quant(segment(ctx, plan, p_begin), p_end - p_begin, inv, inv ? k : 1,
                                                hidden, hidden_rows, H, q, q_scale, qt, qt_scale,
                                                capacity_rows, static_cast<hipStream_t>(stream)));
}

int ultraep_weight_quant(const ultraep_ctx* ctx, const uint16_t* const* weights, int32_t n,
                         int32_t N, int32_t K, uint8_t* q, uint8_t* q_scale, uint8_t* qt,
                         uint8_t* qt_scale, void* stream) {
  if (!ctx || n < 0 || N <= 0 || K <= 0 || (n > 0 && !weights)) return ULTRAEP_EINVAL;
  if (n > 0 && (half_given(q, q_scale) || half_given(qt, qt_scale) || (!q && !qt))) return ULTRAEP_EINVAL;
  if (N % 8 != 0 || K % 8 != 0 || N > kMaxWidth || K > kMaxWidth || n > ULTRAEP_MAX_EXPERTS ||
      !aligned(weights, 8) || !aligned(q, 16) || !aligned(qt, 16) || !aligned(q_scale, 4) ||
      !aligned(qt_scale, 4))
    return ULTRAEP_EUNSUPPORTED;
  return from_hip(ultraep::launch_weight_quant(weights, n, N, K, q, q_scale, qt, qt_scale,
                                               static_cast<hipStream_t>(stream)));
}

int ultraep_expert_gemm(const ultraep_ctx* ctx, const void* plan, const uint8_t* q,
                        const uint8_t* q_scale, int32_t K, const uint8_t* const* w,
                        const uint8_t* const* w_scale, int32_t N, int32_t p_begin, int32_t p_end,
                        uint16_t* out, int64_t capacity_rows, void* stream) {
  if (!ctx || !plan) return ULTRAEP_EINVAL;
  if (!idle(capacity_rows, p_begin, p_end) && (!q || !q_scale || !w || !w_scale || !out)) return ULTRAEP_EINVAL;
  if (N <= 0 || K <= 0 || capacity_rows < 0 || bad_range(ctx, p_begin, p_end)) return ULTRAEP_EINVAL;
  if (N % 8 != 0 || N > kMaxWidth || K > kMaxWidth || capacity_rows >= kMaxRows || !aligned(plan, 4) ||
      !aligned(q, 16) || !aligned(q_scale, 4) || !aligned(w, 8) || !aligned(w_scale, 8) || !aligned(out, 16) ||
      too_many_tiles(capacity_rows, p_end - p_begin, N))
    return ULTRAEP_EUNSUPPORTED;
  return from_hip(ultraep::launch_expert_gemm(segment(ctx, plan, p_begin), p_end - p_begin, q, q_scale, K, w,
                                              w_scale, N, out, capacity_rows,
                                              static_cast<hipStream_t>(stream)));
}

int ultraep_expert_wgrad(const ultraep_ctx* ctx, const void* plan, const uint8_t* dyt,
                         const uint8_t* dyt_scale, int32_t N, const uint8_t* xt,
                         const uint8_t* xt_scale, int32_t K, int32_t p_begin, int32_t p_end,
                         int64_t capacity_rows, float* const* grads, int32_t accumulate,
                         void* stream) {
  if (!ctx || !plan) return ULTRAEP_EINVAL;
  if (p_begin != p_end && (!dyt || !dyt_scale || !xt || !xt_scale || !grads)) return ULTRAEP_EINVAL;
  if (N <= 0 || K <= 0 || capacity_rows < 0 || bad_range(ctx, p_begin, p_end)) return ULTRAEP_EINVAL;
  if (accumulate != 0 && accumulate != 1) return ULTRAEP_EINVAL;
  if (N % 8 != 0 || K % 8 != 0 || N > kMaxWidth || K > kMaxWidth || capacity_rows >= kMaxRows ||
      !aligned(plan, 4) || !aligned(dyt, 16) || !aligned(xt, 16) || !aligned(grads, 8) ||
      static_cast<int64_t>(p_end - p_begin) * ((N + 255) / 256) * ((K + 255) / 256) > kMaxTiles)
    return ULTRAEP_EUNSUPPORTED;
  return from_hip(ultraep::launch_expert_wgrad(segment(ctx, plan, p_begin), p_end - p_begin, dyt, dyt_scale, N,
                                               xt, xt_scale, K, capacity_rows, grads, accumulate != 0,
                                               static_cast<hipStream_t>(stream)));
}

namespace {
// Shared checks of the two calls over gradient tensors.
int grad_checks(const ultraep_ctx* ctx, const void* const* tensors, const int64_t* numels, int32_t n,
                int32_t dtype, const double* sumsq) {
  if (!ctx || n < 0 || !sumsq || (n > 0 && (!tensors || !numels))) return ULTRAEP_EINVAL;
  if (dtype != ULTRAEP_GRAD_F32 && dtype != ULTRAEP_GRAD_BF16) return ULTRAEP_EINVAL;
  if (n > ULTRAEP_MAX_GRAD_TENSORS || !aligned(tensors, 8) || !aligned(numels, 8) || !aligned(sumsq, 8))
    return ULTRAEP_EUNSUPPORTED;
  return ULTRAEP_OK;
}
}  // namespace

int ultraep_grad_sumsq(const ultraep_ctx* ctx, const void* const* tensors, const int64_t* numels,
                       int32_t n, int32_t dtype, double* sumsq, int32_t accumulate,
                       void* workspace, size_t workspace_bytes, void* stream) {
  const int st = grad_checks(ctx, tensors, numels, n, dtype, sumsq);
  if (st != ULTRAEP_OK) return st;
  if (!workspace || (accumulate != 0 && accumulate != 1)) return ULTRAEP_EINVAL;
  if (!aligned(workspace, 8)) return ULTRAEP_EUNSUPPORTED;
  if (workspace_bytes < ULTRAEP_GRAD_WORKSPACE_BYTES) return ULTRAEP_EWORKSPACE;
  return from_hip(ultraep::launch_grad_sumsq(tensors, numels, n, dtype == ULTRAEP_GRAD_BF16, sumsq,
                                             accumulate != 0, static_cast<double*>(workspace),
                                             static_cast<hipStream_t>(stream)));
}

int ultraep_grad_clip(const ultraep_ctx* ctx, const void* const* tensors, const int64_t* numels,
                      int32_t n, int32_t dtype, const double* sumsq, double max_norm, float* norm,
                      void* const* out, void* stream) {
  const int st = grad_checks(ctx, tensors, numels, n, dtype, sumsq);
  if (st != ULTRAEP_OK) return st;
  if (!(max_norm >= 0.0)) return ULTRAEP_EINVAL;
  if (!aligned(norm, 4) || !aligned(out, 8)) return ULTRAEP_EUNSUPPORTED;
  return from_hip(ultraep::launch_grad_clip(tensors, numels, n, dtype == ULTRAEP_GRAD_BF16, sumsq, max_norm,
                                            norm, out, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
