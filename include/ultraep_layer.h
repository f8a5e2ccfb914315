/*
 * ultraep_layer.h -- C ABI of the steps around the experts of an MoE layer on
 * MI355X (gfx950): the routing that ultraep_balance starts from, the norm with
 * the residual whose rows the dispatch gathers, and the gated activation between
 * the experts' two products, each with its gradients.  It stands beside ultraep.h
 * and ultraep_experts.h and keeps their conventions (context first, device
 * pointers caller-owned and contiguous, stream-ordered, no host synchronisation,
 * host-side argument checks before anything is launched, the same status codes,
 * the 8-bit format of ultraep_experts.h with its rows and columns forms).
 *
 *   ultraep_route                   logits to the top-k experts and their weights
 *   ultraep_route_backward          gradients of the weights to those of the logits
 *   ultraep_residual_norm           residual addition and root-mean-square norm,
 *                                   with the result in bf16, in 8 bits, or both
 *   ultraep_residual_norm_backward  gradients of the stream and of the weight
 *   ultraep_glu_quant               gated activation, quantised
 *   ultraep_glu_quant_backward      its gradient rows, quantised
 *
 * In a training step: residual_norm -> the router's logits -> route ->
 * ultraep_balance -> ultraep_permute_quant of the norm's rows ->
 * ultraep_expert_gemm -> glu_quant -> ultraep_expert_gemm -> ultraep_combine, whose
 * rows the next residual_norm adds.  Backwards ultraep_combine_backward ->
 * ultraep_permute_quant -> ultraep_expert_gemm -> glu_quant_backward ->
 * ultraep_expert_gemm -> ultraep_combine without weights; route_backward takes
 * combine_backward's weight gradients; residual_norm_backward takes the sum of what
 * comes back to the norm's rows, which the caller adds up, with the router's product.
 * permute_quant takes the norm's bf16 rows; its 8-bit rows are for 8-bit products of all
 * rows (a shared expert's, the attention's), which are not in this library.
 *
 * Every result is the same for the same call.  A token's or row's results do not
 * depend on the others' (but for grad_weight, a sum over the rows); the last bits of
 * routing weights go by E, k, groups and the number of tokens, which choose the kernel.
 */
#ifndef ULTRAEP_LAYER_H
#define ULTRAEP_LAYER_H

#include "ultraep_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of logits, residual streams and norm weights. */
#define ULTRAEP_TYPE_F32 0
#define ULTRAEP_TYPE_BF16 1

#define ULTRAEP_ROUTE_SOFTMAX 0
#define ULTRAEP_ROUTE_SIGMOID 1
#define ULTRAEP_MAX_ROUTE_GROUPS 64

#define ULTRAEP_GLU_SILU 0
#define ULTRAEP_GLU_GELU 1

#define ULTRAEP_MAX_NORM_WIDTH 16384

/* Route tokens to their top-k experts.  For every token:
 *  1. An expert whose logit is -inf or NaN is masked: it has the score 0 and is
 *     never chosen (a padded token has all of them masked).  +inf counts as the
 *     largest finite fp32.
 *  2. Scores s: ULTRAEP_ROUTE_SIGMOID s = 1 / (1 + exp(-l)); ULTRAEP_ROUTE_SOFTMAX
 *     the softmax over the experts that are not masked.
 *  3. Keys, by which experts are chosen: s + bias in 64 bits, or the logit itself
 *     without a bias (scores order as logits do).  An expert whose bias is -inf or
 *     NaN is never chosen.
 *  4. With groups > 1, expert e belongs to group e / (E / groups).  A group's key is
 *     the largest of its experts' keys (group_top 1), or the sum in 64 bits of the
 *     two largest s + bias (s without a bias), or of the only one (group_top 2).  The
 *     topk_groups groups with the largest keys stay (ties: the lower group), groups
 *     without an expert to choose never.
 *  5. The k experts with the largest keys, in descending order (ties: the lower
 *     id).  Where fewer are left, the id is -1 (a dropped pair of ultraep_balance)
 *     and the weight 0.
 *  6. Weights: scale * s, the bias not in it; with renormalize scale * s / (the sum
 *     of the chosen experts' s), also where that sum is below fp32's range.
 * Ids are those that 64-bit arithmetic gives; keys (of experts or groups) that differ by
 * no more than its roundings may come in either order.  Weights are fp32: without
 * renormalize scores below 2^-126 may count as zero.
 * Nearly all tokens are settled in 32 bits.  What is not takes about ten times as long:
 *  - tokens in whose choice two pairs of keys are equal or nearly so, or by a softmax with a
 *    bias (also one of zeros) one pair is equal (bf16 logits without a bias excepted);
 *  - fp32 logits without a bias, where the k-th best is more than 16 below the largest;
 *  - group_top 2 without a bias, where three groups or more around the border are within
 *    1e-5 of each other (all are where scores are that small, as in peaked softmaxes), or,
 *    fp32 logits and sigmoids, within 2 / (1 + exp(16 - the largest logit));
 *  - every token of a call whose finite biases span 1e4 or more or reach 2^20 (an expert is
 *    switched off by -inf), or with k > 12, E > 512 or more than 16 groups.
 * In:  logits [tokens][E] of logits_type (E: the context's), bias fp32 [E] or NULL.
 * Out: topk_idx int32 [tokens][k], topk_w fp32 [tokens][k].
 * Errors: EINVAL (null pointers with tokens > 0, tokens < 0, k outside [1, min(E,
 *      64)], unknown type or score, renormalize not 0 or 1, groups < 1 or no divisor
 *      of E, topk_groups outside [1, groups], group_top not 1 or 2, scale not finite);
 *      EUNSUPPORTED (groups > 64, tokens >= 2^31, logits not aligned to their
 *      elements, bias, topk_idx or topk_w not 4-byte aligned). */
int ultraep_route(const ultraep_ctx* ctx, const void* logits, int32_t logits_type, int64_t tokens,
                  int32_t k, int32_t score, const float* bias, int32_t groups, int32_t topk_groups,
                  int32_t group_top, int32_t renormalize, float scale, int32_t* topk_idx,
                  float* topk_w, void* stream);

/* Gradients of the logits of ultraep_route: with g the gradients of the weights w,
 *   sigmoid:                 dl_j = w_j * g_j * (1 - s_j)
 *   sigmoid, renormalised:   dl_j = w_j * (g_j - d) * (1 - s_j),  d = sum_i w_i * g_i / scale
 *   softmax, renormalised:   dl_j = w_j * (g_j - d)
 *   softmax:                 dl_e = (w_e * g_e if chosen) - s_e * sum_i w_i * g_i
 * for the chosen experts (the last: for all that are not masked), zero for the
 * others, in fp32 (scores below 2^-126 may count as zero; the sums of |w * g| have to
 * stay below its largest); the choice has no gradient, nor has the bias.  Weights are
 * computed anew from the logits; an id outside [0, E) or of a masked expert has no weight
 * and its gradient is not looked at; an id that a row names twice counts twice.
 * In:  logits as for ultraep_route, topk_idx int32 [tokens][k], grad_topk_w fp32
 *      [tokens][k] (from ultraep_combine_backward).
 * Out: grad_logits [tokens][E] of logits_type, every element written.
 * Errors: as ultraep_route. */
int ultraep_route_backward(const ultraep_ctx* ctx, const void* logits, int32_t logits_type,
                           int64_t tokens, int32_t k, int32_t score, int32_t renormalize, float scale,
                           const int32_t* topk_idx, const float* grad_topk_w, void* grad_logits,
                           void* stream);

/* Add rows to the residual stream and normalise it.  For every row
 *   h = residual + x, rounded to the stream's type (h = x without a residual)
 *   rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * weight
 * in fp32; y is rounded once to bf16 for y, and from fp32 to e4m3 for the rows form.
 * The sum of a row's squares has to stay below fp32's largest (magnitudes to 2^56);
 * with eps 0 a row whose squares are all below its range has no finite rstd.
 * In:  x [rows][H] bf16; residual [rows][H] of residual_type, or NULL; weight [H] of
 *      weight_type.
 * Out: h [rows][H] of residual_type, or NULL where the sum is not wanted or there is
 *      no residual; y [rows][H] bf16, or NULL; the rows form in q [rows][Hp] and
 *      q_scale [rows][Hs], or both NULL; rstd fp32 [rows], or NULL.
 * h may be the residual itself, and y may be x; apart from that outputs may overlap
 * neither each other nor what the call reads.
 * Errors: EINVAL (null x or weight with rows > 0, h without residual, half a form,
 *      no output, rows < 0, H <= 0, unknown type, eps negative or not finite);
 *      EUNSUPPORTED (H % 8 != 0, H > 16384, rows >= 2^31, x, residual, weight, h, y or
 *      q not 16-byte, q_scale or rstd not 4-byte aligned). */
int ultraep_residual_norm(const ultraep_ctx* ctx, const uint16_t* x, const void* residual,
                          int32_t residual_type, const void* weight, int32_t weight_type, float eps,
                          int64_t rows, int32_t H, void* h, uint16_t* y, uint8_t* q, uint8_t* q_scale,
                          float* rstd, void* stream);

/* Bytes of workspace ultraep_residual_norm_backward needs for grad_weight (EINVAL,
 * EUNSUPPORTED as there). */
int ultraep_residual_norm_workspace_bytes(int64_t rows, int32_t H, size_t* out);

/* Gradients of ultraep_residual_norm.  With z = weight * grad_y, for every row
 *   grad_h = grad_in + rstd * z - h * rstd^3 * mean(z * h)
 *   grad_weight (+)= sum over the rows of grad_y * h * rstd
 * in fp32.  grad_h is the gradient of both the residual and x (and of x alone
 * where there was no residual).
 * In:  grad_y [rows][H] bf16; h [rows][H] of h_type (what the forward wrote, or its x
 *      without a residual), weight, rstd fp32 [rows] as in the forward; grad_in
 *      [rows][H] of h_type, the stream's gradient from behind, or NULL.
 * Out: grad_h [rows][H] of h_type (may be grad_in itself); grad_x [rows][H] bf16: the
 *      same values rounded to bf16, with an fp32 stream only, or NULL; grad_weight
 *      fp32 [H], added to with accumulate = 1, else overwritten (zeros without rows),
 *      or NULL.
 * workspace: scratch of this call, ultraep_residual_norm_workspace_bytes; not
 *      looked at without grad_weight.
 * Errors: EINVAL (null pointers with rows > 0, a grad_weight without workspace,
 *      grad_x with a bf16 stream, rows < 0, H <= 0, unknown type, accumulate not 0 or
 *      1); EUNSUPPORTED (H % 8 != 0, H > 16384, rows >= 2^31, a buffer not 16-byte,
 *      rstd not 4-byte aligned); EWORKSPACE. */
int ultraep_residual_norm_backward(const ultraep_ctx* ctx, const uint16_t* grad_y, const void* h,
                                   int32_t h_type, const void* weight, int32_t weight_type,
                                   const float* rstd, const void* grad_in, int64_t rows, int32_t H,
                                   void* grad_h, uint16_t* grad_x, float* grad_weight,
                                   int32_t accumulate, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* Gated activation of the rows of physical experts [p_begin, p_end), quantised:
 *   a[i][c] = f(h[i][c]) * h[i][F + c] for c < F, f(g) = g / (1 + exp(-z)),
 *   ULTRAEP_GLU_SILU z = g;  ULTRAEP_GLU_GELU z = 2 sqrt(2/pi) (g + 0.044715 g^3)
 * (gelu in its form by the hyperbolic tangent), in fp32, rounded once to e4m3.
 * Magnitudes below 2^-100 become zero, and a sigmoid 1 / (1 + exp(-z)) below 2^-126 may
 * count as zero whatever it is multiplied with.
 * In:  plan (one record); h [capacity_rows][2F] bf16, the segment's rows in order
 *      (the first product's output: gate columns, then the others).
 * Out: the rows form of a in q [capacity_rows][Fp] and q_scale [capacity_rows][Fs],
 *      or both NULL; its columns form in qt and qt_scale, capacity_blocks blocks of F
 *      columns, or both NULL.  Rows and blocks without an expert are left as they are.
 * Errors: EINVAL (null context, plan or h, half a form or no form, F <= 0, unknown
 *      activation, capacity_rows < 0, bad range, capacity_blocks < capacity_rows / 128 +
 *      p_end - p_begin); EUNSUPPORTED (F % 8 != 0, F > 2^22, capacity_rows >= 2^31; h, q
 *      or qt not 16-byte, q_scale not 4-byte aligned). */
int ultraep_glu_quant(const ultraep_ctx* ctx, const void* plan, const uint16_t* h, int32_t F,
                      int32_t activation, int32_t p_begin, int32_t p_end, uint8_t* q,
                      uint8_t* q_scale, uint8_t* qt, uint8_t* qt_scale, int64_t capacity_rows,
                      int64_t capacity_blocks, void* stream);

/* Gradient rows of ultraep_glu_quant, quantised: of d[i] = [grad[i] * h[i][F..] * f'(h[i][..F]),
 * grad[i] * f(h[i][..F])], 2F columns, as there the forms of a.
 * In:  plan, h as there; grad [capacity_rows][F] bf16, the gradients of a.
 * Out: the rows form in q [capacity_rows][(2F)p] and q_scale, the columns form in
 *      qt and qt_scale of 2F columns; either may be left out.
 * Errors: as ultraep_glu_quant, and EINVAL for a null grad, EUNSUPPORTED for one
 *      that is not 16-byte aligned. */
int ultraep_glu_quant_backward(const ultraep_ctx* ctx, const void* plan, const uint16_t* h,
                               const uint16_t* grad, int32_t F, int32_t activation, int32_t p_begin,
                               int32_t p_end, uint8_t* q, uint8_t* q_scale, uint8_t* qt,
                               uint8_t* qt_scale, int64_t capacity_rows, int64_t capacity_blocks,
                               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ULTRAEP_LAYER_H */
