/*
 * ultraep_experts.h -- C ABI of the experts' own steps on MI355X (gfx950):
 * the 8-bit products between dispatch and combine, and the end of the
 * gradients' path.  It stands beside ultraep.h and keeps its conventions
 * (context first, device pointers caller-owned, stream-ordered, no host
 * synchronisation, host-side argument checks before anything is launched,
 * the same status codes).
 *
 *   ultraep_permute_quant  gather bf16 rows into the dispatch layout and
 *                          quantise them, as rows, as columns, or both
 *   ultraep_weight_quant   quantise expert weights by 128 x 128 blocks, as they
 *                          are, transposed, or both
 *   ultraep_expert_gemm    every physical expert's rows times its weights
 *                          (forward; with transposed weights, the gradient of
 *                          the rows)
 *   ultraep_expert_wgrad   every physical expert's weight gradient, fp32
 *   ultraep_grad_sumsq     sum of squares over many gradient tensors
 *   ultraep_grad_clip      scale them to a largest global norm
 *
 * In a training step: permute_quant (rows, columns) -> expert_gemm, activation,
 * permute_quant, expert_gemm -> ultraep_combine; backwards
 * ultraep_combine_backward -> permute_quant of the gradient rows (rows and
 * columns) -> expert_gemm with transposed weights and expert_wgrad into the
 * masters' and replicas' gradients -> ultraep_fold_grads -> grad_sumsq,
 * grad_clip.  The quantised weights of the masters reach the replica slots by
 * ultraep_weight_sync (two bytes are one of its 16-bit elements).
 *
 * Format.  A value is an OCP e4m3 byte q (no infinities; 0x7F and 0xFF are
 * NaN) times 2^(s - 127), where s is the scale byte of the value's block of
 * 128.  s - 127 is the smallest exponent e >= -126 for which the block's
 * largest finite magnitude is at most 448 * 2^e (448 is e4m3's largest value;
 * e = 0 for a block of zeros or of nothing finite); q is the value times 2^-e,
 * rounded to nearest even.  Powers of two make that scaling exact, so the
 * rounding to e4m3 is the only one, and a value of bf16's normal range is a bf16
 * number.  Infinities and NaN become NaN; they do not raise the scale.
 *
 *   rows      q [rows][Hp], scale [rows][Hs]: a block is 128 columns of a row.
 *             Hp = H rounded up to 128, the columns behind H are zeros;
 *             Hs = Hp / 128 rounded up to 4, the bytes behind Hp / 128 are 127.
 *   columns   qt [blocks][H][128], scale [blocks][H]: a block is 128 rows of
 *             one expert in one column, [h][r] holding row r of the block, the
 *             slots behind the expert's last row zeros.  Expert p's blocks
 *             start at (o_p / 128) + (p - p_begin), o_p its first row counted
 *             from the segment's; its ceil(rows / 128) blocks follow each
 *             other.  A segment of n experts needs rows / 128 + n blocks; a
 *             block that belongs to no expert is neither written nor read.
 *   weights   q [N][Kp], scale [ceil(N / 128)][Ks]: a block is 128 x 128.
 *
 * Segments.  plan, p_begin and p_end name a range of physical experts as in
 * ultraep_permute; the rows of the range are counted from its first one, and
 * rows at or beyond capacity_rows are not there for any of these calls.  Without
 * rows (capacity_rows = 0) or experts (p_begin = p_end, n = 0) nothing is read or
 * written, but for the weight gradients of experts without rows, and a buffer that
 * so has no elements may be NULL, as hidden may with hidden_rows = 0.
 */
#ifndef ULTRAEP_EXPERTS_H
#define ULTRAEP_EXPERTS_H

#include "ultraep.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ULTRAEP_QUANT_BLOCK 128
#define ULTRAEP_MAX_GRAD_TENSORS 4096
#define ULTRAEP_GRAD_WORKSPACE_BYTES 16384

/* Element types of the gradients ultraep_grad_sumsq and ultraep_grad_clip take. */
#define ULTRAEP_GRAD_F32 0
#define ULTRAEP_GRAD_BF16 1

/* Quantise the rows of physical experts [p_begin, p_end).
 * In:  plan (one record); hidden [hidden_rows][H] bf16; inv [N] of the layer,
 *      or NULL.  Row i of the segment is hidden[inv[phys_off[p_begin] + i] / k]
 *      as in ultraep_permute (a negative entry or a token at or beyond
 *      hidden_rows: zeros), or, with inv NULL, hidden[i] (zeros at or beyond
 *      hidden_rows; k is not looked at).
 * Out: the rows form in q and q_scale, capacity_rows rows, or both NULL; the
 *      columns form in qt and qt_scale, capacity_blocks blocks, or both NULL.
 *      Together they read the rows once.  Rows and blocks without an expert
 *      are left as they are.
 * Errors: EINVAL (null context, plan or hidden; half a form or no form; H <= 0,
 *      with inv k outside [1, 64], hidden_rows < 0, capacity_rows < 0, bad range;
 *      capacity_blocks < capacity_rows / 128 + p_end - p_begin); EUNSUPPORTED
 *      (H % 8 != 0; hidden, q or qt not 16-byte, q_scale not 4-byte aligned;
 *      capacity_rows >= 2^31, H > 2^24). */
int ultraep_permute_quant(const ultraep_ctx* ctx, const void* plan, const int32_t* inv, int32_t k,
                          const uint16_t* hidden, int64_t hidden_rows, int32_t H, int32_t p_begin,
                          int32_t p_end, uint8_t* q, uint8_t* q_scale, uint8_t* qt,
                          uint8_t* qt_scale, int64_t capacity_rows, int64_t capacity_blocks,
                          void* stream);

/* Quantise the weights [N][K] of n experts by 128 x 128 blocks.
 * In:  weights: DEVICE array of n device pointers to bf16 (any alignment of
 *      two bytes; a NULL entry leaves that expert's outputs as they are).
 * Out: q [n][N][Kp] and q_scale [n][ceil(N/128)][Ks], or both NULL; of the
 *      transposes qt [n][K][Np] and qt_scale [n][ceil(K/128)][Ns], or both
 *      NULL.  A block and its transpose have the same scale and values.
 * Errors: EINVAL (null context or weights with n > 0, half a form or no form,
 *      n < 0, N <= 0, K <= 0); EUNSUPPORTED (N % 8 or K % 8 != 0, N or K > 2^20,
 *      n > 1024, q or qt not 16-byte aligned, scales not 4-byte aligned). */
int ultraep_weight_quant(const ultraep_ctx* ctx, const uint16_t* const* weights, int32_t n,
                         int32_t N, int32_t K, uint8_t* q, uint8_t* q_scale, uint8_t* qt,
                         uint8_t* qt_scale, void* stream);

/* Multiply the rows of physical experts [p_begin, p_end) with their experts'
 * weights: out[i][n] = sum over k < K of x[i][k] * w_p[n][k] for the rows i of
 * expert p, the products and sums in fp32, rounded once to bf16 (nearest even).
 * Values are multiplied as bf16 numbers, exactly those the bytes and scales
 * stand for, but magnitudes below 2^-126 may count as zero and such of 2^128
 * and more as infinities.  The order of the sums, and so a row's last bits, go by
 * K, N, capacity_rows and the number of experts; the same call gives the same bits.
 * In:  q, q_scale: capacity_rows rows of K columns in the rows form;
 *      w, w_scale: DEVICE arrays of p_end - p_begin device pointers, entry
 *      p - p_begin to expert p's weights (16-byte aligned) and scales (4-byte
 *      aligned) in the weights form.  The rows of an expert with a NULL or
 *      misaligned entry are left as they are; entries of experts without rows
 *      are not looked at.
 * Out: out [capacity_rows][N] bf16; rows without an expert are left as they are.
 * The kernel is chosen by capacity_rows: where few rows come, a capacity near
 * them is faster (41 rows by 6 experts of 4096 x 7168: 37 us, 81 from 656 up).
 * With the gradient rows for q (K = the forward's N) and the transposed weights
 * this is the gradient of the forward's rows.
 * Errors: EINVAL (null pointers, N <= 0, K <= 0, bad range, capacity_rows < 0);
 *      EUNSUPPORTED (N % 8 != 0, N or K > 2^20, capacity_rows >= 2^31, more than
 *      2^23 tiles of 256 x 256 with one to spare an expert, q or out not
 *      16-byte, q_scale not 4-byte, the tables not 8-byte aligned). */
int ultraep_expert_gemm(const ultraep_ctx* ctx, const void* plan, const uint8_t* q,
                        const uint8_t* q_scale, int32_t K, const uint8_t* const* w,
                        const uint8_t* const* w_scale, int32_t N, int32_t p_begin, int32_t p_end,
                        uint16_t* out, int64_t capacity_rows, void* stream);

/* Weight gradients of physical experts [p_begin, p_end):
 *   grads[p - p_begin][n][k] (+)= sum over the rows i of expert p of dy[i][n] * x[i][k]
 * in fp32, in a fixed order; a gradient does not depend on the other experts.
 * Values are multiplied as bf16 numbers, exactly those the bytes and scales
 * stand for, but magnitudes below 2^-126 may count as zero and such of 2^128
 * and more as infinities.
 * In:  dyt, dyt_scale (N columns) and xt, xt_scale (K columns): both in the
 *      columns form, capacity_rows / 128 + p_end - p_begin blocks; grads:
 *      DEVICE array of p_end - p_begin device pointers to fp32 [N][K] (any
 *      alignment of four bytes; a NULL entry is skipped; no two may overlap).
 * Out: the gradients, added to with accumulate = 1, else overwritten (zeros for
 *      an expert without rows).
 * Errors: EINVAL (null pointers, N <= 0, K <= 0, bad range, capacity_rows < 0,
 *      accumulate not 0 or 1); EUNSUPPORTED (N % 8 or K % 8 != 0, N or K >
 *      2^20, capacity_rows >= 2^31, more than 2^23 tiles of 256 x 256, dyt or xt
 *      not 16-byte, the table not 8-byte aligned). */
int ultraep_expert_wgrad(const ultraep_ctx* ctx, const void* plan, const uint8_t* dyt,
                         const uint8_t* dyt_scale, int32_t N, const uint8_t* xt,
                         const uint8_t* xt_scale, int32_t K, int32_t p_begin, int32_t p_end,
                         int64_t capacity_rows, float* const* grads, int32_t accumulate,
                         void* stream);

/* sumsq (+)= the sum of the squares of all elements of n tensors, in fp64 in an
 * order that depends on the sizes alone.
 * In:  tensors: DEVICE array of n device pointers (aligned to their elements;
 *      a NULL entry counts as empty); numels: DEVICE array of n int64 (<= 0:
 *      empty); dtype ULTRAEP_GRAD_*; workspace: at least
 *      ULTRAEP_GRAD_WORKSPACE_BYTES, 8-byte aligned, scratch of this call.
 * Out: sumsq, one fp64: added to with accumulate = 1 (tensors of another type),
 *      else overwritten.  Ranks add their sums before the clipping.
 * Errors: EINVAL (null pointers, n < 0, dtype, accumulate not 0 or 1);
 *      EUNSUPPORTED (n > ULTRAEP_MAX_GRAD_TENSORS, tables, sumsq or workspace
 *      not 8-byte aligned); EWORKSPACE. */
int ultraep_grad_sumsq(const ultraep_ctx* ctx, const void* const* tensors, const int64_t* numels,
                       int32_t n, int32_t dtype, double* sumsq, int32_t accumulate,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Clip n gradient tensors to a global norm of at most max_norm: with
 *   norm = sqrt(*sumsq), c = min(1, max_norm / (norm + 1e-6))
 * (both fp64) every element becomes c times it, rounded to fp32 and from there
 * to its type.  An infinite norm gives c = 0 (a finite max_norm taken), NaN
 * gives NaN.  With c = 1 gradients in place are not touched.
 * In:  tensors, numels, n, dtype as above, sumsq from ultraep_grad_sumsq.
 * Out: the tensors, in place (out NULL) or in the tensors that out, a DEVICE
 *      array of n device pointers, names (a NULL entry: that tensor in place);
 *      what is written may overlap nothing else that the call reads or writes (a
 *      tensor named twice would be scaled twice); norm: one fp32, or NULL.
 * Errors: EINVAL (null pointers, n < 0, dtype, max_norm negative or NaN);
 *      EUNSUPPORTED (n > ULTRAEP_MAX_GRAD_TENSORS, tables or sumsq not 8-byte,
 *      norm not 4-byte aligned). */
int ultraep_grad_clip(const ultraep_ctx* ctx, const void* const* tensors, const int64_t* numels,
                      int32_t n, int32_t dtype, const double* sumsq, double max_norm, float* norm,
                      void* const* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ULTRAEP_EXPERTS_H */
