/*
 * libgmm, the operators around the grouped products of a mixture-of-experts
 * layer: the router's choice of experts, the tokens' rows sorted by expert and
 * brought back, and microscaled 4-bit floating point (quantisation, and the
 * grouped product of 4-bit rows with 4-bit weights).
 *
 * Status codes, element types and the conventions for pointers, streams and
 * the workspace are those of libgmm.h: device pointers owned by the caller, no
 * allocation and no synchronisation inside a call, host-checkable errors
 * returned before anything is launched.  Arrays are dense and row-major unless
 * an argument gives their row pitch.  Of these calls only gmm_fp4() takes a
 * workspace, for its error flags.
 */
#ifndef LIBGMM_MOE_H_
#define LIBGMM_MOE_H_

#include "libgmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ the router */

/* gmm_route() score; GMM_SCORE_BIASED may be or-ed to it there: select_bias is the score's. */
enum { GMM_SCORE_SOFTMAX = 0, GMM_SCORE_SIGMOID = 1, GMM_SCORE_BIASED = 16 };

/* Largest topk of gmm_route(). */
#define GMM_MAX_TOPK 32

/*
 * Top-k routing.  For each token t with logits l[e], e < num_experts:
 *   key[e] = l[e] + select_bias[e] in fp32 (l[e] without select_bias); with
 *            GMM_SCORE_BIASED s(l)[e] + select_bias[e], s the softmax over all experts or
 *            the sigmoid in fp32 (the form of biases that balance the experts' loads);
 *   the topk experts with the largest keys are chosen, in falling order, equal
 *   keys by rising index (-0 equals 0).  An expert whose key is -inf or NaN is
 *   never chosen, nor is one whose logit is -inf: that switches it off for the token.
 *   (A NaN logit, and for the softmax +inf, makes the weights that its score enters NaN,
 *   and with GMM_SCORE_BIASED the keys.)
 *   Without renormalize the weight of a chosen expert is scale * s(l)[e], with s
 *   the softmax over all experts or the sigmoid; with renormalize those scores
 *   are divided by their sum over the chosen experts.  select_bias moves the
 *   choice only, never the weights.
 * All sums and exponentials are fp32.  Slots past the number of experts that can
 * be chosen hold expert -1 and weight 0; a token whose token_mask is 0 has only
 * such slots, whatever its logits hold.
 *
 *   logits       [tokens, num_experts] BF16 or F32, row pitch logits_ld elements
 *   topk         1 .. min(num_experts, GMM_MAX_TOPK); num_experts <= GMM_MAX_GROUPS
 *   select_bias  NULL or f32 [num_experts];  token_mask  NULL or one byte per token
 *   weights      f32 [tokens, topk];  experts  int32 [tokens, topk]
 */
int gmm_route(const void* logits, int logits_dtype, int64_t tokens, int32_t num_experts, int64_t logits_ld,
              int32_t topk, int score, int renormalize, float scale, const float* select_bias,
              const uint8_t* token_mask, float* weights, int32_t* experts, void* stream);

/*
 * Gradient of gmm_route()'s weights with respect to the logits (the choice itself
 * has none): dlogits [tokens, num_experts] of logits_dtype, dense, from dweights
 * f32 [tokens, topk] and the experts that gmm_route() chose.  Slots with expert -1
 * give nothing (their dweights are not read into any result); a token with only
 * such slots has zeros.  The weights are computed again from the logits.
 */
int gmm_route_backward(const float* dweights, const int32_t* experts, const void* logits, int logits_dtype,
                       int64_t tokens, int32_t num_experts, int64_t logits_ld, int32_t topk, int score,
                       int renormalize, float scale, void* dlogits, void* stream);

/* ------------------------------------------------------------------ tokens by expert and back */

/*
 * The stable counting sort of the slots (t, j) by expert.  A slot whose expert is
 * outside [0, num_experts) is dropped.
 *   group_sizes [num_experts]  rows of each expert (gmm()'s group_sizes)
 *   rows [tokens, topk]        the row of slot (t, j) in expert order; -1: dropped
 *   source [tokens * topk]     the slot t * topk + j of each row; -1 past the groups
 * Rows of one expert keep the order of their slots.  tokens * topk is at most 2^31 - 1024;
 * 1 <= num_experts <= GMM_MAX_GROUPS; here and in the calls below 1 <= topk <= GMM_MAX_TOPK.
 */
int gmm_sort_by_expert(const int32_t* experts, int64_t tokens, int32_t topk, int32_t num_experts,
                       int32_t* group_sizes, int32_t* rows, int32_t* source, void* stream);

/*
 * out[rows[t, j]] = x[t] for every slot that is not dropped; the rows of out past
 * the groups (source < 0) are zero.  x [tokens, d] BF16 or F32 with row pitch x_ld
 * elements, out [tokens * topk, d] dense of the same dtype.  rows and source as
 * gmm_sort_by_expert() writes them (an entry of rows that is no row counts as dropped).  Any d >= 1.
 */
int gmm_dispatch(const void* x, int dtype, int64_t tokens, int64_t d, int64_t x_ld, int32_t topk, const int32_t* rows,
                 const int32_t* source, void* out, void* stream);

/*
 * out[t] = sum over the slots of t that are not dropped of weights[t, j] *
 * in[rows[t, j]], in fp32 with one rounding to dtype; a token without slots gives
 * zeros.  weights f32 [tokens, topk], or NULL for ones (which makes this the
 * gradient of gmm_dispatch()).  in [tokens * topk, d], out [tokens, d], both dense,
 * BF16 or F32.
 */
int gmm_combine(const void* in, int dtype, int64_t tokens, int64_t d, int32_t topk, const int32_t* rows,
                const float* weights, void* out, void* stream);

/*
 * Gradients of gmm_combine():
 *   din[rows[t, j]] = weights[t, j] * dout[t], rounded once; rows past the groups zero;
 *   dweights[t, j]  = sum over c of dout[t, c] * in[rows[t, j], c] in fp32; 0 if dropped.
 * Sums have a fixed order: the same inputs give the same bits.
 */
int gmm_combine_backward(const void* dout, const void* in, int dtype, int64_t tokens, int64_t d, int32_t topk,
                         const int32_t* rows, const int32_t* source, const float* weights, void* din, float* dweights,
                         void* stream);

/* ------------------------------------------------------------------ microscaled 4-bit floating point */

/* A matrix [rows, k] in one of the formats below is
 *   codes        [rows, k / 2] e2m1, two per byte, the even k in the low nibble
 *   block_scale  [ceil(k / (16 * block)), rows, 16] bytes: the scales of a row's blocks
 *                by windows of 16 blocks; bytes past the last block are 0 (gmm_fp4() reads
 *                whole windows: a NaN there would reach its sums)
 *   row_scale    f32 [rows], NVFP4 only
 * and stands for code * block_scale * row_scale.  A batch of matrices (the experts'
 * weights) has a leading dimension in each array.
 *   GMM_FP4_NVFP4  block 16, e4m3 scales, row scales powers of two
 *   GMM_FP4_MXFP4  block 32, E8M0 scales: byte e is 2^(e - 127), 255 is NaN
 */
enum { GMM_FP4_NVFP4 = 0, GMM_FP4_MXFP4 = 1 };

/*
 * Quantises x [batch * rows_per_batch, k].
 *   NVFP4: row_scale = the least 2^e (e >= -126) with max|row| <= 6 * 448 * 2^e (1 for a
 *          row of zeros); block scale = max|block| / (6 row_scale) rounded to e4m3, ties to
 *          even; code = x / (block scale * row_scale) rounded to e2m1, ties to even,
 *          saturating at +-6; codes of a block whose scale is 0 are 0.
 *   MXFP4: block scale = the least 2^e (e >= -127) with max|block| <= 6 * 2^e (byte 0 for a
 *          block of zeros); codes likewise.
 * Every rounding is that of the exact quotient.  Codes keep x's sign, zeros included.  A block
 * with an infinity or NaN gets a NaN scale and zero codes, and does not count towards its
 * row's scale.
 *   x         BF16 or F32, row pitch x_ld elements; k % 32 == 0
 *   rows, source, topk  NULL, NULL, 1; or an order of gmm_sort_by_expert() over
 *             rows_per_batch tokens (batch 1): then row rows[t, j] of the result is x[t]
 *             quantised, rows past the groups are zeros, and the result has
 *             rows_per_batch * topk rows.
 * codes and block_scale 16-byte aligned.
 */
int gmm_quantize_fp4(const void* x, int x_dtype, int32_t batch, int64_t rows_per_batch, int64_t k, int64_t x_ld,
                     int format, const int32_t* rows, const int32_t* source, int32_t topk, void* codes,
                     void* block_scale, float* row_scale, void* stream);

/* The values a quantised matrix stands for, rounded once to out_dtype, whatever row_scale holds
 * (with the powers of two of gmm_quantize_fp4() BF16 holds them exactly while they are in its
 * normal range). */
int gmm_dequantize_fp4(const void* codes, const void* block_scale, const float* row_scale, int format, int32_t batch,
                       int64_t rows_per_batch, int64_t k, void* out, int out_dtype, void* stream);

/*
 * Grouped product of 4-bit rows with 4-bit weights on the block-scaled tensor cores:
 * for every local group g and row r of it
 *   out[r, c] = rs[r] * ws[g, c] * sum over blocks of
 *               (row block scale * weight block scale * sum of code products) + bias[g, c]
 * with fp32 sums and one rounding to out_dtype; every other row of out is zero, as in gmm().
 * Both operands have the same format.
 *   lhs_*      [m, k] quantised rows;  rhs_*  [num_local_groups][n, k] quantised weights
 *   k % 32 == 0, n % 8 == 0; m, k and n at most 2^31 - 1024; codes, block scales and out
 *   16-byte aligned
 *   group_sizes, group_offset (a host value), bias, workspace and stream as in gmm().
 */
int gmm_fp4(const void* lhs_codes, const void* lhs_block_scale, const float* lhs_row_scale, int64_t m, int64_t k,
            const void* rhs_codes, const void* rhs_block_scale, const float* rhs_row_scale, int format,
            int32_t num_local_groups, int64_t n, const int32_t* group_sizes, int32_t num_total_groups,
            int32_t group_offset, const void* rhs_bias, int bias_dtype, void* out, int out_dtype, void* workspace,
            size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBGMM_MOE_H_ */
