/*
 * libgmm, more operators of a mixture-of-experts layer: the losses that balance
 * the router with their gradient, the gated activation between an expert's two
 * products with its gradient, weights in 4-bit integers with group scales, and
 * their products with few tokens.
 *
 * Status codes, element types and the conventions for pointers, streams and
 * errors are those of libgmm.h and libgmm_moe.h; GMM_MAX_TOPK and the scores are
 * libgmm_moe.h's.
 */
#ifndef LIBGMM_EXPERTS_H_
#define LIBGMM_EXPERTS_H_

#include "libgmm_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ balance of the router */

/* Bytes of scratch that gmm_balance_loss() needs (0 for few tokens, and for sizes that it refuses);
 * no content is expected, none is kept. */
size_t gmm_balance_scratch_bytes(int64_t tokens, int32_t num_experts, int64_t sequences);

/*
 * The balance loss and the z loss of a router, and its experts' loads.  The tokens
 * are `sequences` runs of tokens / sequences consecutive ones.  A token counts if
 * its token_mask is not 0 (NULL: all) and not every logit of it is -inf; N is how
 * many do.  With p[t] the softmax of token t's logits (GMM_SCORE_SIGMOID: their
 * sigmoids over the sum of these) and
 *   counts[s, e] = slots of sequence s's tokens that count whose expert is e,
 *   f[s, e]      = counts[s, e] / sum over e of counts[s, e]  (0 without any),
 *   losses[0] = num_experts / N * sum over t of sum over e of f[s(t), e] p[t, e]
 *   losses[1] = 1 / N * sum over t of (log sum over e of exp(l[t, e]))^2
 * (0 where N is 0).  losses[0] is 1 where all loads or all p are equal.  Slots whose
 * expert is outside [0, num_experts) are dropped.  Sums are fp32 in a fixed order:
 * the same inputs give the same bits.
 *
 *   logits   [tokens, num_experts] BF16 or F32, row pitch logits_ld elements; the
 *            rows of tokens that a mask takes out are not read into any result
 *   experts  int32 [tokens, topk], as gmm_route() chose them; topk <= GMM_MAX_TOPK
 *   losses   f32 [2];  counts  int32 [sequences, num_experts];  counted  int32 [1]: N
 *   scratch  gmm_balance_scratch_bytes() bytes, 16-byte aligned (NULL for none); calls that may run at
 *            the same time need one each
 * sequences >= 1 divides tokens; tokens * topk at most 2^31 - 1024.
 */
int gmm_balance_loss(const void* logits, int logits_dtype, int64_t tokens, int32_t num_experts, int64_t logits_ld,
                     const int32_t* experts, int32_t topk, int score, const uint8_t* token_mask, int64_t sequences,
                     float* losses, int32_t* counts, int32_t* counted, void* scratch, size_t scratch_bytes,
                     void* stream);

/*
 * Gradient of dlosses[0] * losses[0] + dlosses[1] * losses[1] with respect to the
 * logits (the counts have none): dlogits [tokens, num_experts] of logits_dtype,
 * dense; zeros for tokens that do not count.  counts and counted as
 * gmm_balance_loss() wrote them, dlosses f32 [2] on the device.
 */
int gmm_balance_loss_backward(const float* dlosses, const int32_t* counts, const int32_t* counted, const void* logits,
                              int logits_dtype, int64_t tokens, int32_t num_experts, int64_t logits_ld, int score,
                              const uint8_t* token_mask, int64_t sequences, void* dlogits, void* stream);

/* ------------------------------------------------------------------ the experts' activation */

/* act(g): GMM_ACT_SILU g / (1 + exp(-g)); GMM_ACT_GELU g / 2 * (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))). */
enum { GMM_ACT_NONE = 0, GMM_ACT_SILU = 1, GMM_ACT_GELU = 2 };

/*
 * out[r, c] = act(h[r, c]) * h[r, f + c], in fp32 with one rounding: h [rows, 2 f] with
 * row pitch h_ld elements, the gates before the values they gate; out [rows, f] dense.
 * BF16 or F32; any f >= 1.  Rows of zeros give zeros.
 */
int gmm_gated_act(const void* h, int dtype, int64_t rows, int64_t f, int64_t h_ld, int act, void* out, void* stream);

/* Gradient of gmm_gated_act(): dh [rows, 2 f] dense from dout [rows, f] dense and h. */
int gmm_gated_act_backward(const void* dout, const void* h, int dtype, int64_t rows, int64_t f, int64_t h_ld, int act,
                           void* dh, void* stream);

/* ------------------------------------------------------------------ weights in 4-bit integers */

/* A matrix [rows, k] is
 *   codes [rows, k / 2]   two per byte, the even k in the low nibble
 *   scale [ceil(k / 256), rows, 256 / group]  bf16: a row's scales by windows of 256 k
 *   zero  like scale, one byte each, 0 .. 15; or NULL
 * and stands for scale * code, code two's complement (-8 .. 7), without zero points, and
 * for scale * (code - zero), code 0 .. 15, with them.  group is 32, 64 or 128 and divides
 * k.  Entries past the last group are not read.  A batch of matrices (the experts'
 * weights) has a leading dimension in each array.
 */

/*
 * Quantises x [batch * rows_per_batch, k], BF16 or F32, row pitch x_ld elements.  For each group
 *   zero == NULL: scale = max|x| / 7, code = x / scale, within -8 .. 7;
 *   else          scale = (hi - lo) / 15, hi and lo the largest and least of x and 0,
 *                 zero = -lo / scale, code = x / scale + zero, within 0 .. 15;
 * scales are fp32 quotients rounded to bf16, zero points and x / scale the exact quotients rounded
 * to whole numbers, ties to even.  Codes and zero points of a group whose scale is 0 are 0, as are
 * those of a group with an infinity or NaN (or with hi - lo past fp32), whose scale is NaN.
 * Entries past the last group are 0.  codes and scale 16-byte aligned, zero 4-byte.
 */
int gmm_quantize_int4(const void* x, int x_dtype, int32_t batch, int64_t rows_per_batch, int64_t k, int64_t x_ld,
                      int32_t group, void* codes, void* scale, void* zero, void* stream);

/* The values that a quantised matrix stands for, rounded once to out_dtype (BF16 or F32).  codes
 * 4-byte aligned, scale 2-byte. */
int gmm_dequantize_int4(const void* codes, const void* scale, const void* zero, int32_t group, int32_t batch,
                        int64_t rows_per_batch, int64_t k, void* out, int out_dtype, void* stream);

/* Bytes of scratch that gmm_matvec_int4() needs (0 for few tokens, and for sizes that it refuses);
 * no content is expected, none is kept. */
size_t gmm_matvec_scratch_bytes(int64_t tokens, int64_t k, int32_t group, int has_zero, int32_t topk, int x_per_slot);

/*
 * Products of few tokens with the 4-bit weights of the experts that each chose, in the
 * order of the tokens (no sort):
 *   h[t, j] = W(experts[t, j]) x[t, j]
 *           = sum over groups of scale * sum of (code - zero) x
 *             (exact differences and products, fp32 sums)
 *   y[t, j] = h[t, j], or with act: act(first half of h[t, j]) * second half
 *   out[t, j] = y[t, j], or with weights: out[t] = sum over j of weights[t, j] * y[t, j]
 * rounded once to out_dtype.  A slot whose expert is outside [0, num_experts) gives zeros,
 * and nothing to a sum.  Each expert's weights are read once for every 8 of its tokens (for
 * every 8 tokens, with weights), so this is for the few rows an expert has in decoding, some 3
 * to 8 at most.  For more, gmm() takes the codes of groups of 128 without zero points as GMM_DTYPE_INT4
 * weights, with rhs_scale [num_experts, k / 128, 1, n] the scales in f32; other groups, and zero
 * points, it takes as gmm_dequantize_int4()'s bf16 values.
 * The same inputs give the same bits.  A row of x with an infinity or NaN gives NaN.  Sums are held to
 * at least 2^-129 of the row's largest |x|: terms below 2^-105 of it lose bits, before or after their
 * scale.
 *
 *   x        BF16 [tokens, k] with row pitch x_ld (x_per_slot 0: all slots of a token share
 *            it) or dense [tokens, topk, k] (x_per_slot 1; x_ld is not used)
 *   codes, scale, zero   [num_experts][n, k] as above; zero NULL or not
 *   experts  int32 [tokens, topk], or NULL: topk is 1 and every token's expert is 0
 *   weights  NULL or f32 [tokens, topk]; not with act
 *   scratch  gmm_matvec_scratch_bytes() bytes, 16-byte aligned (NULL for none); calls that may run
 *            at the same time need one each
 *   out      [tokens, topk, n] or (weights) [tokens, n], n / 2 with act; BF16 or F32
 * k % group == 0, n % 8 == 0 (% 16 with act); x, codes, scale, zero 16-byte aligned, x_ld a
 * multiple of 8; topk <= GMM_MAX_TOPK; num_experts <= GMM_MAX_GROUPS.
 */
int gmm_matvec_int4(const void* x, int64_t tokens, int64_t k, int64_t x_ld, int x_per_slot, const void* codes,
                    const void* scale, const void* zero, int32_t group, int32_t num_experts, int64_t n,
                    const int32_t* experts, int32_t topk, const float* weights, int act, void* out, int out_dtype,
                    void* scratch, size_t scratch_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBGMM_EXPERTS_H_ */
