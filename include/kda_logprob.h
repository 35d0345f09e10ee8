/*
 * kda_logprob.h — log probabilities of tokens from logits (libkda.so).
 *
 * Of each row of logits x over a vocabulary of V tokens, with
 * z = log sum_t e^{x_t} and p_t = e^{x_t - z}: the log probability x_t - z of a
 * given token, the entropy - sum_t p_t log p_t, z itself, and the most probable
 * tokens with theirs.  What a training loss and its gradient, the verification
 * of drafted tokens and the scores of a prompt's tokens are made of.
 *
 * As in kda_beam.h, -inf and NaN are masked tokens (probability zero) and +inf
 * counts as the largest finite number.  A row that is masked throughout has
 * z = -inf, entropy 0, log probabilities -inf and no gradient.
 *
 * The conventions of kda.h hold (device pointers, streams, statuses).  The
 * device the stream belongs to has to be the current one.
 */
#ifndef KDA_LOGPROB_H_
#define KDA_LOGPROB_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_LOGPROB_TOP_MAX 16 /* alternatives of a row */

/*
 * One pass over the logits; no workspace.
 *
 *   logits        [rows, vocab] dtype (KDA_DTYPE_F32 or _BF16), row r at
 *                 logits + r * row_stride elements (row_stride >= vocab), of
 *                 any alignment
 *   tokens        [rows] int32 or NULL.  A row whose token is outside
 *                 0 .. vocab - 1 has the log probability 0 (padding).
 *   rows          0 .. 2^21
 *   top           0 .. min(vocab, KDA_LOGPROB_TOP_MAX) alternatives
 *                 (more: KDA_ERR_UNSUPPORTED)
 *   logprobs      [rows] fp32, given exactly when tokens is
 *   entropy, log_sum   [rows] fp32, each or NULL
 *   top_logprobs  [rows, top] fp32, descending, and
 *   top_tokens    [rows, top] int32, given exactly when top > 0: ties go to the
 *                 lowest token, masked tokens come last
 * Sums of exponentials are taken relative to the row's largest logit and are
 * accurate to fp32.  They run in a fixed order: repeated calls give the same
 * bits.  No output may overlap an input or another output.
 */
kda_status kda_token_logprobs_fwd(const void* logits, const int32_t* tokens, int64_t rows, int vocab,
                                  int64_t row_stride, int top, kda_dtype dtype, float* logprobs, float* entropy,
                                  float* log_sum, float* top_logprobs, int32_t* top_tokens, hipStream_t stream);

/*
 * The gradient of  L = sum_r d_logprobs_r logprob_r + d_entropy_r entropy_r:
 *
 *     d x_t = d_logprobs (1{t = token} - p_t) - d_entropy p_t (log p_t + entropy)
 *
 *   log_sum, entropy  the forward call's (entropy: with d_entropy, else ignored).
 *                     p comes from x - log_sum in fp32: its relative error is
 *                     half a step of log_sum, at most 2^-15 (bf16: 2^-13).
 *                     Rows whose log_sum is 1024 (4096) or more in size are
 *                     read once more, by one workgroup each, and p is taken
 *                     relative to their largest logit; a log_sum that is not
 *                     the row's own is taken as it is.
 *   d_logprobs    [rows] fp32; not read where the token is outside 0 .. vocab - 1
 *   d_entropy     [rows] fp32 or NULL (zero)
 *   d_logits      [rows, vocab] dtype, row r at d_logits + r * d_row_stride; may
 *                 be exactly logits with the same stride (in place).  Elements
 *                 between the rows are not touched.
 */
kda_status kda_token_logprobs_bwd(const void* logits, const int32_t* tokens, const float* log_sum,
                                  const float* entropy, const float* d_logprobs, const float* d_entropy, int64_t rows,
                                  int vocab, int64_t row_stride, int64_t d_row_stride, kda_dtype dtype, void* d_logits,
                                  hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LOGPROB_H_ */
