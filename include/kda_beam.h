/*
 * kda_beam.h — beam search over recurrent states (libkda.so).
 *
 * A group is one prompt with `beams` hypotheses; beam k of group b is row
 * b * beams + k of every tensor that holds something per sequence (the states
 * of kda_decode_step, kda_decode_replay and kda_linear_decode_step, the
 * convolution histories).  One step of the search: decode a token for every
 * row, kda_beam_select over the logits, kda_beam_reorder of the states.
 *
 * The conventions of kda.h hold (device pointers, streams, statuses).  The
 * device the stream belongs to has to be the current one.
 */
#ifndef KDA_BEAM_H_
#define KDA_BEAM_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_BEAM_MAX 16         /* beams of a group */
#define KDA_BEAM_REORDER_MAX 8  /* state tensors of one kda_beam_reorder call */

/* Bytes of device workspace kda_beam_select needs (0 for invalid sizes). */
size_t kda_beam_select_workspace_bytes(int groups, int beams, int vocab, kda_dtype dtype);

/*
 * The best `beams` continuations of each group.  Candidate (k, t) has the score
 *
 *     scores[k] + logits[k][t] - log sum_t' exp(logits[k][t'])
 *
 * and a finished beam has only its end_token, at scores[k]; everything else of
 * it counts as -inf.  The candidates with the largest scores are taken, in
 * descending order, ties to the lowest k * vocab + t.  Within a beam, logits
 * are compared exactly; between beams, scores in fp64 (the sum of
 * exponentials is accurate to fp32).
 *
 *   logits       [groups, beams, vocab] dtype (KDA_DTYPE_F32 or _BF16), rows of
 *                any length and alignment.  -inf and NaN are masked tokens,
 *                +inf counts as the largest finite number.  A row that is
 *                masked throughout has only candidates at -inf.
 *   scores       [groups, beams] fp32, finite or -inf (a beam that does not
 *                exist: at the first step all but one; its logits are not read)
 *   finished     [groups, beams] bytes (0 or 1), or NULL; the logits of a
 *                finished beam are not read
 *   end_token    0 .. vocab - 1 with finished, else ignored
 *   beams        1 .. KDA_BEAM_MAX (more: KDA_ERR_UNSUPPORTED)
 *   out_scores   [groups, beams] fp32, may be exactly `scores`
 *   out_tokens   [groups, beams] int32
 *   out_parents  [groups, beams] int32: the beam of the group that was continued
 *   out_finished [groups, beams] bytes, given exactly when finished is; may be
 *                exactly `finished`.  Set where the parent was finished or the
 *                token is end_token.
 *   workspace    at least kda_beam_select_workspace_bytes() bytes
 * Where fewer than `beams` candidates are above -inf, the rest are those at
 * -inf with the lowest k * vocab + t.
 */
kda_status kda_beam_select(const void* logits, const float* scores, const uint8_t* finished, int groups, int beams,
                           int vocab, int end_token, kda_dtype dtype, float* out_scores, int32_t* out_tokens,
                           int32_t* out_parents, uint8_t* out_finished, void* workspace, size_t workspace_bytes,
                           hipStream_t stream);

/*
 * Rows of the states follow the selected parents, in place:
 *
 *     states[s][b * beams + k] <- states[s][b * beams + parents[b][k]]
 *
 * for every k of a group at once.  No workspace; rows that stay are not
 * touched, and neither are rows whose parent is outside 0 .. beams - 1.
 *
 *   states     num_states device pointers (host array), each to groups * beams
 *              rows of row_bytes[s] bytes, of any type and alignment (16-byte
 *              aligned rows move as vectors)
 *   row_bytes  host array
 *   num_states 1 .. KDA_BEAM_REORDER_MAX (more: KDA_ERR_UNSUPPORTED)
 *   parents    [groups, beams] int32
 * The tensors must not overlap one another or parents.
 */
kda_status kda_beam_reorder(void* const* states, const int64_t* row_bytes, int num_states, const int32_t* parents,
                            int groups, int beams, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_BEAM_H_ */
