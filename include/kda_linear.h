/*
 * kda_linear.h — linear attention with one decay per head (libkda.so).
 *
 * The operation.  For one sequence and one head, with a d_k x d_v state S
 * (rows = key channels, columns = value channels), every token t applies
 *
 *     S_t = a_t S_{t-1} + k_t v_t^T
 *     o_t = S_t^T q_t                      (read after token t's own write)
 *
 * with a_t = exp(log_decay_t) one scalar per token and head, or one constant
 * per head: the recurrence of kda.h without its erase term and with the same
 * decay for every key channel.  There is no scale on q: o is linear in q, so
 * a caller folds one into it.
 *
 * The conventions of kda.h hold (device pointers, streams, statuses, dense
 * layouts, d_k = d_v = 128, KDA_DEBUG_CHECKS), with these shapes:
 *
 *   q, k        [T_total, num_qk_heads, 128] dtype.  num_heads is a multiple
 *               of num_qk_heads: head h reads query and key head
 *               h / (num_heads / num_qk_heads).
 *   v, o        [T_total, num_heads, 128] dtype
 *   log_decay   [T_total, num_heads] fp32, or [num_heads] fp32 when
 *               decay_per_head is nonzero.  Any value <= 0, -inf included
 *               (the state is dropped before the token's write, whatever it
 *               holds); positive values and NaN are outside the preconditions.
 *   states      [N, num_heads, 128, 128] fp32
 *
 * Preconditions not checked on the fast path: log_decay as above; q, k, v and
 * the gradients finite, and so are states that no decay of -inf drops before
 * they are read; sums of k v^T below 2^97 (the walk holds up to 2^30 times the
 * state); cu_seqlens non-decreasing from 0 to total_tokens.
 * Outside them the results are undefined but every access stays in bounds.
 * The device the stream belongs to has to be the current one.
 *
 * Accuracy.  fp32 results (fp32 I/O, states, d_log_decay) are computed to
 * fp32 accuracy also from bf16 inputs.  bf16 results of the chunk calls carry
 * three roundings to bf16: their own, that of the products q . k as an operand
 * of the last product, and that of the state as one (together 1.4 times the
 * error of the first alone); those of the decode step only their own.  Every
 * sum runs in a fixed order: repeated calls give the same bits, and o and dv do
 * not depend on which states are asked for.  bf16 dq and dk may differ in
 * their last bit with and without d_log_decay, which reads more of the state.
 */
#ifndef KDA_LINEAR_H_
#define KDA_LINEAR_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Bytes of device workspace kda_linear_chunk_fwd needs (host-side; it reads
 * the current device's compute-unit count).  0 is a valid answer (no
 * workspace is needed); invalid sizes give 0 as well.
 */
size_t kda_linear_chunk_fwd_workspace_bytes(int num_seqs, int64_t total_tokens, int num_heads, int num_qk_heads,
                                            int d_k, int d_v, kda_dtype dtype, int segment_tokens);

/*
 * Prefill over a packed batch: sequence n owns tokens
 * [cu_seqlens[n], cu_seqlens[n+1]).
 *
 *   initial_state  [N, H, 128, 128] fp32 or NULL for zeros; may be exactly
 *                  final_state (in-place continuation)
 *   cu_seqlens     device int32 [N+1], or NULL (then N must be 1).  Empty
 *                  sequences are allowed: their final state is the initial one.
 *   num_heads      1 .. 65535
 *   segment_tokens 0: the library chooses whether to cut sequences into
 *                  segments that run side by side; a positive multiple of 64
 *                  forces segments of that length, a negative value keeps
 *                  each sequence in one walk.  The workspace query and the
 *                  call must be given the same value.
 *   o              must not overlap any input
 *   final_state    fp32 output or NULL (not written)
 */
kda_status kda_linear_chunk_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                                const float* initial_state, const int32_t* cu_seqlens, int num_seqs,
                                int64_t total_tokens, int num_heads, int num_qk_heads, int decay_per_head, int d_k,
                                int d_v, kda_dtype dtype, int segment_tokens, void* o, float* final_state,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Bytes of device workspace kda_linear_chunk_bwd needs (0 as above).
 * need_d_log_decay and with_d_final_state: whether the call is given
 * d_log_decay and d_final_state.
 */
size_t kda_linear_chunk_bwd_workspace_bytes(int num_seqs, int64_t total_tokens, int num_heads, int num_qk_heads,
                                            int decay_per_head, int need_d_log_decay, int with_d_final_state, int d_k,
                                            int d_v, kda_dtype dtype, int segment_tokens);

/*
 * Gradients of  L = sum_t <d_o_t, o_t> + <d_final_state, S_T>.
 *
 *   d_o             [T_total, H, 128] dtype
 *   d_final_state   [N, H, 128, 128] fp32 or NULL (zero)
 *   dq, dk          [T_total, num_qk_heads, 128] dtype: summed over the heads
 *                   that share a query and key head (in fp32, then rounded)
 *   dv              [T_total, H, 128] dtype
 *   d_log_decay     fp32, the shape of log_decay (summed over all tokens for
 *                   a constant decay), or NULL (not computed: less work)
 *   d_initial_state [N, H, 128, 128] fp32 or NULL (not written)
 *
 * It needs only the forward's inputs; no output may overlap an input, another
 * output or the workspace.  With d_log_decay, total_tokens * num_heads / 1024
 * (a constant decay: / 256; with segments the largest multiple of 64 up to that
 * which divides their length) + 2 * num_seqs * num_heads is at most 14 * 2^20.
 */
kda_status kda_linear_chunk_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                                const float* initial_state, const int32_t* cu_seqlens, const void* d_o,
                                const float* d_final_state, int num_seqs, int64_t total_tokens, int num_heads,
                                int num_qk_heads, int decay_per_head, int d_k, int d_v, kda_dtype dtype,
                                int segment_tokens, void* dq, void* dk, void* dv, float* d_log_decay,
                                float* d_initial_state, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One token for N independent sequences, the states advanced in place
 * (num_seqs * num_heads below 2^24).
 *
 *   state      [N, H, 128, 128] fp32, 16-byte aligned
 *   q, k       [N, num_qk_heads, 128] dtype;  v, o  [N, H, 128] dtype
 *   log_decay  [N, H] fp32, or [H] with decay_per_head
 */
kda_status kda_linear_decode_step(float* state, const void* q, const void* k, const void* v, const float* log_decay,
                                  int num_seqs, int num_heads, int num_qk_heads, int decay_per_head, int d_k, int d_v,
                                  kda_dtype dtype, void* o, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LINEAR_H_ */
