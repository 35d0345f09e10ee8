/*
 * kda_delta.h — the gated delta rule with one decay per head (libkda.so).
 *
 * The operation.  For one sequence and one head, with a d_k x d_v state S
 * (rows = key channels, columns = value channels), every token t applies
 *
 *     S~_t = a_t S_{t-1}
 *     u_t  = beta_t (v_t - S~_t^T k_t)
 *     S_t  = S~_t + k_t u_t^T
 *     o_t  = S_t^T q_t                      (read after token t's own write)
 *
 * with a_t = exp(log_decay_t) one scalar per token and head: the recurrence of
 * kda.h with the same decay for every key channel, and that of kda_linear.h
 * with the erase term.  Decays of zero logarithm give the plain delta rule.
 * There is no scale on q: o is linear in q, so a caller folds one into it.
 *
 * The conventions of kda.h hold (device pointers, streams, statuses, dense
 * layouts, d_k = d_v = 128, KDA_DEBUG_CHECKS), with these shapes:
 *
 *   q, k        [T_total, num_qk_heads, 128] dtype.  num_heads is a multiple
 *               of num_qk_heads: head h reads query and key head
 *               h / (num_heads / num_qk_heads).
 *   v, o        [T_total, num_heads, 128] dtype
 *   log_decay   [T_total, num_heads] fp32, any value <= 0, -inf included (the
 *               state is dropped before the token reads and writes it)
 *   beta        [T_total, num_heads] fp32 in [0, 1]
 *   states      [N, num_heads, 128, 128] fp32
 *
 * Preconditions not checked on the fast path: log_decay and beta as above; the
 * length of every k row at most 1 (longer ones make the recurrence grow); q, k,
 * v, the gradients and the states finite, but a state that the sequence's first
 * decay drops may hold anything; cu_seqlens non-decreasing from 0 to
 * total_tokens.  Outside them the results are undefined but every access stays
 * in bounds.  The device the stream belongs to has to be the current one.
 *
 * Accuracy.  fp32 results are computed to fp32 accuracy also from bf16 inputs
 * (products of 22 bits, fp32 sums), relative to unit length of the keys, to the
 * largest of the same row of q, and to the largest of the same value channel of
 * the state and of the chunk's beta v, a chunk being up to 64 tokens, later ones
 * included (backwards: of dS, and of d_o times the largest of its row of q): an
 * output may be off by 2^-19 of that largest times its row of q, however small
 * it is itself, and so may the state be that a chunk leaves to the next one, from
 * where on that decays as the state does.  bf16 results are off by their own rounding besides, 1.7e-3 in norm;
 * dq and dk, some of whose operands are fp16, by up to 3e-3 where keys are
 * nearly the same through a chunk and beta is near 1.  A decay below
 * 2^-126 counts as zero.  Every sum runs in a fixed order: repeated calls give
 * the same bits.
 */
#ifndef KDA_DELTA_H_
#define KDA_DELTA_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Bytes of device workspace kda_delta_chunk_fwd needs (host-side; it reads the
 * current device's compute-unit count): about 200 a token and head, and with
 * segments two states for each.  Invalid sizes give 0.
 */
size_t kda_delta_chunk_fwd_workspace_bytes(int num_seqs, int64_t total_tokens, int num_heads, int num_qk_heads,
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
kda_status kda_delta_chunk_fwd(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                               const float* initial_state, const int32_t* cu_seqlens, int num_seqs,
                               int64_t total_tokens, int num_heads, int num_qk_heads, int d_k, int d_v,
                               kda_dtype dtype, int segment_tokens, void* o, float* final_state, void* workspace,
                               size_t workspace_bytes, hipStream_t stream);

/* Bytes of device workspace kda_delta_chunk_bwd needs (0 as above): about 2.6 KiB
 * a token and head in bf16 (5.6 in fp32), every sequence counted as a chunk of 64
 * tokens (32) longer, and 128 KiB a sequence and head. */
size_t kda_delta_chunk_bwd_workspace_bytes(int num_seqs, int64_t total_tokens, int num_heads, int num_qk_heads,
                                           int d_k, int d_v, kda_dtype dtype, int segment_tokens);

/*
 * Gradients of  L = sum_t <d_o_t, o_t> + <d_final_state, S_T>.
 *
 *   d_o             [T_total, H, 128] dtype
 *   d_final_state   [N, H, 128, 128] fp32 or NULL (zero)
 *   dq, dk          [T_total, num_qk_heads, 128] dtype: summed over the heads
 *                   that share a query and key head (in fp32, then rounded)
 *   dv              [T_total, H, 128] dtype
 *   d_log_decay, dbeta  [T_total, H] fp32, each or NULL (not written)
 *   d_initial_state [N, H, 128, 128] fp32 or NULL (not written)
 *
 * It needs only the forward's inputs; no output may overlap an input, another
 * output or the workspace.  total_tokens * num_heads / 512 + 2 * num_seqs *
 * num_heads is at most 14 * 2^20.  bf16 dq and dk take the states and the values
 * written, rounded to fp16, as operands.
 */
kda_status kda_delta_chunk_bwd(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                               const float* initial_state, const int32_t* cu_seqlens, const void* d_o,
                               const float* d_final_state, int num_seqs, int64_t total_tokens, int num_heads,
                               int num_qk_heads, int d_k, int d_v, kda_dtype dtype, int segment_tokens, void* dq,
                               void* dk, void* dv, float* d_log_decay, float* dbeta, float* d_initial_state,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One token for N independent sequences, the states advanced in place
 * (num_seqs * num_heads below 2^24).
 *
 *   state      [N, H, 128, 128] fp32, 16-byte aligned
 *   q, k       [N, num_qk_heads, 128] dtype;  v, o  [N, H, 128] dtype
 *   log_decay, beta  [N, H] fp32
 * A state whose decay is zero is dropped, whatever it holds.
 */
kda_status kda_delta_decode_step(float* state, const void* q, const void* k, const void* v, const float* log_decay,
                                 const float* beta, int num_seqs, int num_heads, int num_qk_heads, int d_k, int d_v,
                                 kda_dtype dtype, void* o, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_DELTA_H_ */
