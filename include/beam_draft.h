/*
 * beam_draft.h -- C ABI of the operators of a decode step that checks drafted tokens
 * (libbeam_boundary.so, sm_103a): a KV cache held in 4 bits, with the write that fills it and the
 * attention that reads it; a whole mixture-of-experts layer for the step's few tokens; and the
 * verification of the drafted tokens against the target's probabilities.
 *
 * The conventions of beam_boundary.h and beam_decode.h hold here too: device pointers on the current
 * device, buffers owned by the caller, no allocation and no synchronisation, every argument checked
 * before anything is launched, calls asynchronous on `stream`, programmatic dependent launch.  The
 * router's weights and bias may be read before earlier kernels of the stream have ended (more than one of them:
 * kernels here let the next one start before they wait themselves); everything else is read, and every output
 * written, only after them.  Calls on different streams need workspaces of their
 * own; a workspace's contents need not be kept or cleared between calls.  A kernel here waits for its own block's or
 * cluster's threads and copies, and attention's, behind the earlier kernels of its stream, for tensor memory, until other
 * streams' kernels on its SM give theirs back.  None holds tensor memory while it waits for another kernel.
 */
#ifndef BEAM_DRAFT_H
#define BEAM_DRAFT_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#include "beam_boundary.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Write of keys and values into a cache held in 4 bits.
 *
 * The cache holds each token's row of a KV head in groups of `group` = 32, 64 or 128 columns:
 *   k_cache, v_cache [num_slots, n_kv_heads, 64] bytes: byte c/2 holds the code 0..15 of column c (even
 *     c) in its low and that of column c + 1 in its high four bits
 *   k_scales, v_scales [num_slots, n_kv_heads, 128 / group, 2] bf16: the group's scale and minimum
 * A code stands for the value minimum + scale * code.  For the values x of a group, with FP32 arithmetic
 * and IEEE division:
 *   minimum = min x (a BF16 value, so held exactly)      scale = bf16((max x - min x) / 15)
 *   code = min(rint((x - minimum) / scale), 15)          (scale 0: code 0)
 * A group that holds an infinity or NaN, or whose max - min is not finite, gets the scale NaN, minimum 0
 * and codes 0: it reads as NaN.  Each value is off by at most half a scale and by what the scale's
 * rounding takes off the top code, 15 * 2^-8 of a scale (half a step of BF16 is at most 2^-8).
 * Token t goes to slot slot_mapping[t]; one outside [0, num_slots) is not written.  Slots must differ
 * (else which of the tokens a slot holds is not defined).  Other slots keep what they hold.
 *
 *   k, v [T, n_kv_heads, 128] bf16, rows k_row_stride / v_row_stride elements apart (>= n_kv_heads*128,
 *     multiples of 8; 16-byte aligned)
 *   slot_mapping [T] int64; the caches 16-byte, the scales 128 / group * 4-byte aligned
 * num_slots in [0, 2^31), T in [0, 2^31), n_kv_heads in [1, 1024]; head_dim must be 128. */
BEAM_API int beam_kv4_write_fwd(void *k_cache, void *v_cache, void *k_scales, void *v_scales,
                                int64_t num_slots, int32_t group, const void *k, int64_t k_row_stride,
                                const void *v, int64_t v_row_stride, const int64_t *slot_mapping,
                                int64_t T, int32_t n_kv_heads, int32_t head_dim, cudaStream_t stream);

/* Attention of a decode batch over a cache held in 4 bits (layout above).
 *
 * The keys of sequence b, in order, are the slots slot_table[b, 0..len_b), len_b = seq_len[b] limited to
 * [0, table_width], the q_len query tokens last.  Query i of sequence b (row t = b*q_len + i) stands at
 * p = len_b - q_len + i; a row with p < 0 is padding and sees nothing.  Others see the keys j <= p with
 * p - j < window or j < n_sink (window 0: all j <= p): a sliding window with the first tokens in sight.
 * A key whose slot lies outside [0, num_slots) is not seen and not read.  For head h, with KV head
 * h / (n_q_heads / n_kv_heads) and the keys and values k_j, v_j that the codes stand for:
 *   s_j = sm_scale * <q, k_j>    lse = log(sum_j exp(s_j))    out = bf16(sum_j exp(s_j - lse) v_j)
 * A row that sees nothing gives out = 0 and lse = -inf.  Nothing of a key reaches a row that does not
 * see it, whatever it holds; NaN in a key that it sees shows, whatever its weight.  <q, k_j> is formed per group as scale * sum q c + minimum * sum q with FP32
 * sums; products q c are exact: the query row is taken in FP16 after an exact scaling by a power of two (at
 * most 2^60) to [2^14, 2^15), so that only elements 2^-27 below the row's largest (or below 2^-74) lose
 * bits.  Maxima, sums and outputs are FP32.  The products exp(s_j - max) * scale that multiply the values'
 * codes are rounded to FP16, scaled up by a power of two: an error of at most 2^-11 of each and of 2^-32 of
 * the largest scale that the row has seen (of 2^-100 if that is less); minima are added in FP32.
 * A row whose largest |q| times |sm_scale| reaches 2^117, or whose keys' |v_j| add up to more than FP32 holds (sums are
 * formed before their division), may give infinities and NaN; other rows are as they are.
 * Results do not depend on the order in which blocks run.
 *
 *   out, q [B*q_len, n_q_heads, 128] bf16, rows *_row_stride elements apart (>= n_q_heads*128, multiples
 *     of 8; 16-byte aligned)
 *   slot_table [B, table_width] int64, rows table_stride elements apart; seq_len [B] int32
 *   lse_out [B*q_len, n_q_heads] fp32 or NULL
 *   workspace: at least beam_attn_kv4_workspace(...) bytes, 16-byte aligned
 * num_slots in [0, 2^31); n_q_heads a multiple of n_kv_heads, at most 1024; head_dim must be 128 and group
 * 32, 64 or 128; sm_scale finite; B*q_len*n_q_heads < 2^31; table_width in [0, 2^30); q_len >= 1;
 * window, n_sink >= 0; B * ceil(table_width / 32) below 2^31.  B == 0 returns BEAM_OK without launching.  No
 * output may overlap anything. */
BEAM_API int beam_attn_kv4_fwd(void *out, int64_t out_row_stride, float *lse_out, const void *q,
                               int64_t q_row_stride, const void *k_cache, const void *v_cache,
                               const void *k_scales, const void *v_scales, int64_t num_slots,
                               int32_t group, const int64_t *slot_table, int64_t table_stride,
                               int64_t table_width, const int32_t *seq_len, int32_t B, int32_t q_len,
                               int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, float sm_scale,
                               int64_t window, int64_t n_sink, void *workspace,
                               int64_t workspace_bytes, cudaStream_t stream);

/* Bytes of workspace the call above needs for these sizes, or a negative beam_status_t.  Host only. */
BEAM_API int64_t beam_attn_kv4_workspace(int32_t B, int32_t q_len, int32_t n_q_heads,
                                         int32_t n_kv_heads, int64_t table_width, int64_t window,
                                         int64_t n_sink);

/* A whole mixture-of-experts layer for a few tokens: router, grouped top-k, experts, weighted sum.
 *
 *   z[t, e] = <x[t], router_w[e]>                             (all 256 experts)
 *   ids, w  = beam_grouped_topk_fwd(z, router_bias)           (8 groups, 4 of them, 8 experts)
 *   g = w_gate_up[e, 0..F) x[t]    u = w_gate_up[e, F..2F) x[t]    a = g / (1 + exp(-g)) * u
 *   out[t] = bf16( sum over k of (routed_scaling * w[t, k]) * w_down[ids[t, k]] a[t, k] )
 * The logits z are sums of the exact products in FP32 pairs, rounded once to FP32, so that the choice does
 * not hang on the order of a sum.  The experts' sums, g, u and the sum over k (in the order of k) are
 * FP32; a goes into the down product as the sum of two BF16 values, its
 * rounding and the rounding of the rest (an error of at most 2^-16 of each).
 * The call computes the part of the experts [first_expert, first_expert + n_local), whose weights it gets
 * (the others are another rank's), with F their intermediate columns on this rank: for expert- and
 * tensor-parallel shares `out` is a partial sum for beam_allreduce_boundary_fwd, for the whole layer it
 * goes to beam_boundary_fwd.  A token none of whose experts is in the range gives a row of zeros.
 * A token with a NaN in x, or whose largest |x| times the largest |router_w| of an expert reaches 2^113 (the sum may pass
 * FP32's range), may give any experts and NaN, and does not touch the other tokens' rows.  The
 * same holds for a token with an activation a beyond BF16's range, which gives NaN.
 *
 *   x, out [T, H] bf16, rows *_row_stride elements apart (>= H, multiples of 8; 16-byte aligned)
 *   router_w [256, H] fp32 (16-byte aligned), router_bias [256] fp32 (16-byte aligned)
 *   w_gate_up [n_local, 2*F, H], w_down [n_local, H, F] bf16, contiguous, 16-byte aligned
 *   topk_ids_out [T, 8] int32, topk_w_out [T, 8] fp32, or NULL: the experts chosen, best first, and their
 *     renormalised weights, as beam_grouped_topk_fwd gives them
 *   workspace: at least beam_moe_layer_workspace(...) bytes, 16-byte aligned
 * T in [0, 256] (BEAM_ERR_UNSUPPORTED above: such batches are for grouped library products); H and F
 * multiples of 8, H in [8, 16384], F in [8, 32768]; n_local in [1, 256], first_expert >= 0 and
 * first_expert + n_local <= 256; routed_scaling finite.  out may not overlap anything. */
BEAM_API int beam_moe_layer_fwd(void *out, int64_t out_row_stride, int32_t *topk_ids_out,
                                float *topk_w_out, const void *x, int64_t x_row_stride,
                                const float *router_w, const float *router_bias, const void *w_gate_up,
                                const void *w_down, int32_t first_expert, int32_t n_local,
                                float routed_scaling, int64_t T, int32_t H, int32_t F, void *workspace,
                                int64_t workspace_bytes, cudaStream_t stream);

/* Bytes of workspace the call above needs, or a negative beam_status_t.  Host only. */
BEAM_API int64_t beam_moe_layer_workspace(int64_t T, int32_t H, int32_t F, int32_t n_local);

/* Verification of drafted tokens against the target's probabilities, from given random numbers.
 *
 * Sequence b has n_b = draft_len[b] (limited to [0, k]; NULL: k) drafted tokens x_0, x_1, ...  With p_i the
 * target's and q_i the draft's distribution at position i (draft_probs NULL: all of q_i on x_i), x_i is
 * accepted if all before it were and  u_accept[b, i] * q_i(x_i) < p_i(x_i)  (exact products; false if one is
 * NaN or x_i lies outside [0, V)).  With a tokens accepted, one more is drawn:
 *   a < n_b:  from the weights max(P_a - Q_a, 0), or P_a where these are all zero
 *   a = n_b:  from the weights P_a
 * where P = rint(2^44 p), Q = rint(2^44 q) are the probabilities in units of 2^-44 (values outside [0, 1] are
 * limited to it, NaN counts as 0).  It is the smallest token v with
 *   sum of the weights up to v  >  floor(u * S),   S the sum of all, u = u_sample[b] limited to [0, 1)
 * and cut off to units of 2^-24 (NaN: 0), or -1 if all weights are zero.  All of it is whole-number arithmetic: results do
 * not depend on the order of any sum.  Over random
 * numbers this draws from the target's distribution, up to the units.
 *
 *   tokens_out [B, k + 1] int64: the accepted tokens, the drawn one, -1 behind them
 *   n_accepted_out [B] int32: a
 *   draft_tokens [B, k] int64; u_accept [B, k] fp32, u_sample [B] fp32, in [0, 1); draft_len [B] int32
 *   target_probs [B, k + 1, V], draft_probs [B, k, V] (or NULL): fp32 (dtype 0) or bf16 (dtype 1), rows of V
 *     contiguous, *_seq_stride elements from sequence to sequence and *_pos_stride from position to position,
 *     aligned to their element size
 * B in [0, 2^31), k in [0, 1024], V in [1, 2^20), strides >= 0. */
BEAM_API int beam_draft_verify_fwd(int64_t *tokens_out, int32_t *n_accepted_out,
                                   const int64_t *draft_tokens, const int32_t *draft_len,
                                   const void *target_probs, int64_t target_seq_stride,
                                   int64_t target_pos_stride, const void *draft_probs,
                                   int64_t draft_seq_stride, int64_t draft_pos_stride, int32_t dtype,
                                   const float *u_accept, const float *u_sample, int64_t B, int32_t k,
                                   int64_t V, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BEAM_DRAFT_H */
