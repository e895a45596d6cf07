/*
 * beam_decode.h -- C ABI of the decode operators of libbeam_boundary.so (sm_103a): attention over
 * the KV cache that the Q/K calls of beam_boundary.h write, for a batch that may share a long
 * prefix; eviction from that cache by accumulated attention weight; and the matrix-vector products
 * with 4-bit weights for the projections around attention.
 *
 * The conventions of beam_boundary.h hold here too: device pointers on the current device, buffers
 * owned by the caller, no allocation and no synchronisation, every argument checked before anything
 * is launched, calls asynchronous on `stream`, programmatic dependent launch.  Model parameters
 * (4-bit weights, scales, zeros) may be read before the preceding kernel of the stream has ended;
 * everything else is read, and every output written, only after it.  Calls on different streams
 * need workspaces of their own.  Waits inside the kernels are bounded; beam_device_faults() also
 * reports one that ran out, or a block that found its shared memory not aligned as its copies need,
 * after which the call's outputs are not to be used.
 */
#ifndef BEAM_DECODE_H
#define BEAM_DECODE_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#include "beam_boundary.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Attention of a decode batch over the slot cache, with a prefix that every sequence shares.
 *
 * The cache is the one beam_qk_norm_rope_kv_fwd / beam_qk_norm_ssmax_kv_fwd write: k_cache, v_cache
 * [num_slots, n_kv_heads, 128], BF16 (cache_dtype 0) or FP8 E4M3 of value / scale (cache_dtype 1).
 * The keys of sequence b, in order, are the n_prefix slots prefix_slots[0..n_prefix) that all
 * sequences share and the suffix slots slot_table[b, 0..len_b), len_b = suffix_len[b] limited to
 * [0, table_width]: the sequence's own tokens, the q_len query tokens last.  Prefix keys and values
 * are read once for the whole batch (a prefix of up to 256 keys: once a sequence, out of the L2 cache).
 *
 * Query i of sequence b (row t = b*q_len + i) stands at suffix index p = len_b - q_len + i.  A row
 * with p < 0 is padding: it sees nothing.  Others see suffix keys j <= p with p - j < window and
 * prefix keys j with n_prefix + p - j < window (window 0: no limit).  A key whose slot lies outside
 * [0, num_slots) is not seen and not read, whatever its row.  For head h, with KV head
 * h / (n_q_heads / n_kv_heads):
 *   s_j = sm_scale * k_scale * <q, k_j>      (FP32 sums of the exact products)
 *   lse = log(sum_j exp(s_j))                 out = bf16(v_scale * sum_j exp(s_j - lse) v_j)
 * A row that sees nothing gives out = 0 and lse = -inf.  Scores, maxima, sums and outputs are FP32;
 * the weights exp(s_j - max) are rounded to BF16 (BF16 cache) or FP16 (FP8 cache) where they
 * multiply the values: an error of at most 2^-8 of each (BF16), of 2^-11 of each and 2^-32 of the
 * largest (FP16, scaled up by a power of two first).  For an FP8 cache the query row is
 * taken in FP16 after an exact scaling by a power of two (at most 2^60) that brings its largest
 * element to [2^14, 2^15), so that only elements 2^-28 below the largest (or below 2^-74) lose bits.
 * If key_weight_out is given, the weight that each suffix key received is added up:
 *   key_weight_out[b, j] = key_weight_in[b, j] + sum over i, h of exp(s_j - lse)   for j < len_b,
 *   and key_weight_in[b, j] for the others    (key_weight_in NULL: 0)
 * Results do not depend on the order in which blocks run.
 *
 *   out  [B*q_len, n_q_heads, 128] bf16, row t at out + t*out_row_stride (elements)
 *   q    the same shape at q_row_stride; both strides >= n_q_heads*128 and multiples of 8
 *   prefix_slots [n_prefix] int64 (NULL if n_prefix is 0)
 *   slot_table [B, table_width] int64, rows table_stride elements apart
 *   suffix_len [B] int32
 *   lse_out [B*q_len, n_q_heads] fp32 or NULL
 *   key_weight_in, key_weight_out [B, table_width] fp32, rows weight_stride elements apart, or
 *     NULL; they may be the same buffer (no other overlap of an output with anything is allowed)
 *   workspace: at least beam_attn_prefix_workspace(...) bytes, 16-byte aligned; its contents need
 *     not be kept or cleared between calls
 * num_slots in [0, 2^31); n_q_heads a multiple of n_kv_heads, at most 1024; head_dim must be 128
 * (BEAM_ERR_UNSUPPORTED otherwise, as for other cache types); sm_scale finite; k_scale, v_scale
 * finite and > 0 for FP8 (ignored for BF16); B*q_len*n_q_heads < 2^31; n_prefix, table_width in
 * [0, 2^31); q_len >= 1; window >= 0.  B == 0 returns BEAM_OK without launching. */
BEAM_API int beam_attn_prefix_fwd(
    void *out, int64_t out_row_stride, float *lse_out, const float *key_weight_in,
    float *key_weight_out, int64_t weight_stride, const void *q, int64_t q_row_stride,
    const void *k_cache, const void *v_cache, int64_t num_slots, int32_t cache_dtype, float k_scale,
    float v_scale, const int64_t *prefix_slots, int64_t n_prefix, const int64_t *slot_table,
    int64_t table_stride, int64_t table_width, const int32_t *suffix_len, int32_t B, int32_t q_len,
    int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, float sm_scale, int64_t window,
    void *workspace, int64_t workspace_bytes, cudaStream_t stream);

/* Bytes of workspace the call above needs for these sizes (key_weights != 0: with
 * key_weight_out), or a negative beam_status_t.  Host only.  Key weights keep every score of the
 * suffixes: 4 bytes for each row, head and (padded to 8) table place, B*q_len*n_q_heads*table_width*4
 * in all (128 sequences of 4 tokens and 48 heads in tables of 32,768: 3.2 GB); the rest is some MB for
 * a decode batch. */
BEAM_API int64_t beam_attn_prefix_workspace(int32_t B, int32_t q_len, int32_t n_q_heads,
                                            int32_t n_kv_heads, int64_t n_prefix,
                                            int64_t table_width, int64_t window,
                                            int32_t key_weights);

/* Eviction from the cache: each sequence keeps at most `budget` entries of its slot table.
 *
 * Row r has n = len_in[r] (limited to [0, width]) entries with their accumulated attention weights.
 * If n <= budget all stay.  Otherwise its last `recent` entries stay, and of the older ones the
 * budget - recent with the largest weight (ties: the lower index stays; NaN below every number;
 * -0 equals +0).  The entries that stay keep their order and move to the row's start:
 *   table_out[r, 0..m), weight_out[r, 0..m), m = len_out[r] = min(n, budget); behind them -1 and 0
 *   freed_out[r, 0..n-m): the slots of the entries that left, in their order; behind them -1
 * Weights are moved, not computed: bit for bit.
 *
 *   table_in, table_out [rows, width] int64; weight_in, weight_out [rows, width] fp32;
 *   len_in, len_out [rows] int32; freed_out [rows, freed_width] int64, freed_width >=
 *   max(0, width - budget) (may be NULL if that is 0).  All contiguous.  Each output may be the
 *   same buffer as its input; no other overlap.
 * rows in [0, 2^31), width in [0, 2^30); 0 <= recent <= budget. */
BEAM_API int beam_kv_evict_fwd(int64_t *table_out, int32_t *len_out, float *weight_out,
                               int64_t *freed_out, int64_t freed_width, const int64_t *table_in,
                               const int32_t *len_in, const float *weight_in, int64_t rows,
                               int64_t width, int64_t budget, int64_t recent, cudaStream_t stream);

/* Products of a few tokens with a matrix of 4-bit weights:
 *   y[t, n] = bf16( sum_k x[t, k] * (w[n, k] - z[n, k / group]) * scale[n, k / group] )
 * The products of 32 to 128 consecutive k of a group are summed in FP32 from exact values
 * x * (w - z), scaled in FP32, and these sums added in FP32 in a fixed order; one rounding to BF16.
 *
 *   y [T, N] bf16, row t at y + t*y_row_stride (elements, >= N; any alignment of 2 bytes)
 *   x [T, K] bf16, row t at x + t*x_row_stride (>= K, a multiple of 8; 16-byte aligned)
 *   w [N, K/2] bytes, contiguous, 16-byte aligned: byte k/2 holds weight k (even k) in its low and
 *     weight k + 1 in its high four bits, 0..15
 *   scales [N, K/group] bf16 (2-byte aligned); zeros [N, K/group] bytes, 0..15 (the low four bits
 *     are taken), or NULL: 8 everywhere
 * group 32, 64 or 128 (else BEAM_ERR_UNSUPPORTED); K a positive multiple of it; N >= 1; T >= 0. */
BEAM_API int beam_w4_matvec_fwd(void *y, int64_t y_row_stride, const void *x, int64_t x_row_stride,
                                const void *w, const void *scales, const void *zeros, int64_t T,
                                int64_t N, int64_t K, int32_t group, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BEAM_DECODE_H */
