// draft_api.cu -- C ABI of the operators of a draft-checking decode step: argument checks and launch.
// Every check runs before any CUDA call, so a rejected call launches nothing, touches no output and needs
// no GPU.

#include <cmath>
#include <cstdint>

#include "../../../include/beam_draft.h"
#include "draft_kernels.h"

namespace {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? BEAM_OK : BEAM_ERR_CUDA; }

constexpr int64_t kMost = (int64_t)1 << 31;
constexpr int32_t kMaxHeads = 1024;
constexpr int64_t kMaxMoeTokens = 256;
constexpr int32_t kExperts = 256;

bool good_group(int32_t group) { return group == 32 || group == 64 || group == 128; }

int check_attn_sizes(int32_t B, int32_t q_len, int32_t n_q, int32_t n_kv, int64_t width,
                     int64_t window, int64_t n_sink)
{
    if (B < 0 || q_len < 1 || n_kv < 1 || n_q < n_kv || n_q > kMaxHeads || n_q % n_kv != 0 ||
        width < 0 || width >= kMost / 2 || window < 0 || n_sink < 0)
        return BEAM_ERR_INVALID_ARG;
    if (B == 0)
        return BEAM_OK;  // nothing is planned: the bounds below, which are the plan's, hold for any other sizes
    // (and the kernel counts tiles of 32 keys in 31 bits)
    if ((int64_t)B * q_len >= kMost || (int64_t)B * q_len * n_q >= kMost ||
        (width + 31) / 32 * B >= kMost)
        return BEAM_ERR_INVALID_ARG;
    return BEAM_OK;
}

int check_moe_sizes(int64_t T, int32_t H, int32_t F, int32_t n_local)
{
    if (T < 0 || H < 8 || H > 16384 || H % 8 != 0 || F < 8 || F > 32768 || F % 8 != 0 ||
        n_local < 1 || n_local > kExperts)
        return BEAM_ERR_INVALID_ARG;
    return T > kMaxMoeTokens ? BEAM_ERR_UNSUPPORTED : BEAM_OK;
}

}  // namespace

extern "C" {

int beam_kv4_write_fwd(void *k_cache, void *v_cache, void *k_scales, void *v_scales,
                       int64_t num_slots, int32_t group, const void *k, int64_t k_row_stride,
                       const void *v, int64_t v_row_stride, const int64_t *slot_mapping, int64_t T,
                       int32_t n_kv_heads, int32_t head_dim, cudaStream_t stream)
{
    if (head_dim != 128 || !good_group(group))
        return BEAM_ERR_UNSUPPORTED;
    if (T < 0 || T >= kMost || n_kv_heads < 1 || n_kv_heads > kMaxHeads || num_slots < 0 ||
        num_slots >= kMost)
        return BEAM_ERR_INVALID_ARG;
    if (T == 0 || num_slots == 0)
        return BEAM_OK;
    const int64_t row = (int64_t)n_kv_heads * head_dim;
    if (!k_cache || !v_cache || !k_scales || !v_scales || !k || !v || !slot_mapping ||
        (T > 1 && (k_row_stride < row || v_row_stride < row)))
        return BEAM_ERR_INVALID_ARG;
    const uintptr_t sa = (uintptr_t)(128 / group * 4);
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scales, sa) ||
        !aligned(v_scales, sa) || !aligned(k, 16) || !aligned(v, 16) || k_row_stride % 8 != 0 ||
        v_row_stride % 8 != 0 || !aligned(slot_mapping, 8))
        return BEAM_ERR_MISALIGNED;
    beam::Kv4WriteArgs a{};
    a.cache[0] = (uint8_t *)k_cache;
    a.cache[1] = (uint8_t *)v_cache;
    a.scales[0] = k_scales;
    a.scales[1] = v_scales;
    a.src[0] = k;
    a.src[1] = v;
    a.src_stride[0] = k_row_stride;
    a.src_stride[1] = v_row_stride;
    a.num_slots = num_slots;
    a.slot = slot_mapping;
    a.T = T;
    a.n_kv = n_kv_heads;
    a.group = group;
    return cuda_status(beam::launch_kv4_write(a, stream));
}

int64_t beam_attn_kv4_workspace(int32_t B, int32_t q_len, int32_t n_q_heads, int32_t n_kv_heads,
                                int64_t table_width, int64_t window, int64_t n_sink)
{
    const int st =
        check_attn_sizes(B, q_len, n_q_heads, n_kv_heads, table_width, window, n_sink);
    if (st != BEAM_OK || B == 0)
        return st;
    // enough for a cache in any groups
    int64_t most = 0;
    for (int32_t group = 32; group <= 128; group *= 2) {
        const int64_t bytes = beam::kv4_attn_plan(B, q_len, n_q_heads, n_kv_heads, table_width, window,
                                                  n_sink, group)
                                  .bytes;
        most = bytes > most ? bytes : most;
    }
    return most;
}

int beam_attn_kv4_fwd(void *out, int64_t out_row_stride, float *lse_out, const void *q,
                      int64_t q_row_stride, const void *k_cache, const void *v_cache,
                      const void *k_scales, const void *v_scales, int64_t num_slots, int32_t group,
                      const int64_t *slot_table, int64_t table_stride, int64_t table_width,
                      const int32_t *seq_len, int32_t B, int32_t q_len, int32_t n_q_heads,
                      int32_t n_kv_heads, int32_t head_dim, float sm_scale, int64_t window,
                      int64_t n_sink, void *workspace, int64_t workspace_bytes,
                      cudaStream_t stream)
{
    if (head_dim != 128 || !good_group(group))
        return BEAM_ERR_UNSUPPORTED;
    const int st =
        check_attn_sizes(B, q_len, n_q_heads, n_kv_heads, table_width, window, n_sink);
    if (st != BEAM_OK)
        return st;
    if (num_slots < 0 || num_slots >= kMost || !std::isfinite(sm_scale))
        return BEAM_ERR_INVALID_ARG;
    if (B == 0)
        return BEAM_OK;
    const int64_t row = (int64_t)n_q_heads * head_dim;
    if (!out || !q || !seq_len || !workspace ||
        (num_slots > 0 && (!k_cache || !v_cache || !k_scales || !v_scales)) ||
        (table_width > 0 && !slot_table) || out_row_stride < row || q_row_stride < row ||
        (B > 1 && table_stride < table_width))
        return BEAM_ERR_INVALID_ARG;
    const uintptr_t sa = (uintptr_t)(128 / group * 4);
    if (!aligned(out, 16) || !aligned(q, 16) || out_row_stride % 8 != 0 || q_row_stride % 8 != 0 ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scales, sa) ||
        !aligned(v_scales, sa) || !aligned(slot_table, 8) || !aligned(seq_len, 4) ||
        !aligned(lse_out, 4) || !aligned(workspace, 16))
        return BEAM_ERR_MISALIGNED;
    const beam::Kv4AttnPlan p =
        beam::kv4_attn_plan(B, q_len, n_q_heads, n_kv_heads, table_width, window, n_sink, group);
    if (workspace_bytes < beam_attn_kv4_workspace(B, q_len, n_q_heads, n_kv_heads, table_width, window,
                                                  n_sink))
        return BEAM_ERR_INVALID_ARG;
    beam::Kv4AttnArgs a{};
    a.out = out;
    a.out_stride = out_row_stride;
    a.lse = lse_out;
    a.q = q;
    a.q_stride = q_row_stride;
    a.cache[0] = (const uint8_t *)k_cache;
    a.cache[1] = (const uint8_t *)v_cache;
    a.scales[0] = k_scales;
    a.scales[1] = v_scales;
    a.num_slots = num_slots;
    a.group = group;
    a.table = slot_table;
    a.table_stride = table_stride;
    a.width = table_width;
    a.len = seq_len;
    a.B = B;
    a.q_len = q_len;
    a.n_q = n_q_heads;
    a.n_kv = n_kv_heads;
    a.sm_scale = sm_scale;
    // a longer window than any list is none, and no list is longer than the table
    a.window = window > table_width ? 0 : window;
    a.n_sink = n_sink > table_width ? table_width : n_sink;
    a.workspace = (char *)workspace;
    return cuda_status(beam::launch_kv4_attn(a, p, stream));
}

int64_t beam_moe_layer_workspace(int64_t T, int32_t H, int32_t F, int32_t n_local)
{
    const int st = check_moe_sizes(T, H, F, n_local);
    if (st != BEAM_OK || T == 0)
        return st;
    return beam::moe_plan(T, H, F).bytes;
}

int beam_moe_layer_fwd(void *out, int64_t out_row_stride, int32_t *topk_ids_out, float *topk_w_out,
                       const void *x, int64_t x_row_stride, const float *router_w,
                       const float *router_bias, const void *w_gate_up, const void *w_down,
                       int32_t first_expert, int32_t n_local, float routed_scaling, int64_t T,
                       int32_t H, int32_t F, void *workspace, int64_t workspace_bytes,
                       cudaStream_t stream)
{
    const int st = check_moe_sizes(T, H, F, n_local);
    if (st != BEAM_OK)
        return st;
    if (first_expert < 0 || first_expert > kExperts - n_local || !std::isfinite(routed_scaling))
        return BEAM_ERR_INVALID_ARG;
    if (T == 0)
        return BEAM_OK;
    if (!out || !x || !router_w || !router_bias || !w_gate_up || !w_down || !workspace ||
        (T > 1 && (out_row_stride < H || x_row_stride < H)))
        return BEAM_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(x, 16) || out_row_stride % 8 != 0 || x_row_stride % 8 != 0 ||
        !aligned(router_w, 16) || !aligned(router_bias, 16) || !aligned(w_gate_up, 16) ||
        !aligned(w_down, 16) || !aligned(topk_ids_out, 4) || !aligned(topk_w_out, 4) ||
        !aligned(workspace, 16))
        return BEAM_ERR_MISALIGNED;
    const beam::MoePlan p = beam::moe_plan(T, H, F);
    if (workspace_bytes < p.bytes)
        return BEAM_ERR_INVALID_ARG;
    beam::MoeArgs a{};
    a.out = out;
    a.out_stride = out_row_stride;
    a.ids = topk_ids_out;
    a.weights = topk_w_out;
    a.x = x;
    a.x_stride = x_row_stride;
    a.router_w = router_w;
    a.router_bias = router_bias;
    a.w13 = w_gate_up;
    a.w2 = w_down;
    a.first = first_expert;
    a.local = n_local;
    a.scaling = routed_scaling;
    a.T = (int32_t)T;
    a.H = H;
    a.F = F;
    a.workspace = (char *)workspace;
    return cuda_status(beam::launch_moe_layer(a, p, stream));
}

int beam_draft_verify_fwd(int64_t *tokens_out, int32_t *n_accepted_out, const int64_t *draft_tokens,
                          const int32_t *draft_len, const void *target_probs,
                          int64_t target_seq_stride, int64_t target_pos_stride,
                          const void *draft_probs, int64_t draft_seq_stride,
                          int64_t draft_pos_stride, int32_t dtype, const float *u_accept,
                          const float *u_sample, int64_t B, int32_t k, int64_t V,
                          cudaStream_t stream)
{
    if (dtype != 0 && dtype != 1)
        return BEAM_ERR_UNSUPPORTED;
    if (B < 0 || B >= kMost || k < 0 || k > 1024 || V < 1 || V >= (1 << 20) ||
        target_seq_stride < 0 || target_pos_stride < 0 || draft_seq_stride < 0 ||
        draft_pos_stride < 0)
        return BEAM_ERR_INVALID_ARG;
    if (B == 0)
        return BEAM_OK;
    if (!tokens_out || !n_accepted_out || !target_probs || !u_sample ||
        (k > 0 && (!draft_tokens || !u_accept)))
        return BEAM_ERR_INVALID_ARG;
    const uintptr_t ea = dtype == 0 ? 4 : 2;
    if (!aligned(tokens_out, 8) || !aligned(n_accepted_out, 4) || !aligned(draft_tokens, 8) ||
        !aligned(draft_len, 4) || !aligned(target_probs, ea) || !aligned(draft_probs, ea) ||
        !aligned(u_accept, 4) || !aligned(u_sample, 4))
        return BEAM_ERR_MISALIGNED;
    beam::VerifyArgs a{};
    a.tokens_out = tokens_out;
    a.accepted = n_accepted_out;
    a.tokens = draft_tokens;
    a.len = draft_len;
    a.target = target_probs;
    a.draft = draft_probs;
    a.target_seq = target_seq_stride;
    a.target_pos = target_pos_stride;
    a.draft_seq = draft_seq_stride;
    a.draft_pos = draft_pos_stride;
    a.bf16 = dtype == 1;
    a.u_accept = u_accept;
    a.u_sample = u_sample;
    a.B = B;
    a.k = k;
    a.V = V;
    return cuda_status(beam::launch_draft_verify(a, stream));
}

}  // extern "C"
