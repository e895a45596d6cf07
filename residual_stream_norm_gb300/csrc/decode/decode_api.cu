// decode_api.cu -- C ABI of the decode operators: argument checks and launch.  Every check runs before
// any CUDA call, so a rejected call launches nothing, touches no output and needs no GPU.

#include <cmath>
#include <cstdint>

#include "../../../include/beam_decode.h"
#include "decode_kernels.h"

namespace {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? BEAM_OK : BEAM_ERR_CUDA; }

constexpr int64_t kMost = (int64_t)1 << 31;
constexpr int32_t kMaxHeads = 1024;

int check_attn_sizes(int32_t B, int32_t q_len, int32_t n_q, int32_t n_kv, int64_t n_prefix,
                     int64_t width, int64_t window)
{
    if (B < 0 || q_len < 1 || n_kv < 1 || n_q < n_kv || n_q > kMaxHeads || n_q % n_kv != 0 ||
        n_prefix < 0 || n_prefix >= kMost || width < 0 || width >= kMost || window < 0)
        return BEAM_ERR_INVALID_ARG;
    if ((int64_t)B * q_len * n_q >= kMost)
        return BEAM_ERR_INVALID_ARG;
    return BEAM_OK;
}

bool bad_scale(float s) { return !(s > 0.0f) || !std::isfinite(s); }

}  // namespace

extern "C" {

int64_t beam_attn_prefix_workspace(int32_t B, int32_t q_len, int32_t n_q_heads, int32_t n_kv_heads,
                                   int64_t n_prefix, int64_t table_width, int64_t window,
                                   int32_t key_weights)
{
    const int st =
        check_attn_sizes(B, q_len, n_q_heads, n_kv_heads, n_prefix, table_width, window);
    if (st != BEAM_OK || B == 0)
        return st;
    // the larger of what the call takes with and without the tensor-core kernel
    int64_t most = 0;
    for (int tc = 0; tc < 2; ++tc) {
        const int64_t bytes = beam::attn_plan(B, q_len, n_q_heads, n_kv_heads, n_prefix,
                                              table_width, window, key_weights != 0, false, tc != 0)
                                  .bytes;
        most = bytes > most ? bytes : most;
    }
    return most;
}

int beam_attn_prefix_fwd(void *out, int64_t out_row_stride, float *lse_out,
                         const float *key_weight_in, float *key_weight_out, int64_t weight_stride,
                         const void *q, int64_t q_row_stride, const void *k_cache,
                         const void *v_cache, int64_t num_slots, int32_t cache_dtype,
                         float k_scale, float v_scale, const int64_t *prefix_slots,
                         int64_t n_prefix, const int64_t *slot_table, int64_t table_stride,
                         int64_t table_width, const int32_t *suffix_len, int32_t B, int32_t q_len,
                         int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, float sm_scale,
                         int64_t window, void *workspace, int64_t workspace_bytes,
                         cudaStream_t stream)
{
    if (head_dim != 128 || (cache_dtype != 0 && cache_dtype != 1))
        return BEAM_ERR_UNSUPPORTED;
    const int st =
        check_attn_sizes(B, q_len, n_q_heads, n_kv_heads, n_prefix, table_width, window);
    if (st != BEAM_OK)
        return st;
    if (num_slots < 0 || num_slots >= kMost || !std::isfinite(sm_scale) ||
        (cache_dtype == 1 && (bad_scale(k_scale) || bad_scale(v_scale))))
        return BEAM_ERR_INVALID_ARG;
    if (B == 0)
        return BEAM_OK;
    const int64_t row = (int64_t)n_q_heads * head_dim;
    if (!out || !q || !suffix_len || (num_slots > 0 && (!k_cache || !v_cache)) ||
        (n_prefix > 0 && !prefix_slots) || (table_width > 0 && !slot_table) || !workspace ||
        out_row_stride < row || q_row_stride < row || (B > 1 && table_stride < table_width) ||
        (key_weight_in && !key_weight_out) ||
        (key_weight_out && B > 1 && weight_stride < table_width))
        return BEAM_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || out_row_stride % 8 != 0 || q_row_stride % 8 != 0 ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(prefix_slots, 8) ||
        !aligned(slot_table, 8) || !aligned(suffix_len, 4) || !aligned(lse_out, 4) ||
        !aligned(key_weight_in, 4) || !aligned(key_weight_out, 4) || !aligned(workspace, 16))
        return BEAM_ERR_MISALIGNED;
    if (workspace_bytes < beam_attn_prefix_workspace(B, q_len, n_q_heads, n_kv_heads, n_prefix,
                                                     table_width, window, key_weight_out != nullptr))
        return BEAM_ERR_INVALID_ARG;
    // a longer window than any list is none
    window = window > n_prefix + table_width ? 0 : window;
    // the tensor-core kernel takes the largest score before the scale and scales masked scores of
    // -inf: the scale must keep order and not underflow
    const float scale = sm_scale * (cache_dtype == 1 ? k_scale : 1.0f);
    const beam::AttnPlan p = beam::attn_plan(B, q_len, n_q_heads, n_kv_heads, n_prefix,
                                             table_width, window, key_weight_out != nullptr,
                                             cache_dtype == 1, scale > 1.0e-15f);
    beam::AttnArgs a{};
    a.out = out;
    a.out_stride = out_row_stride;
    a.lse = lse_out;
    a.weight_in = key_weight_in;
    a.weight_out = key_weight_out;
    a.weight_stride = weight_stride;
    a.q = q;
    a.q_stride = q_row_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.num_slots = num_slots;
    a.fp8 = cache_dtype == 1;
    a.k_scale = a.fp8 ? k_scale : 1.0f;
    a.v_scale = a.fp8 ? v_scale : 1.0f;
    a.prefix = prefix_slots;
    a.n_prefix = n_prefix;
    a.table = slot_table;
    a.table_stride = table_stride;
    a.width = table_width;
    a.len = suffix_len;
    a.B = B;
    a.q_len = q_len;
    a.n_q = n_q_heads;
    a.n_kv = n_kv_heads;
    a.sm_scale = sm_scale;
    a.window = window;
    a.workspace = (char *)workspace;
    return cuda_status(beam::launch_attn_prefix(a, p, stream));
}

int beam_kv_evict_fwd(int64_t *table_out, int32_t *len_out, float *weight_out, int64_t *freed_out,
                      int64_t freed_width, const int64_t *table_in, const int32_t *len_in,
                      const float *weight_in, int64_t rows, int64_t width, int64_t budget,
                      int64_t recent, cudaStream_t stream)
{
    if (rows < 0 || rows >= kMost || width < 0 || width >= kMost / 2 || budget < 0 || recent < 0 ||
        recent > budget || freed_width < 0 || freed_width < width - budget)
        return BEAM_ERR_INVALID_ARG;
    if (rows == 0)
        return BEAM_OK;
    if (!len_out || !len_in || (freed_width > 0 && !freed_out) ||
        (width > 0 && (!table_out || !table_in || !weight_out || !weight_in)))
        return BEAM_ERR_INVALID_ARG;
    if (!aligned(table_out, 8) || !aligned(table_in, 8) || !aligned(freed_out, 8) ||
        !aligned(weight_out, 4) || !aligned(weight_in, 4) || !aligned(len_out, 4) ||
        !aligned(len_in, 4))
        return BEAM_ERR_MISALIGNED;
    beam::EvictArgs a{};
    a.table_out = table_out;
    a.len_out = len_out;
    a.weight_out = weight_out;
    a.freed_out = freed_out;
    a.freed_width = freed_width;
    a.table_in = table_in;
    a.len_in = len_in;
    a.weight_in = weight_in;
    a.rows = rows;
    a.width = width;
    a.budget = budget;
    a.recent = recent;
    return cuda_status(beam::launch_kv_evict(a, stream));
}

int beam_w4_matvec_fwd(void *y, int64_t y_row_stride, const void *x, int64_t x_row_stride,
                       const void *w, const void *scales, const void *zeros, int64_t T, int64_t N,
                       int64_t K, int32_t group, cudaStream_t stream)
{
    if (group != 32 && group != 64 && group != 128)
        return BEAM_ERR_UNSUPPORTED;
    if (T < 0 || T >= kMost || N < 1 || N >= kMost || K < group || K >= kMost || K % group != 0)
        return BEAM_ERR_INVALID_ARG;
    if (T == 0)
        return BEAM_OK;
    if (!y || !x || !w || !scales || (T > 1 && (y_row_stride < N || x_row_stride < K)))
        return BEAM_ERR_INVALID_ARG;
    if (!aligned(y, 2) || !aligned(x, 16) || x_row_stride % 8 != 0 || !aligned(w, 16) ||
        !aligned(scales, 2))
        return BEAM_ERR_MISALIGNED;
    beam::W4Args a{};
    a.y = y;
    a.y_stride = y_row_stride;
    a.x = x;
    a.x_stride = x_row_stride;
    a.w = w;
    a.scales = scales;
    a.zeros = (const uint8_t *)zeros;
    a.T = T;
    a.N = N;
    a.K = K;
    a.group = group;
    return cuda_status(beam::launch_w4_matvec(a, stream));
}

}  // extern "C"
