// draft_kernels.h -- launch interface between the C ABI of the operators of a draft-checking decode step
// (draft_api.cu) and their kernels.  Arguments arrive validated; the launchers only pick a configuration
// and launch.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "beam_kernels.h"
#include "draft_plan.h"

namespace beam {

struct Kv4WriteArgs {
    uint8_t *cache[2];     // K, V: [num_slots, n_kv, 64]
    void *scales[2];       // [num_slots, n_kv, 128 / group, 2] bf16
    const void *src[2];    // [T, n_kv, 128] bf16
    int64_t src_stride[2];  // elements
    int64_t num_slots;
    const int64_t *slot;
    int64_t T;
    int32_t n_kv;
    int32_t group;
};

cudaError_t launch_kv4_write(const Kv4WriteArgs &a, cudaStream_t stream);

struct Kv4AttnArgs {
    void *out;
    int64_t out_stride;  // elements
    float *lse;          // [T, n_q] or nullptr
    const void *q;
    int64_t q_stride;
    const uint8_t *cache[2];
    const void *scales[2];
    int64_t num_slots;
    int32_t group;
    const int64_t *table;
    int64_t table_stride;
    int64_t width;
    const int32_t *len;
    int32_t B, q_len, n_q, n_kv;
    float sm_scale;
    int64_t window;  // 0: none
    int64_t n_sink;
    char *workspace;
};

cudaError_t launch_kv4_attn(const Kv4AttnArgs &a, const Kv4AttnPlan &p, cudaStream_t stream);

struct MoeArgs {
    void *out;
    int64_t out_stride;
    int32_t *ids;
    float *weights;
    const void *x;
    int64_t x_stride;
    const float *router_w;
    const float *router_bias;
    const void *w13;
    const void *w2;
    int32_t first, local;
    float scaling;
    int32_t T, H, F;
    char *workspace;
};

// Byte offsets in the workspace.
struct MoePlan {
    int64_t logits, ids, weights, passes, act, sums, bytes;
    int64_t sum_rows;
};

MoePlan moe_plan(int64_t T, int32_t H, int32_t F);
cudaError_t launch_moe_layer(const MoeArgs &a, const MoePlan &p, cudaStream_t stream);

struct VerifyArgs {
    int64_t *tokens_out;
    int32_t *accepted;
    const int64_t *tokens;
    const int32_t *len;  // or nullptr
    const void *target, *draft;  // draft may be nullptr
    int64_t target_seq, target_pos, draft_seq, draft_pos;  // elements
    bool bf16;
    const float *u_accept, *u_sample;
    int64_t B;
    int32_t k;
    int64_t V;
};

cudaError_t launch_draft_verify(const VerifyArgs &a, cudaStream_t stream);

}  // namespace beam
