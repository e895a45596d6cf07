// decode_kernels.h -- launch interface between the decode operators' C ABI (decode_api.cu) and their
// kernels.  Arguments arrive validated; the launchers only pick a configuration and launch.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "beam_kernels.h"

namespace beam {

// SMs that the work is divided for.  A constant of the GB300, not a query: the workspace size must
// be known without a device, and a plan must not depend on where it is made.
constexpr int kPlanSms = 152;

struct AttnArgs {
    void *out;
    int64_t out_stride;  // elements
    float *lse;          // [T, n_q] or nullptr
    const float *weight_in;
    float *weight_out;   // [B, width] or nullptr
    int64_t weight_stride;
    const void *q;
    int64_t q_stride;
    const void *k_cache;
    const void *v_cache;
    int64_t num_slots;
    bool fp8;
    float k_scale, v_scale;  // 1 for BF16
    const int64_t *prefix;
    int64_t n_prefix;
    const int64_t *table;
    int64_t table_stride;
    int64_t width;
    const int32_t *len;
    int32_t B, q_len, n_q, n_kv;
    float sm_scale;
    int64_t window;  // 0: none
    char *workspace;
};

// How one call is divided; a function of its sizes alone (attn_plan).  Rows are counted per KV head:
// R = q_len * (n_q / n_kv) of each sequence, sequence by sequence.  A unit is a tile of rows with the
// list of keys that they see: first the prefix's units, then the suffixes' (by sequence, KV head and
// row tile).  The units' key tiles, one after the other, are shared out evenly among `ctas` blocks.
struct AttnPlan {
    int32_t group, R;
    uint32_t group_magic;
    int32_t tile_keys;    // keys of a tile of the rows kernel
    int64_t rows;         // B * R
    int32_t nt;           // 8-row tiles of a unit's rows: 1, 2 or 3
    int64_t in_line;      // prefix keys that stand in front of each sequence's own (all or none)
    int32_t s_rtiles;     // row tiles of a sequence
    int64_t p_rtiles;     // row tiles of the prefix's units (0: no prefix)
    int64_t p_first;      // first prefix key that any row can see
    int64_t p_tiles;      // key tiles of a prefix unit
    int64_t units;        // all units
    int32_t ctas;
    bool whole;           // shares are of whole units: the rows kernel writes every result itself
    // the tensor-core kernel (tc_parts 0: not used): tiles of rows, blocks along the keys, steps of a
    // block (128 keys; 256 with tc_split), and parts that it leaves of each row
    int32_t tc_rtiles, tc_blocks, tc_steps, tc_parts;
    bool tc_split;
    int64_t score_width;  // padded width of the score rows (key weights only)
    // workspace, in bytes from its start
    int64_t cum_off, o_off, ml_off, lse_off, tc_o_off, tc_ml_off, score_off, bytes;
};

AttnPlan attn_plan(int32_t B, int32_t q_len, int32_t n_q, int32_t n_kv, int64_t n_prefix,
                   int64_t width, int64_t window, bool weights, bool fp8, bool tc);
cudaError_t launch_attn_prefix(const AttnArgs &a, const AttnPlan &p, cudaStream_t stream);
struct CacheMaps;
cudaError_t launch_attn_tc(const AttnArgs &a, const AttnPlan &p, const CacheMaps &maps,
                           cudaStream_t stream);
cudaError_t read_attn_tc_fault_word(unsigned int *value, bool clear);
// The decode operators' fault word of the current device (as read_fault_word).
cudaError_t read_decode_fault_word(unsigned int *value, bool clear);

struct EvictArgs {
    int64_t *table_out;
    int32_t *len_out;
    float *weight_out;
    int64_t *freed_out;
    int64_t freed_width;
    const int64_t *table_in;
    const int32_t *len_in;
    const float *weight_in;
    int64_t rows, width, budget, recent;
};

cudaError_t launch_kv_evict(const EvictArgs &a, cudaStream_t stream);

struct W4Args {
    void *y;
    int64_t y_stride;
    const void *x;
    int64_t x_stride;
    const void *w;
    const void *scales;
    const uint8_t *zeros;  // or nullptr
    int64_t T, N, K;
    int32_t group;
};

cudaError_t launch_w4_matvec(const W4Args &a, cudaStream_t stream);

// The kernel may use all of the shared memory: set once per device.
template <auto Kernel>
cudaError_t allow_smem(int bytes)
{
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done[dev]))
        return e;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64)
        done[dev] = true;
    return e;
}

}  // namespace beam
