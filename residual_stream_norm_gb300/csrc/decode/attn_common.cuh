// attn_common.cuh -- what the attention kernels share.
#pragma once

#include "beam_device.cuh"
#include "decode_kernels.h"

namespace beam {

constexpr int kD = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int64_t seq_len(const AttnArgs &a, int64_t b)
{
    const int64_t n = a.len[b];
    return n < 0 ? 0 : (n > a.width ? a.width : n);
}

// The keys that any row of a sequence of n entries sees: [first, n).
__device__ __forceinline__ int64_t first_key(int64_t n, int q_len, int64_t window)
{
    const int64_t lo = n - q_len + 1 - window;
    return window > 0 && lo > 0 ? lo : 0;
}

// The same from a multiple of 16 on, where runs of slots are taken to start.
__device__ __forceinline__ int64_t first_tile_key(int64_t n, int q_len, int64_t window)
{
    return first_key(n, q_len, window) & ~(int64_t)15;
}

// Factor 2^k, k <= 60, that brings a row of largest magnitude bits `mx` (FP32) to [2^14, 2^15), and
// its inverse; 1 for zero, infinite and NaN rows.
__device__ __forceinline__ void f16_row_factor(uint32_t mx, float &f, float &inv)
{
    const int e = (int)(mx >> 23);
    int k = e == 255 || mx == 0u ? 0 : 141 - e;
    k = min(k, 60);
    f = __uint_as_float((uint32_t)(127 + k) << 23);
    inv = __uint_as_float((uint32_t)(127 - k) << 23);
}

// Row rr (of `rows`, per KV head): its token; the query's index and the head within the group.
__device__ __forceinline__ int64_t row_token(const AttnArgs &a, const AttnPlan &p, int64_t rr,
                                             int &i, int &hg)
{
    const uint32_t b = (uint32_t)rr / (uint32_t)p.R;  // B * q_len * n_q < 2^31
    const uint32_t r = (uint32_t)rr - b * p.R;
    i = (int)(r / (uint32_t)p.group);
    hg = (int)r - i * p.group;
    return (int64_t)b * a.q_len + i;
}

}  // namespace beam
