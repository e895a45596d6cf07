// beam_routing.cuh -- grouped top-k routing of one token by one warp, for the kernels that route (the method
// and its exactness are described in routing.cu).
#pragma once

#include "beam_device.cuh"
#include "beam_exp.cuh"

namespace beam {
namespace {

constexpr int kExperts = 256;
constexpr int kGroups = 8;
constexpr int kTopkGroups = 4;
constexpr int kTopK = 8;
constexpr int kPerLane = kExperts / 32;  // 8

// Order-preserving key of an FP32 value: larger values, larger keys; NaN gets 1, below every
// number (the smallest numeric key, that of -inf, is 0x007fffff); 0 marks an ineligible expert.
__device__ __forceinline__ uint32_t rank_key(float v)
{
    const uint32_t u = __float_as_uint(v);
    if (v != v)
        return 1u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t key)
{
    if (key <= 1u)
        return __uint_as_float(0x7fc00000u);
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// (key, index) order: a above b
__device__ __forceinline__ bool above(uint32_t ka, int ia, uint32_t kb, int ib)
{
    return ka > kb || (ka == kb && ia < ib);
}

// Fast FP32 sigmoid for the ranking pass: 1 / (1 + __expf(-z)) with the hardware reciprocal.
// For |z| <= 17 it is within kFastSigmoidErr of the correctly rounded sigmoid.  That bound
// follows from __expf's documented error (2 + 1.173 |x| ulps) through ds = -s (1 - s) de/e, plus
// three FP32 roundings, with room to spare; a sweep of 22.9M arguments measured 1.8e-7.  For
// z > 17 both give exactly 1; for z < -17 both are below 4.2e-8 and closer than 1e-12.
constexpr float kFastSigmoidErr = 1.9073486328125e-06f;  // 2^-19

__device__ __forceinline__ float sigmoid_fast(float z)
{
    const float d = __fadd_rn(1.0f, __expf(-z));
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
    return r;
}

// The choice for one token by one warp, from the lane's 8 scores s (of experts e0..e0+7) and its biases.
// Lanes k < 8 receive slot k's expert id.  With `certify`, the scores are within kFastSigmoidErr of the exact
// ones, and the function returns true only if the ranking decisions provably match those the exact scores
// would give:
// - the 4th and 5th group scores are more than twice their error bound apart;
// - so are every two consecutive chosen experts and the 8th and 9th.
// Sorting is 1-Lipschitz in the max norm, so a gap larger than twice the bound on every score
// leaves the order, the chosen sets and the slot order unchanged.
__device__ __forceinline__ bool route_token(const float (&s)[kPerLane],
                                            const float (&bias)[kPerLane], int e0, int lane,
                                            int group, bool certify, int &my_id)
{
    uint32_t key[kPerLane];
    float cmax = 0.0f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const float c = __fadd_rn(s[i], bias[i]);  // choice score c = s + bias
        key[i] = rank_key(c);
        cmax = fmaxf(cmax, fabsf(c));
        finite = finite && isfinite(c);
    }
    // ---- group score: the FP32 sum of the group's two best choice scores -------------------
    uint32_t k1 = key[0], k2 = 0u;
#pragma unroll
    for (int i = 1; i < kPerLane; ++i) {
        k2 = max(k2, min(k1, key[i]));
        k1 = max(k1, key[i]);
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {  // merge the two-best lists of the quad
        const uint32_t ok1 = __shfl_xor_sync(0xffffffffu, k1, off);
        const uint32_t ok2 = __shfl_xor_sync(0xffffffffu, k2, off);
        k2 = max(max(k2, ok2), min(k1, ok1));
        k1 = max(k1, ok1);
    }
    const float gscore = __fadd_rn(key_value(k1), key_value(k2));
    // ---- the topk_groups best groups stay eligible --------------------------------------------
    const uint32_t gkey = rank_key(gscore);
    int rank = 0;
#pragma unroll
    for (int j = 0; j < kGroups; ++j)
        rank += above(__shfl_sync(0xffffffffu, gkey, 4 * j), j, gkey, group) ? 1 : 0;
    const bool eligible = rank < kTopkGroups;
    // ---- this lane's eligible experts, best first (odd-even transposition sort) -------------
    uint32_t hk[kPerLane];
    int hi[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        hk[i] = eligible ? key[i] : 0u;
        hi[i] = e0 + i;
    }
#pragma unroll
    for (int pass = 0; pass < kPerLane; ++pass)
#pragma unroll
        for (int i = pass & 1; i + 1 < kPerLane; i += 2)
            if (hk[i + 1] > hk[i]) {  // equal keys keep their order: the lower index first
                const uint32_t tk = hk[i];
                const int ti = hi[i];
                hk[i] = hk[i + 1], hi[i] = hi[i + 1];
                hk[i + 1] = tk, hi[i + 1] = ti;
            }
    // ---- the rounds: the warp's best head, then the owner moves on --------------------------
    float cprev = 0.0f, mingap = 3.0e38f;
    const int rounds = certify ? kTopK + 1 : kTopK;  // the ninth only to certify the cut
#pragma unroll 1
    for (int k = 0; k < rounds; ++k) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, hk[0]);
        const uint32_t idx =
            __reduce_min_sync(0xffffffffu, hk[0] == best ? (uint32_t)hi[0] : 0xffffffffu);
        const float ck = key_value(best);
        if (k > 0)
            mingap = fminf(mingap, __fsub_rn(cprev, ck));
        cprev = ck;
        if (lane == k)
            my_id = (int)idx;
        if (lane == (int)idx / kPerLane) {
#pragma unroll
            for (int i = 0; i + 1 < kPerLane; ++i)
                hk[i] = hk[i + 1], hi[i] = hi[i + 1];
            hk[kPerLane - 1] = 0u;
        }
    }
    if (!certify)
        return true;
    // ---- certificate ---------------------------------------------------------------------------
    // error bounds (generous FP32 arithmetic): a choice score within dc of the exact one, a group
    // score within dg; every |value| <= cm
    const float cm = __int_as_float(__reduce_max_sync(0xffffffffu, __float_as_int(cmax)));
    const bool all_finite = __all_sync(0xffffffffu, finite);
    const float dc = kFastSigmoidErr + cm * 2.384185791015625e-07f;  // + 2 ulp(cm), 2^-22
    const float dg = 2.0f * dc + cm * 4.76837158203125e-07f;          // + 2 ulp(2 cm), 2^-21
    // the 4th and 5th best group scores
    const float g4 =
        key_value(__reduce_max_sync(0xffffffffu, rank == kTopkGroups - 1 ? gkey : 0u));
    const float g5 = key_value(__reduce_max_sync(0xffffffffu, rank == kTopkGroups ? gkey : 0u));
    return all_finite && cm < 1.0e30f && __fsub_rn(g4, g5) > 2.0f * dg && mingap > 2.0f * dc;
}

// One copy of the exact sigmoid's code for all of a kernel's calls: where eight of them stood in line, fetching
// them took most of the time of the rare token that needs all scores exactly.
__device__ __noinline__ float sigmoid_exact(float z) { return sigmoid_rounded(z); }

// Expert ids of one token by one warp, from its 8 logits and biases a lane: lanes k < 8 return slot k's.  The
// ranking runs on fast sigmoids, unless it is not certified: then on exact ones of every score.
__device__ __forceinline__ int route_ids(const float (&z)[kPerLane], const float (&bias)[kPerLane], int lane)
{
    const int e0 = lane * kPerLane, group = lane >> 2;
    float s[kPerLane];
    int my_id = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
        s[i] = sigmoid_fast(z[i]);
    if (!route_token(s, bias, e0, lane, group, true, my_id)) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            s[i] = sigmoid_exact(z[i]);
        route_token(s, bias, e0, lane, group, false, my_id);
    }
    return my_id;
}

// The renormalised weight of slot `lane` < 8 from the chosen experts' logits, one a lane: exact sigmoids over
// their FP32 sum in slot order.
__device__ __forceinline__ float route_weight(float z)
{
    const float s = sigmoid_exact(z);
    float wsum = __shfl_sync(0xffffffffu, s, 0);
#pragma unroll
    for (int k = 1; k < kTopK; ++k)
        wsum = __fadd_rn(wsum, __shfl_sync(0xffffffffu, s, k));
    return __fdiv_rn(s, wsum);
}

}  // namespace
}  // namespace beam
