// routing.cu -- DeepSeek-V3-style grouped top-k routing (sm_103a).
//
// Pages cited (titles as printed):
//   [vLLM]  "Serving Reflection Beam auf vLLM ab Tag 0"
//   [SGL]   "SGLang 支撑编程模型 Beam 生产部署"
//
// Beam routes 256 experts the way DeepSeek-V3 does: sigmoid scores plus a correction bias pick
// the best 4 of 8 expert groups, then the top 8 experts, whose renormalised scores weight the
// combine ([vLLM] "MoE und Residual-Stream", bullets "MoE im DeepSeek-V3-Stil" and
// "FP32-Router"; [SGL] "稠密层与分组 MoE 路由").  The kernel produces exactly what the MoE
// combine takes: the expert ids per token, best first, and the renormalised FP32 weights
// (the routed scaling is applied by the combine).
//
// One warp per token.  Lane l holds experts 8l..8l+7, so the four lanes of a quad hold one group
// of 32.
// - The ranking decisions are those of the correctly rounded FP32 sigmoids (beam_exp.cuh), the
//   oracle's (see below for how most of them are made on cheaper values).
// - A group's score is the FP32 sum of its two best choice scores.  The quad finds them with two
//   shuffle steps on their keys.
// - Every lane ranks the eight group scores.
// - Then eight rounds pick the experts: each lane keeps its eligible experts sorted.  A round
//   takes the warp's best head with two `redux.sync` reductions (the largest key, then the
//   lowest index among the lanes holding it), and the owning lane moves to its next expert.
// The ranking first runs on fast sigmoids (hardware exp) with a proven error bound.  When every
// deciding gap exceeds twice that bound, the decisions are those of the exact scores, and only
// the eight chosen experts need correctly rounded sigmoids, for their weights.  Otherwise, for a
// few tokens in a thousand, all 256 are computed exactly and ranked again.
//
// Ranking order: keys map FP32 values to integers in the same order, so that larger values
// rank higher.  NaN ranks below every number, ineligible experts below NaN, and ties go to the
// lower index.

#include "beam_kernels.h"
#include "beam_routing.cuh"

namespace beam {
namespace {

constexpr int kRouteThreads = 256;      // up to 8 tokens per CTA pass

// At least 3 CTAs per SM: more warps to cover the ranking's dependent-instruction latency.  The kernel takes 63
// registers, so four fit: 37.7 us at T = 16384, 2.6 us for one token (51.6 and 4.4 with index pairs in the group
// scores and the exact sigmoid's code in several places, at 80 registers).
__global__ void __launch_bounds__(kRouteThreads, 3)
    grouped_topk_kernel(const RouteArgs a)
{
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int e0 = lane * kPerLane;
    pdl_launch_dependents();
    float bias[kPerLane];  // model parameter: read before waiting on the previous kernel
    {
        const float4 b0 = *reinterpret_cast<const float4 *>(a.bias + e0);
        const float4 b1 = *reinterpret_cast<const float4 *>(a.bias + e0 + 4);
        bias[0] = b0.x, bias[1] = b0.y, bias[2] = b0.z, bias[3] = b0.w;
        bias[4] = b1.x, bias[5] = b1.y, bias[6] = b1.z, bias[7] = b1.w;
    }
    pdl_wait();
    const int per = blockDim.x / 32;
    const int64_t warps = (int64_t)gridDim.x * per;
    for (int64_t t = (int64_t)blockIdx.x * per + warp; t < a.T; t += warps) {
        const float *zp = a.logits + t * kExperts + e0;
        const float4 z0 = ld_stream_f4(zp), z1 = ld_stream_f4(zp + 4);
        const float z[kPerLane] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
        const int my_id = route_ids(z, bias, lane);
        const float my_w = route_weight(lane < kTopK ? a.logits[t * kExperts + my_id] : 0.0f);
        if (lane < kTopK) {
            a.ids[t * kTopK + lane] = my_id;
            a.weights[t * kTopK + lane] = my_w;
        }
    }
}

}  // namespace

cudaError_t launch_grouped_topk(const RouteArgs &a, cudaStream_t stream)
{
    // few tokens are spread over the SMs, a warp for each of their schedulers first (1024 tokens 6.9 us, 13.0 with 8 warps
    // to a block)
    const int64_t even = (a.T + 4 * 152 - 1) / (4 * 152);
    const int per = even < 1 ? 1 : (even < kRouteThreads / 32 ? (int)even : kRouteThreads / 32);
    const int64_t ctas = (a.T + per - 1) / per;
    const unsigned grid = (unsigned)(ctas < (1 << 20) ? ctas : (1 << 20));
    const cudaError_t e =
        launch_pdl(grouped_topk_kernel, dim3(grid), dim3(32 * per), 0, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace beam
