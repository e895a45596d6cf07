// draft_verify.cu -- verification of drafted tokens from given random numbers (sm_103a).
//
// A sequence's accepted tokens need two numbers a position; the token drawn behind them needs one row of the
// target's probabilities and, after a rejection, one of the draft's: V weights, their sum S, and the first
// place where the running sum passes u S.  Probabilities are whole numbers of 2^-44, so sums are 64-bit
// integers, exact in any order, and V < 2^20 of them stay below 2^64.
//
// One cluster of up to 8 blocks takes a sequence: each warp sums a stretch of the row, the first block reads
// all stretches' sums out of its peers' shared memory, picks the stretch that holds the border, and its
// threads search it (it is in the L2 cache by then).  The row is read from memory once.

#include <cooperative_groups.h>

#include "beam_device.cuh"
#include "draft_kernels.h"

namespace cg = cooperative_groups;

namespace beam {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

template <bool BF16>
__device__ __forceinline__ float prob(const void *row, int64_t v)
{
    if constexpr (BF16)
        return __uint_as_float((uint32_t)((const uint16_t *)row)[v] << 16);
    else
        return ((const float *)row)[v];
}

// rint(2^44 p), p limited to [0, 1]; NaN: 0.  The scaling is exact.
__device__ __forceinline__ int64_t units(float p)
{
    return __float2ll_rn(__fmul_rn(fminf(fmaxf(p, 0.0f), 1.0f), 17592186044416.0f));
}

// The rows that a sequence's last token is drawn from.
struct Rows {
    const void *target;
    const void *draft;  // nullptr: none (or all on token `spike`)
    int64_t spike;      // -1: none
};

// Weight of token v; `plain` its target's probability.
template <bool BF16>
__device__ __forceinline__ void weight_of(float p, float q, bool has_q, bool spike, int64_t &w,
                                          int64_t &plain)
{
    plain = units(p);
    w = plain - (has_q ? units(q) : 0);
    w = w < 0 || spike ? 0 : w;
}

// Sums of the weights and of the target's probabilities of tokens [v0, v1), one lane's share.
template <bool BF16>
__device__ __forceinline__ void sum_stretch(const Rows &r, int64_t v0, int64_t v1, int lane,
                                            uint64_t &sw, uint64_t &sp)
{
    constexpr int kEach = 8;
    for (int64_t v = v0 + lane; v < v1; v += 32 * kEach) {
        float p[kEach], q[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const bool in = v + 32 * i < v1;
            p[i] = in ? prob<BF16>(r.target, v + 32 * i) : 0.0f;
            q[i] = in && r.draft ? prob<BF16>(r.draft, v + 32 * i) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            int64_t w, plain;
            weight_of<BF16>(p[i], q[i], r.draft != nullptr, v + 32 * i == r.spike, w, plain);
            sw += (uint64_t)w;
            sp += (uint64_t)plain;
        }
    }
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Sum over the lanes below this one, and the warp's whole sum.
__device__ __forceinline__ uint64_t warp_below64(uint64_t v, int lane, uint64_t &all)
{
    uint64_t s = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off)
            s += o;
    }
    all = __shfl_sync(0xffffffffu, s, 31);
    return s - v;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) draft_verify_kernel(const VerifyArgs a)
{
    __shared__ uint64_t s_w[kWarps], s_p[kWarps];  // the stretches' sums, read by the first block
    __shared__ uint64_t s_scan[kWarps];
    __shared__ int s_found;
    const cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int64_t b = blockIdx.x / ranks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();

    // ---- accepted tokens: every warp by itself ----------------------------------------------------
    const int k = a.k;
    int n = a.len ? a.len[b] : k;
    n = n < 0 ? 0 : (n > k ? k : n);
    const char *target = (const char *)a.target + b * a.target_seq * (BF16 ? 2 : 4);
    const char *draft = (const char *)a.draft + b * a.draft_seq * (BF16 ? 2 : 4);
    int acc = 0;
    while (acc < n) {
        const int i = acc + lane;
        bool ok = false;
        if (i < n) {
            const int64_t x = a.tokens[b * k + i];
            if (x >= 0 && x < a.V) {
                const float p = prob<BF16>(target + i * a.target_pos * (BF16 ? 2 : 4), x);
                const float q =
                    a.draft ? prob<BF16>(draft + i * a.draft_pos * (BF16 ? 2 : 4), x) : 1.0f;
                // the FP32 factors' product is exact in 64 bits
                ok = (double)a.u_accept[b * k + i] * (double)q < (double)p;
            }
        }
        const uint32_t no = ~__ballot_sync(0xffffffffu, ok);
        acc += no ? __ffs((int)no) - 1 : 32;
        if (no)
            break;
    }
    Rows r;
    r.target = target + acc * a.target_pos * (BF16 ? 2 : 4);
    r.draft = nullptr;
    r.spike = -1;
    if (acc < n) {
        if (a.draft)
            r.draft = draft + acc * a.draft_pos * (BF16 ? 2 : 4);
        else
            r.spike = a.tokens[b * k + acc];
    }

    // ---- sums of this warp's stretch --------------------------------------------------------------
    const int64_t stretches = (int64_t)ranks * kWarps;
    const int64_t each = (a.V + stretches - 1) / stretches;
    const int64_t mine = (int64_t)rank * kWarps + warp;
    const int64_t v0 = mine * each < a.V ? mine * each : a.V;
    const int64_t v1 = v0 + each < a.V ? v0 + each : a.V;
    uint64_t sw = 0, sp = 0;
    sum_stretch<BF16>(r, v0, v1, lane, sw, sp);
    sw = warp_sum64(sw);
    sp = warp_sum64(sp);
    if (lane == 0) {
        s_w[warp] = sw;
        s_p[warp] = sp;
    }
    cluster.sync();
    if (rank == 0) {
        // ---- every warp: all stretches' sums (at most 4 a lane, in order), the border, its stretch ----
        uint64_t w[4], p[4], lw = 0, lp = 0;
        const int per = (int)((stretches + 31) / 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t s = (int64_t)lane * per + i;
            w[i] = p[i] = 0;
            if (i < per && s < stretches) {
                w[i] = *cluster.map_shared_rank(&s_w[s % kWarps], (int)(s / kWarps));
                p[i] = *cluster.map_shared_rank(&s_p[s % kWarps], (int)(s / kWarps));
            }
            lw += w[i];
            lp += p[i];
        }
        uint64_t total;
        uint64_t below = warp_below64(lw, lane, total);
        const bool plain = total == 0;  // no weight left: the target's own probabilities
        if (plain) {
            below = warp_below64(lp, lane, total);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = p[i];
            r.draft = nullptr;
            r.spike = -1;
        }
        float u = a.u_sample[b];
        u = fminf(fmaxf(u, 0.0f), 0.99999994f);  // NaN: 0
        // u in units of 2^-64, in two steps of 32 bits: its 24 bits stand anywhere
        const double ud = (double)u * 4294967296.0;
        const uint64_t u_hi = (uint64_t)ud;
        const uint64_t u64 = (u_hi << 32) | (uint64_t)((ud - (double)u_hi) * 4294967296.0);
        const uint64_t border = __umul64hi(u64, total);
        int at = -1;
        uint64_t start = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (at < 0 && below <= border && border - below < w[i]) {
                at = lane * per + i;
                start = below;
            }
            below += w[i];
        }
        const uint32_t has = __ballot_sync(0xffffffffu, at >= 0);
        const int owner = has ? __ffs((int)has) - 1 : 0;
        at = __shfl_sync(0xffffffffu, at, owner);
        start = __shfl_sync(0xffffffffu, start, owner);
        // ---- the block searches the stretch: a thread takes consecutive tokens --------------------
        int64_t token = -1;
        if (at >= 0) {
            const int64_t f0 = at * each, f1 = f0 + each < a.V ? f0 + each : a.V;
            const int64_t few = (f1 - f0 + kThreads - 1) / kThreads;
            const int64_t t0 = f0 + threadIdx.x * few;
            uint64_t own = 0;
            for (int64_t v = t0; v < t0 + few && v < f1; ++v) {
                int64_t x, y;
                weight_of<BF16>(prob<BF16>(r.target, v), r.draft ? prob<BF16>(r.draft, v) : 0.0f,
                                r.draft != nullptr, v == r.spike, x, y);
                own += (uint64_t)x;
            }
            uint64_t all;
            uint64_t run = warp_below64(own, lane, all);
            if (lane == 0)
                s_scan[warp] = all;
            if (threadIdx.x == 0)
                s_found = -1;
            __syncthreads();
            run += start;
            for (int i = 0; i < warp; ++i)
                run += s_scan[i];
            if (run <= border && border - run < own) {
                for (int64_t v = t0; v < t0 + few && v < f1; ++v) {
                    int64_t x, y;
                    weight_of<BF16>(prob<BF16>(r.target, v),
                                    r.draft ? prob<BF16>(r.draft, v) : 0.0f, r.draft != nullptr,
                                    v == r.spike, x, y);
                    if (border - run < (uint64_t)x) {
                        s_found = (int)v;
                        break;
                    }
                    run += (uint64_t)x;
                }
            }
            __syncthreads();
            token = s_found;
        }
        for (int i = threadIdx.x; i <= k; i += kThreads)
            a.tokens_out[b * (k + 1) + i] = i < acc ? a.tokens[b * k + i] : (i == acc ? token : -1);
        if (threadIdx.x == 0)
            a.accepted[b] = acc;
    }
    cluster.sync();  // the first block has read its peers' shared memory
}

template <bool BF16>
cudaError_t launch(const VerifyArgs &a, cudaStream_t stream)
{
    // Blocks of a sequence: 8 while each warp's stretch has some 128 tokens.
    int ranks = kMaxCluster;
    while (ranks > 1 && a.V < (int64_t)ranks * kWarps * 128)
        ranks /= 2;
    while (ranks > 1 && a.B * ranks >= ((int64_t)1 << 31))
        ranks /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, draft_verify_kernel<BF16>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyArgs &a, cudaStream_t stream)
{
    return a.bf16 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace beam
