// draft_verify.cu -- verification of drafted tokens from given random numbers (sm_103a).
//
// A sequence's accepted tokens need two numbers a position; the token drawn behind them needs one row of the
// target's probabilities and, after a rejection, one of the draft's: V weights, their sum S, and the first
// place where the running sum passes u S.  Probabilities are whole numbers of 2^-44, so sums are 64-bit
// integers, exact in any order, and V < 2^20 of them stay below 2^64.
//
// One cluster of up to 8 blocks takes a sequence: each warp sums a stretch of the row, every block reads all
// stretches' sums out of its peers' shared memory, and the one whose stretch holds the border searches it (it
// is in the L2 cache by then).  The row is read from memory once.

#include <cooperative_groups.h>

#include "beam_device.cuh"
#include "beam_f32x2.cuh"
#include "draft_kernels.h"

namespace cg = cooperative_groups;

namespace beam {
namespace {

constexpr int kWarps = kVerifyWarps;
constexpr int kThreads = kWarps * 32;

template <bool BF16>
__device__ __forceinline__ float prob(const void *row, int v)
{
    if constexpr (BF16)
        return __uint_as_float((uint32_t)((const uint16_t *)row)[v] << 16);
    else
        return ((const float *)row)[v];
}

// rint(2^44 p) = 2^22 hi + lo of a pair of values p in [0, 1].  A conversion to 64 bits goes through the FP64 pipe, which
// is narrow here: two FP32 additions do it, which leave a whole number in the mantissa's bits, x = 2^22 p rounded to hi by
// an addition to 2^23, what is left of it, exact and at most a half, to lo by one to 1.5 2^23.  2^22 hi is even, so
// lo's ties are those of the whole.  Both parts come with the constants' bits on top.
struct Units {
    uint32_t hi, lo;
};
constexpr Units kNone = {0x4b000000u, 0x4b400000u};  // the parts of 0

struct Units2 {
    f2 hi, lo;
};

__device__ __forceinline__ Units2 units(f2 p)
{
    const f2 k22 = splat(4194304.0f), k23 = splat(8388608.0f);
    Units2 u;
    u.hi = fma2(p, k22, k23);
    const f2 rest = fma2(p, k22, fma2(u.hi, splat(-1.0f), k23));
    u.lo = fma2(rest, k22, splat(12582912.0f));
    return u;
}

// p limited to [0, 1]; NaN: 0.
__device__ __forceinline__ float limited(float p) { return __saturatef(p); }

__device__ __forceinline__ uint64_t whole(int32_t hi, int32_t lo)
{
    return (uint64_t)(((int64_t)hi << 22) + lo);
}

// The rows that a sequence's last token is drawn from.
struct Rows {
    const void *target;
    const void *draft;  // nullptr: none
    int32_t spike;      // the draft is all on this token (-1: not so)
};

// Adds the weights of two tokens, P or max(P - Q, 0), to 2^22 hi + lo (all modulo 2^32, without a draft with what kNone
// adds).  P grows with p: where q > p, P - Q is at most 0, and P less the units of min(p, q) is 0.
template <bool Draft>
__device__ __forceinline__ void add_weights(uint32_t &hi, uint32_t &lo, float p0, float p1, float q0, float q1)
{
    p0 = limited(p0);
    p1 = limited(p1);
    const Units2 a = units(make_f2(p0, p1));
    hi += __float_as_uint(lo_of(a.hi)) + __float_as_uint(hi_of(a.hi));
    lo += __float_as_uint(lo_of(a.lo)) + __float_as_uint(hi_of(a.lo));
    if (Draft) {
        const Units2 b = units(make_f2(fminf(limited(q0), p0), fminf(limited(q1), p1)));
        hi -= __float_as_uint(lo_of(b.hi)) + __float_as_uint(hi_of(b.hi));
        lo -= __float_as_uint(lo_of(b.lo)) + __float_as_uint(hi_of(b.lo));
    }
}

// What `pairs` calls of it added up.
template <bool Draft>
__device__ __forceinline__ uint64_t sum_of(uint32_t hi, uint32_t lo, int pairs)
{
    const uint32_t n = Draft ? 0u : 2u * (uint32_t)pairs;
    return whole((int32_t)(hi - n * kNone.hi), (int32_t)(lo - n * kNone.lo));
}

template <bool Draft>
__device__ __forceinline__ uint64_t weight_of(float p, float q)
{
    uint32_t hi = 0, lo = 0;
    add_weights<Draft>(hi, lo, p, 0.0f, q, 0.0f);
    return sum_of<Draft>(hi, lo, 1);
}

template <bool BF16>
__device__ __forceinline__ uint64_t weight_at(const Rows &r, int v)
{
    if (v == r.spike)
        return 0;
    return r.draft ? weight_of<true>(prob<BF16>(r.target, v), prob<BF16>(r.draft, v))
                   : weight_of<false>(prob<BF16>(r.target, v), 0.0f);
}

// 16 bytes of probabilities.
template <bool BF16>
__device__ __forceinline__ void unpack(float (&p)[BF16 ? 8 : 4], const uint4 &v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            p[2 * i] = bf_lo(word(v, i));
            p[2 * i + 1] = bf_hi(word(v, i));
        } else {
            p[i] = __uint_as_float(word(v, i));
        }
    }
}

// Sum of the weights of tokens [v0, v1), one lane's share, but for a spike.  Rows that stand the same way to 16 bytes
// (or one row) are read 16 bytes a lane between the first and the last such places, others token by token.
template <bool BF16, bool Draft>
__device__ __forceinline__ uint64_t sum_stretch(const Rows &r, int v0, int v1, int lane)
{
    constexpr int kSize = BF16 ? 2 : 4, kVec = 16 / kSize;
    uint64_t sum = 0;
    int v = v0;
    if (!Draft || ((uintptr_t)r.target - (uintptr_t)r.draft) % 16 == 0) {
        constexpr int kAhead = 4;
        const int lead = (int)((16 - ((uintptr_t)r.target + (uintptr_t)v0 * kSize) % 16) % 16) / kSize;
        const int first = min(v0 + lead, v1), vecs = (v1 - first) / kVec;
        // in front and behind: less than a vector each, a token a lane
        const int edge = lane < 16 ? v0 + lane : first + vecs * kVec + lane - 16;
        if (lane < 16 ? edge < first : edge < v1) {
            sum += weight_of<Draft>(prob<BF16>(r.target, edge), Draft ? prob<BF16>(r.draft, edge) : 0.0f);
        }
        const char *tp = (const char *)r.target + (int64_t)first * kSize;
        const char *dp = (const char *)r.draft + (int64_t)first * kSize;
#pragma unroll 1
        for (int i0 = 0; i0 < vecs; i0 += 32 * kAhead) {
            uint4 p[kAhead], q[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + k * 32 + lane;
                p[k] = q[k] = make_uint4(0, 0, 0, 0);
                if (i < vecs) {
                    p[k] = ld_cached(tp + i * 16);
                    if (Draft)
                        q[k] = ld_cached(dp + i * 16);
                }
            }
            uint32_t hi = 0, lo = 0;  // of at most 32 tokens: within 31 bits
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                float x[kVec], y[kVec];
                unpack<BF16>(x, p[k]);
                unpack<BF16>(y, q[k]);
#pragma unroll
                for (int j = 0; j < kVec; j += 2)
                    add_weights<Draft>(hi, lo, x[j], x[j + 1], y[j], y[j + 1]);
            }
            sum += sum_of<Draft>(hi, lo, kAhead * kVec / 2);
        }
        return sum;
    }
    constexpr int kAhead = 8;
#pragma unroll 1
    for (; v < v1; v += 32 * kAhead) {
        float p[kAhead], q[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = v + k * 32 + lane;
            p[k] = i < v1 ? prob<BF16>(r.target, i) : 0.0f;
            q[k] = Draft && i < v1 ? prob<BF16>(r.draft, i) : 0.0f;
        }
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int k = 0; k < kAhead; k += 2)
            add_weights<Draft>(hi, lo, p[k], p[k + 1], q[k], q[k + 1]);
        sum += sum_of<Draft>(hi, lo, kAhead / 2);
    }
    return sum;
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
__global__ void __launch_bounds__(kThreads, 4) draft_verify_kernel(const VerifyArgs a)
{
    __shared__ uint64_t s_w[2][kWarps];  // the stretches' sums, read by all blocks of the cluster
    __shared__ uint64_t s_scan[kWarps];
    __shared__ int s_found;
    const cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int64_t b = blockIdx.x / ranks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();

    // ---- accepted tokens: every warp by itself ----------------------------------------------------
    // (the draft's length and the last random number are loaded beside the rest, not in front of and behind it)
    const int k = a.k;
    const float u_last = a.u_sample[b];
    int n = a.len ? a.len[b] : k;
    const char *target = (const char *)a.target + b * a.target_seq * (BF16 ? 2 : 4);
    const char *draft = (const char *)a.draft + b * a.draft_seq * (BF16 ? 2 : 4);
    int acc = 0;
    while (true) {
        const int i = acc + lane;
        float p = 0.0f, q = 1.0f, u = 1.0f;  // not accepted
        if (i < k) {
            const int64_t x = a.tokens[b * k + i];
            if (x >= 0 && x < a.V) {
                p = prob<BF16>(target + i * a.target_pos * (BF16 ? 2 : 4), (int)x);
                if (a.draft)
                    q = prob<BF16>(draft + i * a.draft_pos * (BF16 ? 2 : 4), (int)x);
                u = a.u_accept[b * k + i];
            }
        }
        n = n < 0 ? 0 : (n > k ? k : n);
        // the FP32 factors' product is exact in 64 bits
        const bool ok = i < n && (double)u * (double)q < (double)p;
        const uint32_t no = ~__ballot_sync(0xffffffffu, ok);
        acc += no ? __ffs((int)no) - 1 : 32;
        if (no || acc >= n)
            break;
    }
    Rows r;
    r.target = target + acc * a.target_pos * (BF16 ? 2 : 4);
    r.draft = nullptr;
    r.spike = -1;
    if (acc < n) {
        if (a.draft)
            r.draft = draft + acc * a.draft_pos * (BF16 ? 2 : 4);
        else {
            const int64_t x = a.tokens[b * k + acc];
            r.spike = x >= 0 && x < a.V ? (int)x : -1;
        }
    }

    // ---- sums of this warp's stretch --------------------------------------------------------------
    const int V = (int)a.V, stretches = ranks * kWarps;
    const int each = ((V + stretches - 1) / stretches + 7) & ~7;
    const int v0 = min((rank * kWarps + warp) * each, V), v1 = min(v0 + each, V);
    uint64_t w[4], below = 0, total = 0;
    const int per = (int)((stretches + 31) / 32);
    for (int again = 0;; ++again) {
        uint64_t sum = warp_sum64(r.draft ? sum_stretch<BF16, true>(r, v0, v1, lane)
                                          : sum_stretch<BF16, false>(r, v0, v1, lane));
        if (lane == 0) {
            if (r.spike >= v0 && r.spike < v1) {
                sum -= weight_of<false>(prob<BF16>(r.target, r.spike), 0.0f);
            }
            s_w[again][warp] = sum;
        }
        cluster.sync();
        // every warp of every block: all stretches' sums, at most 4 a lane, in order
        uint64_t own = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = lane * per + i;
            w[i] = i < per && s < stretches
                       ? *cluster.map_shared_rank(&s_w[again][s % kWarps], s / kWarps)
                       : 0;
            own += w[i];
        }
        below = warp_below64(own, lane, total);
        if (total != 0 || again == 1 || (!r.draft && r.spike < 0))
            break;
        r.draft = nullptr;  // no weight left: the target's own probabilities
        r.spike = -1;
    }
    cluster.sync();  // all have read their peers' shared memory: the others need not stay for the search
    {
        const float u = fminf(fmaxf(u_last, 0.0f), 0.99999994f);  // NaN: 0
        // floor(floor(2^24 u) S / 2^24)
        const uint64_t border = __umul64hi((uint64_t)(u * 16777216.0f) << 40, total);
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
        // ---- the stretch's block searches it: a thread takes consecutive tokens -------------------
        int token = -1;
        const bool here = rank == (at >= 0 ? at / kWarps : 0);
        if (here && at >= 0) {
            const int f0 = at * each, f1 = min(f0 + each, V);
            const int few = (each + kThreads - 1) / kThreads;
            const int t0 = f0 + threadIdx.x * few, t1 = min(t0 + few, f1);
            uint64_t own = 0;
#pragma unroll 1
            for (int v = t0; v < t1; v += 8) {
                float p[8], q[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool on = v + i < t1 && v + i != r.spike;
                    p[i] = on ? prob<BF16>(r.target, v + i) : 0.0f;
                    q[i] = on && r.draft ? prob<BF16>(r.draft, v + i) : 0.0f;
                }
                uint32_t hi = 0, lo = 0;
#pragma unroll
                for (int i = 0; i < 8; i += 2)
                    add_weights<true>(hi, lo, p[i], p[i + 1], q[i], q[i + 1]);
                own += sum_of<true>(hi, lo, 4);
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
                for (int v = t0; v < t1; ++v) {
                    const uint64_t x = weight_at<BF16>(r, v);
                    if (border - run < x) {
                        s_found = v;
                        break;
                    }
                    run += x;
                }
            }
            __syncthreads();
            token = s_found;
        }
        if (here) {
            for (int i = threadIdx.x; i <= k; i += kThreads)
                a.tokens_out[b * (k + 1) + i] =
                    i < acc ? a.tokens[b * k + i] : (i == acc ? token : -1);
            if (threadIdx.x == 0)
                a.accepted[b] = acc;
        }
    }
}

template <bool BF16>
cudaError_t launch(const VerifyArgs &a, cudaStream_t stream)
{
    const int ranks = verify_ranks(a.B, a.V);
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
