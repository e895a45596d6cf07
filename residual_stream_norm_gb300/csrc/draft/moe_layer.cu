// moe_layer.cu -- a whole mixture-of-experts layer for a few tokens (sm_103a).
//
// With up to 256 tokens and 8 of 256 experts each, an expert has a handful of tokens: the layer is bound by
// reading the chosen experts' weights, each once.  Four kernels:
//  1. router: z = x router_w^T, one block an expert, in FP32 pairs;
//  2. the grouped top-k of beam_grouped_topk_fwd;
//  3. up: g, u and a = silu(g) u for each (token, expert) pair;
//  4. down: each block owns some of the H output columns and adds up all experts' shares of them.
//
// Kernels 3 and 4 stream weights through a ring of stages in shared memory: one warp copies rows of weights,
// and the tokens' rows that they meet, by bulk copies; eight warps multiply, each its own columns of the
// stage, with m16n8k16 instructions whose left operand is 16 rows of weights (for up: 8 of the gate and the
// same 8 of the up projection, so that one thread holds g and u of the same place) and whose right one is up
// to 8 tokens.  Both operands are read 16 bytes a thread: the instruction's columns are the row's in another
// order, the same for both.  The warps' sums meet in shared memory, in order.  An expert with more than 8 tokens is
// taken in several passes, the later ones out of the L2 cache.

#include "beam_device.cuh"
#include "beam_tma.cuh"
#include "decode/decode_mma.cuh"
#include "draft_kernels.h"

namespace beam {
namespace {

constexpr int kSms = 152;
constexpr int kExperts = 256;
constexpr int kTopK = 8;
constexpr int kMaxTokens = 256;
constexpr int kMaxPasses = kExperts + kMaxTokens;  // sum over experts of ceil(pairs / 8)
constexpr int kPassTokens = 8;
constexpr int kWarps = 8;                           // that multiply
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;           // and one that copies
constexpr int kMaxStages = 12;
constexpr int kMaxStageBytes = 30 * 1024;
constexpr int kSmem = 227 * 1024;

__device__ unsigned int g_moe_fault_word = 0u;

// ---------------------------------------------------------------------------------------------
// router
// ---------------------------------------------------------------------------------------------

constexpr int kRouterThreads = 128;
constexpr int kRouterTokens = 4;  // at a time

__global__ void __launch_bounds__(kRouterThreads)
    moe_router_kernel(float *logits, const uint16_t *x, int64_t x_stride, const float *router_w,
                      int T, int H)
{
    __shared__ Sum2 s_part[kRouterThreads / 32][kRouterTokens];
    const int e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float *w = router_w + (int64_t)e * H;
    pdl_launch_dependents();
    // a model parameter: on its way while the kernel before still runs
    for (int i = threadIdx.x * 32; i < H; i += kRouterThreads * 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(w + i));
    pdl_wait();
    for (int t0 = 0; t0 < T; t0 += kRouterTokens) {
        Sum2 acc[kRouterTokens];
#pragma unroll
        for (int i = 0; i < kRouterTokens; ++i)
            acc[i] = Sum2{0.0f, 0.0f};
        for (int k = threadIdx.x * 4; k < H; k += kRouterThreads * 4) {
            const float4 wv = *reinterpret_cast<const float4 *>(w + k);
            const float ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
            for (int i = 0; i < kRouterTokens; ++i) {
                if (t0 + i >= T)
                    continue;
                const uint2 xv = *reinterpret_cast<const uint2 *>(x + (t0 + i) * x_stride + k);
                const float xs[4] = {bf_lo(xv.x), bf_hi(xv.x), bf_lo(xv.y), bf_hi(xv.y)};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = __fmul_rn(xs[j], ws[j]);
                    const float low = __fmaf_rn(xs[j], ws[j], -p);  // exact
                    float s, err;
                    two_sum(acc[i].hi, p, s, err);
                    acc[i] = Sum2{s, __fadd_rn(acc[i].lo, __fadd_rn(err, low))};
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRouterTokens; ++i) {
            const Sum2 v = warp_sum(acc[i]);
            if (lane == 0)
                s_part[warp][i] = v;
        }
        __syncthreads();
        if (threadIdx.x < kRouterTokens && t0 + (int)threadIdx.x < T) {
            Sum2 v = s_part[0][threadIdx.x];
            for (int i = 1; i < kRouterThreads / 32; ++i)
                v = sum_merge(v, s_part[i][threadIdx.x]);
            logits[(int64_t)(t0 + threadIdx.x) * kExperts + e] = sum_value(v);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------------------------
// passes: an expert of this rank with up to 8 of its pairs
// ---------------------------------------------------------------------------------------------

struct Passes {
    int count;
    int16_t expert[kMaxPasses];
    int16_t tokens[kMaxPasses];
    int16_t pair[kMaxPasses][kPassTokens];  // token * 8 + k
};

struct Ring {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int fail;
};

// All threads; `scratch` holds an expert for each pair.  In the order of experts, then of tokens.
__device__ __forceinline__ void build_passes(Passes &ps, int16_t *scratch, const int32_t *ids, int T,
                                             int first, int local)
{
    __shared__ int s_sum[kExperts / 32];
    const int n = T * kTopK;
    for (int i = threadIdx.x; i < n; i += kThreads)
        scratch[i] = (int16_t)(ids[i] - first);
    __syncthreads();
    const int e = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int mine = 0;
    if (e < local)
        for (int i = 0; i < n; ++i)
            mine += scratch[i] == e;
    const int need = (mine + kPassTokens - 1) / kPassTokens;
    int at = need;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, at, off);
        if (lane >= off)
            at += o;
    }
    if (lane == 31 && warp < kExperts / 32)
        s_sum[warp] = at;
    __syncthreads();
    at -= need;
    for (int i = 0; i < warp && i < kExperts / 32; ++i)
        at += s_sum[i];
    if (e < local && mine > 0) {
        int put = 0;
        for (int i = 0; i < n; ++i)
            if (scratch[i] == e) {
                ps.pair[at + put / kPassTokens][put % kPassTokens] = (int16_t)i;
                ++put;
            }
        for (int i = 0; i < need; ++i) {
            ps.expert[at + i] = (int16_t)e;
            ps.tokens[at + i] =
                (int16_t)(mine - i * kPassTokens < kPassTokens ? mine - i * kPassTokens : kPassTokens);
        }
    }
    if (threadIdx.x == kExperts - 1)
        ps.count = at + need;
    __syncthreads();
}

// ---------------------------------------------------------------------------------------------
// the ring
// ---------------------------------------------------------------------------------------------

// How rows of K columns are cut: segments of `cols` columns (a multiple of 32), the last one shorter.
struct Cut {
    int32_t K, cols, segs;
    int32_t rows;    // rows of weights of a stage
    int32_t pitch;   // bytes from row to row of a stage: 64 modulo 128, so that eight threads that read
                     // 16 bytes each of two rows meet all banks
    int32_t stage_bytes, stages;
};

Cut make_cut(int K, int rows, int other_bytes)
{
    Cut c;
    c.K = K;
    c.rows = rows;
    int most = kMaxStageBytes / (2 * (rows + kPassTokens)) / 32 * 32;
    most = most > 512 ? 512 : most;
    c.segs = (K + most - 1) / most;
    c.cols = ((K + c.segs - 1) / c.segs + 31) / 32 * 32;
    c.segs = (K + c.cols - 1) / c.cols;
    c.pitch = (c.cols * 2 + 127) / 128 * 128 + 64;
    c.stage_bytes = (rows + kPassTokens) * c.pitch;
    c.stages = (kSmem - other_bytes) / c.stage_bytes;
    c.stages = c.stages > kMaxStages ? kMaxStages : c.stages;
    return c;
}

// Where copying or multiplying stands in the ring.
struct Turn {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages)
    {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// The copying warp: all segments of a job, whose row i of weights is at row(i) and goes to the stage's row
// place(i), and whose token j's row is at token(j).
template <typename Row, typename Place, typename Token>
__device__ __forceinline__ void copy_job(char *stages, Ring &ring, Turn &turn, const Cut &c, int rows,
                                         int tokens, Row row, Place place, Token token)
{
    const int lane = threadIdx.x & 31;
    for (int s = 0; s < c.segs; ++s) {
        if (!mbar_wait_or_fail(&ring.empty[turn.stage], turn.phase ^ 1u, &ring.fail))
            return;
        const int cols = c.K - s * c.cols < c.cols ? c.K - s * c.cols : c.cols;
        const uint32_t bytes = (uint32_t)cols * 2;
        uint64_t *bar = &ring.full[turn.stage];
        if (lane == 0)
            mbar_arrive_expect_tx(bar, bytes * (uint32_t)(rows + tokens));
        __syncwarp();
        char *dst = stages + turn.stage * c.stage_bytes;
        for (int i = lane; i < rows + tokens; i += 32) {
            const uint16_t *src = i < rows ? row(i) : token(i - rows);
            bulk_g2s(dst + (i < rows ? place(i) : c.rows + i - rows) * c.pitch, src + s * c.cols, bytes,
                     bar);
        }
        __syncwarp();
        turn.next(c.stages);
    }
}

// A multiplying warp: its columns of all segments of a job.  Row i of the left operand's 16 MT is the stage's
// row place(i); acc[m] are rows 16 m + g, 16 m + g + 8 of tokens 2t, 2t + 1.
template <int MT, typename Place>
__device__ __forceinline__ void multiply_job(float (&acc)[MT][4], const char *stages, Ring &ring, Turn &turn,
                                             const Cut &c, int tokens, Place place)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    uint32_t at[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            at[m][h] = place(m * 16 + h * 8 + g) * c.pitch + t * 16;
            acc[m][2 * h] = acc[m][2 * h + 1] = 0.0f;
        }
    const uint32_t xat = (c.rows + (g < tokens ? g : tokens - 1)) * c.pitch + t * 16;
    for (int s = 0; s < c.segs; ++s) {
        mbar_wait_or_fail(&ring.full[turn.stage], turn.phase, &ring.fail);
        const int cols = c.K - s * c.cols < c.cols ? c.K - s * c.cols : c.cols;
        const uint32_t base = smem_addr(stages + turn.stage * c.stage_bytes);
        for (int k = warp * 32; k < cols; k += kWarps * 32) {
            const bool in = k + t * 8 < cols;  // columns come by eights: all or none of a thread's
            const uint4 none = make_uint4(0, 0, 0, 0);
            const uint4 x = in ? lds128(base + xat + k * 2) : none;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint4 lo = in ? lds128(base + at[m][0] + k * 2) : none;
                const uint4 hi = in ? lds128(base + at[m][1] + k * 2) : none;
                const uint32_t f0[4] = {lo.x, hi.x, lo.y, hi.y}, f1[4] = {lo.z, hi.z, lo.w, hi.w};
                mma16816<false>(acc[m], f0, x.x, x.y);
                mma16816<false>(acc[m], f1, x.z, x.w);
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&ring.empty[turn.stage]);
        turn.next(c.stages);
    }
}

// This warp's sums to its place of the meeting area: [row][token].
template <int MT>
__device__ __forceinline__ void leave_sums(const float (&acc)[MT][4], float *mine)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        *reinterpret_cast<float2 *>(mine + (m * 16 + g) * 8 + 2 * t) = make_float2(acc[m][0], acc[m][1]);
        *reinterpret_cast<float2 *>(mine + (m * 16 + 8 + g) * 8 + 2 * t) =
            make_float2(acc[m][2], acc[m][3]);
    }
}

__device__ __forceinline__ void init_ring(Ring &ring, int stages)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&ring.full[i], 1);
            mbar_init(&ring.empty[i], kWarps);
        }
        ring.fail = 0;
        fence_mbar_init();
    }
}

// After a wait that ran out: the copies that are still under way end before the block's shared memory goes.
__device__ __forceinline__ void end_ring(Ring &ring, int stages, Turn turn)
{
    if (threadIdx.x < kConsumers || !*(volatile int *)&ring.fail)
        return;
    for (int i = 0; i < stages; ++i) {  // the stages before `turn`, latest first
        if (turn.stage == 0) {
            turn.stage = stages;
            turn.phase ^= 1u;
        }
        --turn.stage;
        mbar_wait(&ring.full[turn.stage], turn.phase, 20000000ull);
    }
    if ((threadIdx.x & 31) == 0)
        atomicOr(&g_moe_fault_word, kFaultCopyTimeout);
}

// ---------------------------------------------------------------------------------------------
// up: a = bf16(silu(g) u)
// ---------------------------------------------------------------------------------------------

constexpr int kUpPlaces = 8;  // places (of F) of a job

__host__ __device__ constexpr int meeting_bytes(int MT) { return 2 * kWarps * MT * 16 * 8 * 4; }

struct ShareArgs {
    const uint16_t *x;
    int64_t x_stride;
    const uint16_t *w13, *w2;
    uint16_t *act;             // [T * 8, F]
    uint16_t *out;
    int64_t out_stride;
    const int32_t *ids;
    const float *weights;
    int32_t first, local, T, H, F;
    float scaling;
    Cut cut;
    int32_t block_rows;        // down: most rows of a job
};

// A block's share of the places of all passes: jobs of up to 8 places of one pass.
struct UpJobs {
    int64_t at, end;
    int F;
    int pass, f, n;  // the job at hand
    int left, jobs;  // places and jobs left of this block's run in the pass
    __device__ __forceinline__ bool next()
    {
        if (jobs == 0) {
            if (at >= end)
                return false;
            pass = (int)(at / F);
            f = (int)(at - (int64_t)pass * F);
            n = 0;
            const int64_t stop = ((int64_t)pass + 1) * F < end ? ((int64_t)pass + 1) * F : end;
            left = (int)(stop - at);
            jobs = (left + kUpPlaces - 1) / kUpPlaces;
            at = stop;
        }
        f += n;
        n = (left + jobs - 1) / jobs;  // even: none much smaller than the others
        left -= n;
        --jobs;
        return true;
    }
};

__global__ void __launch_bounds__(kThreads, 1) moe_up_kernel(const ShareArgs a)
{
    extern __shared__ __align__(128) char smem[];
    __shared__ Passes ps;
    __shared__ Ring ring;
    char *stages = smem;
    float *meet = reinterpret_cast<float *>(smem + a.cut.stages * a.cut.stage_bytes);
    pdl_launch_dependents();
    init_ring(ring, a.cut.stages);
    pdl_wait();
    build_passes(ps, reinterpret_cast<int16_t *>(meet), a.ids, a.T, a.first, a.local);
    const int64_t places = (int64_t)ps.count * a.F;
    UpJobs jobs{};
    jobs.F = a.F;
    jobs.at = places * blockIdx.x / gridDim.x;
    jobs.end = places * (blockIdx.x + 1) / gridDim.x;
    Turn turn;
    if (threadIdx.x >= kConsumers) {
        while (jobs.next() && !*(volatile int *)&ring.fail) {
            const uint16_t *w = a.w13 + (int64_t)ps.expert[jobs.pass] * 2 * a.F * a.H;
            const int n = jobs.n, f = jobs.f, pass = jobs.pass;
            copy_job(
                stages, ring, turn, a.cut, 2 * n, ps.tokens[pass],
                [&](int i) { return w + (int64_t)(i < n ? f + i : a.F + f + i - n) * a.H; },
                [&](int i) { return i < n ? i : kUpPlaces + i - n; },
                [&](int j) { return a.x + (ps.pair[pass][j] / kTopK) * a.x_stride; });
        }
    } else {
        const int warp = threadIdx.x >> 5;
        int buf = 0;
        while (jobs.next()) {
            const int n = jobs.n, tokens = ps.tokens[jobs.pass];
            float acc[1][4];
            multiply_job<1>(acc, stages, ring, turn, a.cut, tokens, [&](int i) {
                const int r = i & 7;
                return (i & 8) + (r < n ? r : n - 1);
            });
            float *area = meet + buf * kWarps * 128;
            leave_sums<1>(acc, area + warp * 128);
            named_sync(1, kConsumers);
            // places run fastest: neighbouring threads write neighbouring values
            const int r = threadIdx.x & 7, j = threadIdx.x >> 3;
            if (r < n && j < tokens) {
                float g = 0.0f, u = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    g += area[w * 128 + r * 8 + j];
                    u += area[w * 128 + (8 + r) * 8 + j];
                }
                const float v = __fdiv_rn(g, 1.0f + expf(-g)) * u;
                a.act[(int64_t)ps.pair[jobs.pass][j] * a.F + jobs.f + r] =
                    (uint16_t)pack_bf16x2(v, 0.0f);
            }
            buf ^= 1;
        }
    }
    end_ring(ring, a.cut.stages, turn);
}

// ---------------------------------------------------------------------------------------------
// down: out = sum over the pairs of scaling * weight * w2 a
// ---------------------------------------------------------------------------------------------

template <int MT>
__global__ void __launch_bounds__(kThreads, 1) moe_down_kernel(const ShareArgs a)
{
    extern __shared__ __align__(128) char smem[];
    __shared__ Passes ps;
    __shared__ Ring ring;
    char *stages = smem;
    float *meet = reinterpret_cast<float *>(smem + a.cut.stages * a.cut.stage_bytes);
    float *sums = meet + meeting_bytes(MT) / 4;  // [token][row of the block's]
    pdl_launch_dependents();
    init_ring(ring, a.cut.stages);
    pdl_wait();
    build_passes(ps, reinterpret_cast<int16_t *>(meet), a.ids, a.T, a.first, a.local);
    const int r_end = (int)((int64_t)a.H * (blockIdx.x + 1) / gridDim.x);
    Turn turn;
    int r0 = (int)((int64_t)a.H * blockIdx.x / gridDim.x);
    if (threadIdx.x >= kConsumers) {
        for (; r0 < r_end && !*(volatile int *)&ring.fail; r0 += a.block_rows) {
            const int n = r_end - r0 < a.block_rows ? r_end - r0 : a.block_rows;
            for (int p = 0; p < ps.count && !*(volatile int *)&ring.fail; ++p) {
                const uint16_t *w = a.w2 + ((int64_t)ps.expert[p] * a.H + r0) * a.F;
                copy_job(
                    stages, ring, turn, a.cut, n, ps.tokens[p],
                    [&](int i) { return w + (int64_t)i * a.F; }, [](int i) { return i; },
                    [&](int j) { return a.act + (int64_t)ps.pair[p][j] * a.F; });
            }
        }
    } else {
        const int warp = threadIdx.x >> 5;
        int buf = 0;
        for (; r0 < r_end; r0 += a.block_rows) {
            const int n = r_end - r0 < a.block_rows ? r_end - r0 : a.block_rows;
            for (int i = threadIdx.x; i < a.T * a.block_rows; i += kConsumers)
                sums[i] = 0.0f;
            for (int p = 0; p < ps.count; ++p) {
                const int tokens = ps.tokens[p];
                float acc[MT][4];
                multiply_job<MT>(acc, stages, ring, turn, a.cut, tokens,
                                 [&](int i) { return i < n ? i : n - 1; });
                float *area = meet + buf * kWarps * MT * 128;
                leave_sums<MT>(acc, area + warp * MT * 128);
                named_sync(1, kConsumers);
                for (int i = threadIdx.x; i < n * 8; i += kConsumers) {
                    const int j = i & 7;
                    if (j < tokens) {
                        float v = 0.0f;
#pragma unroll
                        for (int w = 0; w < kWarps; ++w)
                            v += area[w * MT * 128 + i];
                        const int pair = ps.pair[p][j];
                        float *s = sums + (pair / kTopK) * a.block_rows + (i >> 3);
                        *s = __fmaf_rn(a.scaling * a.weights[pair], v, *s);
                    }
                }
                buf ^= 1;
            }
            named_sync(1, kConsumers);
            for (int i = threadIdx.x; i < a.T * n; i += kConsumers) {
                const int t = i / n, r = i - t * n;
                a.out[t * a.out_stride + r0 + r] =
                    (uint16_t)pack_bf16x2(sums[t * a.block_rows + r], 0.0f);
            }
            named_sync(1, kConsumers);
        }
    }
    end_ring(ring, a.cut.stages, turn);
}

template <auto Kernel>
cudaError_t launch_share(const ShareArgs &s, int grid, int smem, cudaStream_t stream)
{
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !done[dev])) {
        e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmem - (int)(sizeof(Passes) + sizeof(Ring) + 64));
        if (e == cudaSuccess && dev < 64)
            done[dev] = true;
    }
    return e == cudaSuccess
               ? launch_pdl(Kernel, dim3((unsigned)grid), dim3(kThreads), (size_t)smem, stream, s)
               : e;
}

}  // namespace

MoePlan moe_plan(int64_t T, int32_t H, int32_t F)
{
    MoePlan p;
    p.logits = 0;
    p.ids = T * kExperts * 4;
    p.weights = p.ids + T * kTopK * 4;
    p.act = p.weights + T * kTopK * 4;
    p.bytes = p.act + T * kTopK * F * 2;
    return p;
}

cudaError_t launch_moe_layer(const MoeArgs &a, const MoePlan &p, cudaStream_t stream)
{
    float *logits = (float *)(a.workspace + p.logits);
    ShareArgs s{};
    s.x = (const uint16_t *)a.x;
    s.x_stride = a.x_stride;
    s.w13 = (const uint16_t *)a.w13;
    s.w2 = (const uint16_t *)a.w2;
    s.act = (uint16_t *)(a.workspace + p.act);
    s.out = (uint16_t *)a.out;
    s.out_stride = a.out_stride;
    int32_t *ids = a.ids ? a.ids : (int32_t *)(a.workspace + p.ids);
    float *weights = a.weights ? a.weights : (float *)(a.workspace + p.weights);
    s.ids = ids;
    s.weights = weights;
    s.first = a.first;
    s.local = a.local;
    s.T = a.T;
    s.H = a.H;
    s.F = a.F;
    s.scaling = a.scaling;
    cudaError_t e = launch_pdl(moe_router_kernel, dim3(kExperts), dim3(kRouterThreads), 0, stream, logits,
                               s.x, s.x_stride, a.router_w, a.T, a.H);
    if (e == cudaSuccess) {
        RouteArgs r{};
        r.logits = logits;
        r.bias = a.router_bias;
        r.ids = ids;
        r.weights = weights;
        r.T = a.T;
        e = launch_grouped_topk(r, stream);
    }
    const int fixed = (int)(sizeof(Passes) + sizeof(Ring) + 64);
    if (e == cudaSuccess) {
        // the pairs' experts lie in the meeting area while the passes are made
        const int other = meeting_bytes(1);
        s.cut = make_cut(a.H, 2 * kUpPlaces, fixed + other);
        e = launch_share<moe_up_kernel>(s, kSms, s.cut.stages * s.cut.stage_bytes + other, stream);
    }
    if (e == cudaSuccess) {
        const int grid = a.H < kSms ? a.H : kSms;
        const int own = (a.H + grid - 1) / grid;
        s.block_rows = (own + (own + 47) / 48 - 1) / ((own + 47) / 48);
        const int MT = (s.block_rows + 15) / 16;
        const int other = meeting_bytes(MT) + a.T * s.block_rows * 4;
        s.cut = make_cut(a.F, s.block_rows, fixed + other);
        const int smem = s.cut.stages * s.cut.stage_bytes + other;
        e = MT == 1   ? launch_share<moe_down_kernel<1>>(s, grid, smem, stream)
            : MT == 2 ? launch_share<moe_down_kernel<2>>(s, grid, smem, stream)
                      : launch_share<moe_down_kernel<3>>(s, grid, smem, stream);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t read_draft_fault_word(unsigned int *value, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(value, g_moe_fault_word, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0u;
        e = cudaMemcpyToSymbol(g_moe_fault_word, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace beam
