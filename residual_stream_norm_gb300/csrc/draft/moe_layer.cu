// moe_layer.cu -- a whole mixture-of-experts layer for a few tokens (sm_103a).
//
// With up to 256 tokens and 8 of 256 experts each, an expert has a handful of tokens: the layer is bound by
// reading the chosen experts' weights, each once.  Kernels:
//  1. router: z = x router_w^T in FP32 pairs;
//  2. the grouped top-k of beam_grouped_topk_fwd: for up to 16 tokens in every block of the next kernel, two
//     tokens a warp at most, else as that kernel;
//  3. up: g, u and a = silu(g) u for each (token, expert) pair;
//  4. down: each block owns some of the H output columns and adds up all experts' shares of them.
//
// Kernels 3 and 4 give each of a block's eight warps a stream of its own: 16 rows of weights by 64 columns at a
// time, copied with cp.async some stages ahead into the warp's part of shared memory together with the tokens'
// rows that they meet (bulk copies of a row's kilobyte, one instruction each, ran at 1.9 TB/s: 1.17 ms for 64 tokens of a
// tensor-parallel eighth, 0.55 this way).  They are multiplied with m16n8k16 instructions whose left operand is
// the weights (for up: 8 rows of the gate and the same 8 of the up projection, so that one thread holds g and u of the
// same place) and whose right one is up to 8 tokens.  Both operands are read 16 bytes a thread: the
// instruction's columns are the row's in another order, the same for both.  Warps take parts of the columns of
// the same tile, or where rows are short tiles of their own; their sums meet in shared memory, in order.  An expert
// with more than 8 tokens is taken in several passes, the later ones out of the L2 cache.

#include "beam_device.cuh"
#include "beam_routing.cuh"
#include "decode/decode_mma.cuh"
#include "draft_kernels.h"

namespace beam {
namespace {

constexpr int kSms = 152;
constexpr int kMaxTokens = 256;
constexpr int kMaxPasses = kExperts + kMaxTokens;  // sum over experts of ceil(pairs / 8)
constexpr int kPassTokens = 8;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kFusedTokens = 16;   // tokens that the up kernel routes itself
constexpr int kCols = 64;          // columns of a stage: 128 bytes of a row
constexpr int kUpStages = 8;
constexpr int kDownStages = 6;
constexpr int kSumRows = 512;      // least rows of the down kernel's sums

// ---------------------------------------------------------------------------------------------
// router
// ---------------------------------------------------------------------------------------------

// A block takes two experts and up to 8 tokens; a thread the columns 4 i, i = its number modulo 256, of both.
// A sum starts at a power of two times 1.5 that is larger than twice all of its terms together: each
// addition rounds to a grid that the running sum never leaves, so that the part taken up, acc' - acc, is exact, and what is left of
// the product, one fused multiply-add, goes into a second sum: four instructions a product, where pairs by
// TwoSum take ten.
constexpr int kRouterExperts = 2;
constexpr int kRouterTokens = 8;
constexpr int kRouterVecs = 5;    // float4s of an expert's row a thread holds: 5,120 columns at a time
constexpr int kRouterSums = kRouterExperts * kRouterTokens;

__device__ __forceinline__ Sum2 merge_across(Sum2 keep, Sum2 give, int off)
{
    Sum2 o;
    o.hi = __shfl_xor_sync(0xffffffffu, give.hi, off);
    o.lo = __shfl_xor_sync(0xffffffffu, give.lo, off);
    return sum_merge(keep, o);
}

__global__ void __launch_bounds__(kThreads)
    moe_router_kernel(float *logits, const uint16_t *x, int64_t x_stride, const float *router_w,
                      int T, int H)
{
    __shared__ Sum2 s_part[kWarps][kRouterSums];
    const int e0 = blockIdx.x * kRouterExperts, t0 = blockIdx.y * kRouterTokens;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = T - t0 < kRouterTokens ? T - t0 : kRouterTokens;
    pdl_launch_dependents();
    Sum2 total[kRouterSums];  // [expert][token]
#pragma unroll
    for (int i = 0; i < kRouterSums; ++i)
        total[i] = Sum2{0.0f, 0.0f};
    for (int k0 = 0; k0 < H; k0 += kThreads * 4 * kRouterVecs) {
        float4 w[kRouterExperts][kRouterVecs];
        float mw[kRouterExperts];
#pragma unroll
        for (int e = 0; e < kRouterExperts; ++e) {
            mw[e] = 0.0f;
#pragma unroll
            for (int v = 0; v < kRouterVecs; ++v) {
                const int k = k0 + (v * kThreads + threadIdx.x) * 4;
                w[e][v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (k < H)  // a model parameter: read before waiting on the previous kernel
                    w[e][v] = *reinterpret_cast<const float4 *>(router_w + (int64_t)(e0 + e) * H + k);
            }
        }
        if (k0 == 0)
            pdl_wait();
#pragma unroll
        for (int e = 0; e < kRouterExperts; ++e)
#pragma unroll
            for (int v = 0; v < kRouterVecs; ++v)
                mw[e] = fmaxf(fmaxf(fmaxf(mw[e], fabsf(w[e][v].x)), fabsf(w[e][v].y)),
                              fmaxf(fabsf(w[e][v].z), fabsf(w[e][v].w)));
#pragma unroll
        for (int t = 0; t < kRouterTokens; ++t) {
            if (t >= n)
                continue;
            uint2 xv[kRouterVecs];
            float mx = 0.0f;
#pragma unroll
            for (int v = 0; v < kRouterVecs; ++v) {
                const int k = k0 + (v * kThreads + threadIdx.x) * 4;
                xv[v] = make_uint2(0u, 0u);
                if (k < H)
                    xv[v] = *reinterpret_cast<const uint2 *>(x + (t0 + t) * x_stride + k);
            }
            float xs[kRouterVecs][4];
#pragma unroll
            for (int v = 0; v < kRouterVecs; ++v) {
                xs[v][0] = bf_lo(xv[v].x), xs[v][1] = bf_hi(xv[v].x);
                xs[v][2] = bf_lo(xv[v].y), xs[v][3] = bf_hi(xv[v].y);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mx = fmaxf(mx, fabsf(xs[v][j]));
            }
#pragma unroll
            for (int e = 0; e < kRouterExperts; ++e) {
                // 20 terms of at most mx mw each are below 2^(E + 1), E the exponent of 32 mx mw; 1.5 2^(E + 2)
                const float bound = __fmul_rn(__fmul_rn(mx, 32.0f), mw[e]);
                const float seed = __fmul_rn(
                    __uint_as_float(max(__float_as_uint(bound) & 0x7f800000u, 0x01000000u)), 6.0f);
                float acc = seed, lo = 0.0f;
#pragma unroll
                for (int v = 0; v < kRouterVecs; ++v) {
                    const float ws[4] = {w[e][v].x, w[e][v].y, w[e][v].z, w[e][v].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float next = __fmaf_rn(xs[v][j], ws[j], acc);
                        lo = __fadd_rn(lo, __fmaf_rn(xs[v][j], ws[j], -__fsub_rn(next, acc)));
                        acc = next;
                    }
                }
                Sum2 &s = total[e * kRouterTokens + t];
                // a NaN or infinite term: seed or sum is not finite, and the logit is NaN
                s = sum_merge(s, Sum2{__fsub_rn(acc, seed), lo});
            }
        }
    }
    // 16 sums over 32 lanes: each step hands half of the sums to the other half of the lanes
#pragma unroll
    for (int half = kRouterSums / 2; half > 0; half /= 2) {
        const int off = half * 2;  // lanes 16, 8, 4, 2 apart
        const bool upper = lane & off;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const Sum2 a = total[i], b = total[i + half];
            total[i] = merge_across(upper ? b : a, upper ? a : b, off);
        }
    }
    const Sum2 mine = merge_across(total[0], total[0], 1);
    if ((lane & 1) == 0)
        s_part[warp][lane >> 1] = mine;
    __syncthreads();
    if (threadIdx.x < kRouterSums) {
        const int e = threadIdx.x / kRouterTokens, t = threadIdx.x % kRouterTokens;
        Sum2 v = s_part[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < kWarps; ++i)
            v = sum_merge(v, s_part[i][threadIdx.x]);
        if (t < n)
            logits[(int64_t)(t0 + t) * kExperts + e0 + e] = sum_value(v);
    }
}

// ---------------------------------------------------------------------------------------------
// passes: an expert of this rank with up to 8 of its pairs
// ---------------------------------------------------------------------------------------------

struct Passes {
    int count;
    int info[kMaxPasses];                   // expert, and the number of its tokens times 2^16
    uint4 pairs[kMaxPasses];                // 8 16-bit numbers: token * 8 + k
    __device__ __forceinline__ int expert(int p) const { return info[p] & 0xffff; }
    __device__ __forceinline__ int tokens(int p) const { return info[p] >> 16; }
    __device__ __forceinline__ int pair(int p, int j) const
    {
        return reinterpret_cast<const int16_t *>(&pairs[p])[j];
    }
};

// What building them takes.
struct PassScratch {
    int scan[kWarps];
    int16_t begin[kExperts];                // an expert's first pass
    int16_t fill[kWarps][kExperts];         // its pairs, by the warp that counted them
    int32_t ids[kFusedTokens * kTopK];      // of tokens that this block routed
};

__host__ __device__ constexpr int most_passes(int T)
{
    return T * kTopK < kExperts + T ? T * kTopK : kExperts + T;
}

// All threads.  Passes are in the order of experts, an expert's pairs in their own: every block makes the same ones,
// since blocks share a pass's places.  A warp takes T pairs and counts them by expert, 32 at a time.
__device__ __forceinline__ void build_passes(Passes &list, PassScratch &ps, const int32_t *ids, int T,
                                             int first, int local)
{
    constexpr int kEach = kMaxTokens / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kWarps * kExperts; i += kThreads)
        ps.fill[i / kExperts][i % kExperts] = 0;
    __syncthreads();
    int expert[kEach], place[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        expert[i] = -1;
        if (i * 32 >= T)
            continue;
        const int at = i * 32 + lane;
        const int e = at < T ? ids[warp * T + at] - first : -1;
        const bool in = e >= 0 && e < local;
        const uint32_t same = __match_any_sync(0xffffffffu, in ? e : -1);
        const uint32_t before = same & ((1u << lane) - 1u);
        const int had = in ? ps.fill[warp][e] : 0;
        __syncwarp();
        if (in) {
            expert[i] = e;
            place[i] = had + __popc(before);
            if (before == 0u)
                ps.fill[warp][e] = (int16_t)(had + __popc(same));
        }
        __syncwarp();
    }
    __syncthreads();
    int mine = 0;  // of expert threadIdx.x; its counts become the pairs in front of each warp's
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int n = ps.fill[w][threadIdx.x];
        ps.fill[w][threadIdx.x] = (int16_t)mine;
        mine += n;
    }
    const int need = (mine + kPassTokens - 1) / kPassTokens;
    int at = need;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, at, off);
        if (lane >= off)
            at += o;
    }
    if (lane == 31)
        ps.scan[warp] = at;
    __syncthreads();
    at -= need;
    for (int i = 0; i < warp; ++i)
        at += ps.scan[i];
    ps.begin[threadIdx.x] = (int16_t)at;
    for (int i = 0; i < need; ++i)
        list.info[at + i] = (int)threadIdx.x | min(mine - i * kPassTokens, kPassTokens) << 16;
    if (threadIdx.x == kThreads - 1)
        list.count = at + need;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (expert[i] >= 0) {
            const int n = ps.fill[warp][expert[i]] + place[i];
            reinterpret_cast<int16_t *>(
                &list.pairs[ps.begin[expert[i]] + n / kPassTokens])[n % kPassTokens] =
                (int16_t)(warp * T + i * 32 + lane);
        }
    __syncthreads();
}

// ---------------------------------------------------------------------------------------------
// the warps' streams
// ---------------------------------------------------------------------------------------------

// Where the 16 bytes `c` of row `row` of a stage stand: rows that eight neighbouring threads read together, 2r and
// 2r + 1, take different halves of the 128 bytes that a row has.
__device__ __forceinline__ uint32_t swizzled(int row, int c)
{
    return (uint32_t)(row * 128 + ((c ^ (((row & 1) << 2) | ((row >> 1) & 3))) << 4));
}

// Rows of a tile that a lane copies: rows lane / 8 + 4 i of the weights and of the tokens; nullptr: none.
template <int XR>
struct Rows {
    const uint16_t *w[4];
    const uint16_t *x[XR / 4];
};

// How a block's tiles are shared out: `parts` warps take a part of a tile's columns each.
struct Cut {
    int32_t K, steps, parts;  // columns, stages of a whole tile
};

Cut make_cut(int K)
{
    Cut c;
    c.K = K;
    c.steps = (K + kCols - 1) / kCols;
    c.parts = c.steps >= 32 ? 8 : (c.steps >= 16 ? 4 : (c.steps >= 8 ? 2 : 1));
    return c;
}

__host__ __device__ constexpr int stage_bytes(int XR) { return (16 + XR) * 128; }
constexpr int kAreaBytes = 2 * kWarps * 128 * 4;

// All tiles of the block.  rows_of(tile) gives the rows that this lane copies; drained() is called once by each
// warp when its last copy is under way.  Joint: done(round, area) is called by all threads behind a barrier, with the
// sums [warp][16 rows][8 tokens] of the round's 8 / parts tiles.  Otherwise warps go on by themselves, and a warp calls
// done(tile, part, its sums).  XR is 8, or 16: the tokens' rows in two parts whose sum they are.
template <int XR, int D, bool Joint, typename RowsOf, typename Done, typename Drained>
__device__ __forceinline__ void run_tiles(char *smem, float *area, const Cut &c, int tiles, RowsOf rows_of,
                                          Done done, Drained drained)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int at_once = kWarps / c.parts, rounds = (tiles + at_once - 1) / at_once;
    const int first = warp / c.parts, part = warp % c.parts;
    const int s0 = c.steps * part / c.parts, steps = c.steps * (part + 1) / c.parts - s0;
    const int mine = tiles > first ? (tiles - first + at_once - 1) / at_once : 0;
    const uint32_t base = smem_addr(smem) + warp * D * stage_bytes(XR);

    // copying
    Rows<XR> rows;
    int tile = first, step = 0, left = mine * steps, put = 0;
    const int chunk = lane & 7, row = lane >> 3;
    auto open_tile = [&]() {
        rows = rows_of(tile);
        // past the last column nothing is read, and zeros take its place; rows that are not there are not
        // copied: what stands in their places reaches only their own sums, which nobody takes
        const int k = s0 * kCols + chunk * 8 < c.K ? s0 * kCols + chunk * 8 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            rows.w[i] = rows.w[i] ? rows.w[i] + k : nullptr;
#pragma unroll
        for (int i = 0; i < XR / 4; ++i)
            rows.x[i] = rows.x[i] ? rows.x[i] + k : nullptr;
    };
    auto copy_next = [&]() {
        if (left > 0) {
            if (step == 0)
                open_tile();
            const uint32_t to = base + put * stage_bytes(XR);
            const bool in = (s0 + step) * kCols + chunk * 8 < c.K;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (rows.w[i])
                    cp_async16(to + swizzled(i * 4 + row, chunk), rows.w[i] + (in ? step * kCols : 0),
                               in ? 16u : 0u);
            }
#pragma unroll
            for (int i = 0; i < XR / 4; ++i) {
                if (rows.x[i])
                    cp_async16(to + 2048 + swizzled(i * 4 + row, chunk),
                               rows.x[i] + (in ? step * kCols : 0), in ? 16u : 0u);
            }
            put = put + 1 == D ? 0 : put + 1;
            if (++step == steps) {
                step = 0;
                tile += at_once;
            }
            if (--left == 0)
                drained();
        }
        cp_async_commit();
    };
    if (mine == 0)
        drained();
    // not unrolled: code that runs once is bound by its fetching
#pragma unroll 1
    for (int i = 0; i < D - 1; ++i)
        copy_next();

    int get = 0;
    for (int round = 0; round < rounds; ++round) {
        float *sums = area + (round & 1) * kWarps * 128;
        if (round * at_once + first < tiles) {
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
            for (int s = 0; s < steps; ++s) {
                cp_async_wait<D - 2>();
                __syncwarp();
                copy_next();
                const uint32_t from = base + get * stage_bytes(XR);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t a = from + swizzled(g, h * 4 + t);
                    const uint4 lo = lds128(a), hi = lds128(a + 1024);
                    const uint32_t f0[4] = {lo.x, hi.x, lo.y, hi.y}, f1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
                    for (int y = 0; y < XR / 8; ++y) {
                        const uint4 x = lds128(a + 2048 + y * 1024);
                        mma16816<false>(acc, f0, x.x, x.y);
                        mma16816<false>(acc, f1, x.z, x.w);
                    }
                }
                get = get + 1 == D ? 0 : get + 1;
            }
            if constexpr (Joint) {
                float *to = sums + warp * 128;
                *reinterpret_cast<float2 *>(to + g * 8 + 2 * t) = make_float2(acc[0], acc[1]);
                *reinterpret_cast<float2 *>(to + (8 + g) * 8 + 2 * t) = make_float2(acc[2], acc[3]);
            } else {
                done(round * at_once + first, part, acc);
            }
        }
        if constexpr (Joint) {
            __syncthreads();
            done(round, sums);
        }
    }
    cp_async_wait<0>();
}

struct ShareArgs {
    const uint16_t *x;
    int64_t x_stride;
    const uint16_t *w13, *w2;
    uint16_t *act;             // [2][T * 8, F]: the activations in two BF16 parts
    uint16_t *out;
    int64_t out_stride;
    const float *logits, *bias;
    int32_t *ids;
    float *weights;
    Passes *passes;
    int32_t first, local, T, H, F;
    float scaling;
    Cut cut;
    float *sums;               // [sum_rows][H]: a pair's share of the output, by part and pair
    int32_t sum_rows;
};

// The block's rows of the down projection: [from, to).
__device__ __forceinline__ void down_rows(const ShareArgs &a, int block, int blocks, int &from, int &to)
{
    from = (int)((int64_t)a.H * block / blocks);
    to = (int)((int64_t)a.H * (block + 1) / blocks);
}

// ---------------------------------------------------------------------------------------------
// up: a = silu(g) u
// ---------------------------------------------------------------------------------------------

// A block's share of the places (of F) of all passes, in tiles of up to 8 places of one pass: a first run that
// may start inside a pass, whole passes, a last run.
struct UpTiles {
    int64_t at, end;
    int F, first_pass, first_run, first_tiles, whole_tiles, count;
    __device__ __forceinline__ UpTiles(int64_t from, int64_t to, int F_) : at(from), end(to), F(F_)
    {
        count = first_tiles = first_pass = first_run = 0;
        whole_tiles = (F + 7) / 8;
        if (from >= to)
            return;
        first_pass = (int)(from / F);
        const int64_t stop = ((int64_t)first_pass + 1) * F;
        first_run = (int)((stop < to ? stop : to) - from);
        first_tiles = (first_run + 7) / 8;
        const int64_t rest = to - from - first_run;
        count = first_tiles + (int)(rest / F) * whole_tiles + (int)((rest % F + 7) / 8);
    }
    // its pass, first place and number of places
    __device__ __forceinline__ void get(int i, int &pass, int &f, int &n) const
    {
        int run = first_run, tiles = first_tiles, f0;
        pass = first_pass;
        if (i < first_tiles) {
            f0 = (int)(at - (int64_t)first_pass * F);
        } else {
            i -= first_tiles;
            const int over = i / whole_tiles;
            i -= over * whole_tiles;
            pass += 1 + over;
            f0 = 0;
            const int64_t rest = end - (int64_t)pass * F;
            run = rest < F ? (int)rest : F;
            tiles = (run + 7) / 8;
        }
        // even: none much smaller than the others
        f = run * i / tiles;
        n = run * (i + 1) / tiles - f;
        f += f0;
    }
};

__global__ void __launch_bounds__(kThreads, 1) moe_up_kernel(const ShareArgs a)
{
    extern __shared__ __align__(128) char smem[];
    __shared__ Passes ps;
    __shared__ PassScratch scratch;
    float *area = reinterpret_cast<float *>(smem + kWarps * kUpStages * stage_bytes(8));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const bool fused = a.T <= kFusedTokens;
    if (fused) {
#pragma unroll 1
        for (int t = warp; t < a.T; t += kWarps) {
            const float4 z0 = ld_stream_f4(a.logits + t * kExperts + lane * kPerLane);
            const float4 z1 = ld_stream_f4(a.logits + t * kExperts + lane * kPerLane + 4);
            const float4 b0 = *reinterpret_cast<const float4 *>(a.bias + lane * kPerLane);
            const float4 b1 = *reinterpret_cast<const float4 *>(a.bias + lane * kPerLane + 4);
            const float z[kPerLane] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
            const float bias[kPerLane] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
            const int id = route_ids(z, bias, lane);
            if (lane < kTopK)
                scratch.ids[t * kTopK + lane] = id;
        }
        __syncthreads();
    }
    build_passes(ps, scratch, fused ? scratch.ids : a.ids, a.T, a.first, a.local);
    if (blockIdx.x == 0) {  // for the next kernel
        for (int i = threadIdx.x; i < ps.count; i += kThreads) {
            a.passes->info[i] = ps.info[i];
            a.passes->pairs[i] = ps.pairs[i];
        }
        if (threadIdx.x == 0)
            a.passes->count = ps.count;
    }
    const int64_t places = (int64_t)ps.count * a.F;
    const UpTiles tiles(places * blockIdx.x / gridDim.x, places * (blockIdx.x + 1) / gridDim.x, a.F);
    const int64_t n_act = (int64_t)a.T * kTopK * a.F;
    run_tiles<8, kUpStages, true>(
        smem, area, a.cut, tiles.count,
        [&](int i) {
            int pass, f, n;
            tiles.get(i, pass, f, n);
            const uint16_t *w = a.w13 + ((int64_t)ps.expert(pass) * 2 * a.F + f) * a.H;
            Rows<8> r;
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // rows 0-7: gate; 8-15: up
                const int row = (lane >> 3) + 4 * j;
                r.w[j] = (row & 7) < n ? w + ((row & 7) + (row < 8 ? 0 : (int64_t)a.F)) * a.H : nullptr;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = (lane >> 3) + 4 * j;
                r.x[j] = row < ps.tokens(pass) ? a.x + (ps.pair(pass, row) / kTopK) * a.x_stride : nullptr;
            }
            return r;
        },
        [&](int round, const float *sums) {
            const int parts = a.cut.parts, at_once = kWarps / parts;
            // places run fastest: neighbouring threads write neighbouring values
            for (int i = threadIdx.x; i < at_once * 64; i += kThreads) {
                const int tile = round * at_once + (i >> 6), r = i & 7, j = (i >> 3) & 7;
                if (tile >= tiles.count)
                    break;
                int pass, f, n;
                tiles.get(tile, pass, f, n);
                if (r >= n || j >= ps.tokens(pass))
                    continue;
                const float *from = sums + (i >> 6) * parts * 128 + r * 8 + j;
                float g = 0.0f, u = 0.0f;
                for (int w = 0; w < parts; ++w) {
                    g += from[w * 128];
                    u += from[w * 128 + 64];
                }
                const float v = __fdiv_rn(g, 1.0f + expf(-g)) * u;
                const uint32_t hi = pack_bf16x2(v, 0.0f);
                uint16_t *to = a.act + (int64_t)ps.pair(pass, j) * a.F + f + r;
                to[0] = (uint16_t)hi;
                to[n_act] = (uint16_t)pack_bf16x2(__fsub_rn(v, bf_lo(hi)), 0.0f);
            }
        },
        [&]() {
            // This warp's last weights are on their way.  The choice's own weights are of use to the next kernel only.
            if (fused && blockIdx.x == 0) {
#pragma unroll 1
                for (int t = warp; t < a.T; t += kWarps) {
                    const int id = lane < kTopK ? scratch.ids[t * kTopK + lane] : 0;
                    const float w = route_weight(lane < kTopK ? a.logits[t * kExperts + id] : 0.0f);
                    if (lane < kTopK) {
                        a.ids[t * kTopK + lane] = id;
                        a.weights[t * kTopK + lane] = w;
                    }
                }
            }
            // The first weights that the next kernel's block here reads, up to 192 KB of them, are brought to the L2
            // cache while that kernel starts.
            if (warp != 0)
                return;
            int from, to;
            down_rows(a, blockIdx.x, gridDim.x, from, to);
            const uint32_t bytes = (uint32_t)(to - from) * (uint32_t)a.F * 2u;
            for (int p = lane; p < ps.count && bytes > 0 && (p + 1) * (int64_t)bytes <= 192 * 1024; p += 32)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                 a.w2 + ((int64_t)ps.expert(p) * a.H + from) * a.F),
                             "r"(bytes)
                             : "memory");
        });
}

// ---------------------------------------------------------------------------------------------
// down: out = sum over the pairs of scaling * weight * w2 a
// ---------------------------------------------------------------------------------------------

constexpr uint32_t kAbsent = 0xffffffffu;  // a NaN that no product gives

// A block owns some output columns, so it can add up by itself what its warps leave for each pair: warps never
// wait for one another until then.  Adding round by round in shared memory instead, in order behind barriers, took
// half of the kernel's instructions (64 tokens of an eighth: 308 us, TODO).
__global__ void __launch_bounds__(kThreads, 1) moe_down_kernel(const ShareArgs a)
{
    extern __shared__ __align__(128) char smem[];
    __shared__ Passes ps;
    __shared__ float weight[kMaxTokens * kTopK];  // scaled; kAbsent: the expert is not here
    const int lane = threadIdx.x & 31, g = lane >> 2, t2 = 2 * (lane & 3);
    pdl_launch_dependents();
    pdl_wait();
    const int most = most_passes(a.T);
#pragma unroll 1
    for (int i = threadIdx.x; i < most; i += kThreads) {
        ps.info[i] = a.passes->info[i];
        ps.pairs[i] = ld_plain(&a.passes->pairs[i]);
    }
    if (threadIdx.x == 0)
        ps.count = a.passes->count;
    __syncthreads();
    int r0, r1;
    down_rows(a, blockIdx.x, gridDim.x, r0, r1);
    const int rows = r1 - r0, row_tiles = (rows + 15) / 16, pairs = a.T * kTopK;
    Cut cut = a.cut;
    // few tiles: parts of their columns, so that each warp has some, while there is room for the parts' sums
    while (cut.parts < kWarps && row_tiles * ps.count * cut.parts < 3 * kWarps &&
           cut.steps >= 4 * cut.parts && 2 * cut.parts * pairs <= a.sum_rows)
        cut.parts *= 2;
    const int64_t n_act = (int64_t)pairs * a.F;
    run_tiles<16, kDownStages, false>(
        smem, nullptr, cut, row_tiles * ps.count,
        [&](int i) {
            const int pass = i / row_tiles, rt = i - pass * row_tiles;
            const int from = rows * rt / row_tiles, n = rows * (rt + 1) / row_tiles - from;
            const uint16_t *w = a.w2 + ((int64_t)ps.expert(pass) * a.H + r0 + from) * a.F;
            Rows<16> r;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = (lane >> 3) + 4 * j;
                r.w[j] = row < n ? w + (int64_t)row * a.F : nullptr;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = (lane >> 3) + 4 * j;
                r.x[j] = r.x[j + 2] = nullptr;
                if (row < ps.tokens(pass)) {
                    r.x[j] = a.act + (int64_t)ps.pair(pass, row) * a.F;
                    r.x[j + 2] = r.x[j] + n_act;
                }
            }
            return r;
        },
        [&](int i, int part, const float (&acc)[4]) {
            const int pass = i / row_tiles, rt = i - pass * row_tiles;
            const int from = rows * rt / row_tiles, n = rows * (rt + 1) / row_tiles - from;
            float *to = a.sums + (int64_t)part * pairs * a.H + r0 + from + g;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (t2 + j < ps.tokens(pass)) {
                    float *y = to + (int64_t)ps.pair(pass, t2 + j) * a.H;
                    if (g < n)
                        y[0] = acc[j];
                    if (g + 8 < n)
                        y[8] = acc[2 + j];
                }
        },
        [&]() {
            // with the last copies under way: the pairs' weights
#pragma unroll 1
            for (int i = threadIdx.x; i < pairs; i += kThreads) {
                const int e = a.ids[i] - a.first;
                weight[i] = a.scaling * a.weights[i];
                if (e < 0 || e >= a.local)
                    weight[i] = __uint_as_float(kAbsent);
            }
        });
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * rows; i += kThreads) {
        const int t = i / rows, r = i - t * rows;
        const float *y = a.sums + (int64_t)t * kTopK * a.H + r0 + r;
        float sum = 0.0f;
        float v[kTopK];
#pragma unroll
        for (int k = 0; k < kTopK; ++k) {
            v[k] = 0.0f;
            if (__float_as_uint(weight[t * kTopK + k]) != kAbsent)
                for (int p = 0; p < cut.parts; ++p)
                    v[k] += y[(int64_t)(p * pairs + k) * a.H];
        }
#pragma unroll
        for (int k = 0; k < kTopK; ++k)
            if (__float_as_uint(weight[t * kTopK + k]) != kAbsent)
                sum = __fmaf_rn(weight[t * kTopK + k], v[k], sum);
        a.out[t * a.out_stride + r0 + r] = (uint16_t)pack_bf16x2(sum, 0.0f);
    }
}

template <auto Kernel>
cudaError_t launch_share(const ShareArgs &s, int grid, int smem, cudaStream_t stream)
{
    static int done[64] = {};  // the most shared memory that was asked for
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || done[dev] < smem)) {
        e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && dev < 64)
            done[dev] = smem;
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
    p.passes = p.weights + T * kTopK * 4;
    p.act = p.passes + (int64_t)sizeof(Passes);
    p.sums = p.act + 2 * T * kTopK * F * 2;
    p.sum_rows = T * kTopK > kSumRows ? T * kTopK : kSumRows;
    p.bytes = p.sums + p.sum_rows * H * 4;
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
    s.logits = logits;
    s.bias = a.router_bias;
    s.ids = a.ids ? a.ids : (int32_t *)(a.workspace + p.ids);
    s.weights = a.weights ? a.weights : (float *)(a.workspace + p.weights);
    s.passes = (Passes *)(a.workspace + p.passes);
    s.sums = (float *)(a.workspace + p.sums);
    s.sum_rows = (int32_t)p.sum_rows;
    s.first = a.first;
    s.local = a.local;
    s.T = a.T;
    s.H = a.H;
    s.F = a.F;
    s.scaling = a.scaling;
    cudaError_t e = launch_pdl(moe_router_kernel,
                               dim3(kExperts / kRouterExperts, (a.T + kRouterTokens - 1) / kRouterTokens),
                               dim3(kThreads), 0, stream, logits, s.x, s.x_stride, a.router_w, a.T, a.H);
    if (e == cudaSuccess && a.T > kFusedTokens) {
        RouteArgs r{};
        r.logits = logits;
        r.bias = a.router_bias;
        r.ids = s.ids;
        r.weights = s.weights;
        r.T = a.T;
        e = launch_grouped_topk(r, stream);
    }
    // both kernels have a block an SM: a block of the second finds its first weights in the L2 cache
    const int down = a.H < kSms ? a.H : kSms;
    if (e == cudaSuccess) {
        s.cut = make_cut(a.H);
        e = launch_share<moe_up_kernel>(s, kSms, kWarps * kUpStages * stage_bytes(8) + kAreaBytes, stream);
    }
    if (e == cudaSuccess) {
        s.cut = make_cut(a.F);
        s.cut.parts = 1;
        e = launch_share<moe_down_kernel>(s, down, kWarps * kDownStages * stage_bytes(16), stream);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace beam
