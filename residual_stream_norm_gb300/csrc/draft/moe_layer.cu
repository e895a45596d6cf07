// moe_layer.cu -- a whole mixture-of-experts layer for a few tokens (sm_103a).
//
// With up to 256 tokens and 8 of 256 experts each, an expert has a handful of tokens: the layer is bound by
// reading the chosen experts' weights, each once.  Kernels:
//  1. router: z = x router_w^T in FP32 pairs;
//  2. the grouped top-k of beam_grouped_topk_fwd: for up to 16 tokens in every block of the next kernel (a chain
//     shorter by a kernel), a warp to a token, else as that kernel;
//  3. up: g, u and a = silu(g) u for each (token, expert) pair;
//  4. down: each pair's share of the output, in FP32, by the same code;
//  5. the weighted sum of each token's pairs, in order.
//
// An expert's tokens are taken in passes of up to 8 (up) or 4 (down); all passes' rows of weights, one after the other,
// are cut into equal shares for the blocks, so that a block reads one stretch of memory but where it passes from expert to
// expert (a block that owned columns of the output instead, for all experts: the layer of 64 tokens of a tensor-parallel
// eighth 404 us, 358 this way).  Each of a block's eight warps has a stream of its own: 16 rows of weights by 128 columns
// at a time, copied with cp.async some stages ahead into the warp's part of shared memory together with the tokens'
// rows that they meet (bulk copies of a row's kilobyte, one instruction each, ran at 1.9 TB/s).  They are multiplied
// with m16n8k16 instructions whose left operand is the weights (for up: 8 rows of the gate and the same 8 of the up
// projection, so that one thread holds g and u of the same place) and whose right one is 8 tokens' rows, or for down
// both BF16 parts of 4 tokens' activations.  Both operands are read 16 bytes a thread: the instruction's columns are the
// row's in another order, the same for both.  Up: warps take parts of a tile's columns, and their sums meet in shared
// memory, in order.  Down: a warp's sums go to memory (FP32, one place for each pair, row and part of the columns).
// Later passes of an expert find its weights in the L2 cache.
//
// What bounds it: memory for many tokens (64 of a tensor-parallel eighth, 2.2 GB: 355 us, 0.91 of the measured copy rate;
// kernels 33, 11, 185, 133 and 6 us one at a time, caches cold), the chain of four kernels for one (84 MB: 33 us; 7, 23, 14
// and 9 cold, each a few us of launch, first instructions and first loads).

#include "beam_device.cuh"
#include "beam_f32x2.cuh"
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
constexpr int kCols = 128;         // columns of a stage
constexpr int kSumRows = 512;      // least rows of the down kernel's sums

// ---------------------------------------------------------------------------------------------
// router
// ---------------------------------------------------------------------------------------------

// A block takes two experts and up to 8 tokens; a thread the columns 4 i, i = its number modulo 256, of both.
// A sum starts at a power of two times 1.5 that is larger than twice all of its terms together: each
// addition rounds to a grid that the running sum never leaves, so that the part taken up, acc' - acc, is exact, and
// what is left of the product, one fused multiply-add, goes into a second sum: four operations a product, where pairs
// by TwoSum take ten.  Both experts' go in one packed instruction.
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

__global__ void __launch_bounds__(kThreads, 2)
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
        uint2 ahead[kRouterVecs];  // the next token's columns
        auto load_token = [&](int t) {
#pragma unroll
            for (int v = 0; v < kRouterVecs; ++v) {
                const int k = k0 + (v * kThreads + threadIdx.x) * 4;
                ahead[v] = make_uint2(0u, 0u);
                if (k < H)
                    ahead[v] = *reinterpret_cast<const uint2 *>(x + (t0 + t) * x_stride + k);
            }
        };
        load_token(0);
#pragma unroll
        for (int t = 0; t < kRouterTokens; ++t) {
            if (t >= n)
                continue;
            uint2 xv[kRouterVecs];
            float mx = 0.0f;
#pragma unroll
            for (int v = 0; v < kRouterVecs; ++v)
                xv[v] = ahead[v];
            if (t + 1 < n)
                load_token(t + 1);
            float xs[kRouterVecs][4];
#pragma unroll
            for (int v = 0; v < kRouterVecs; ++v) {
                xs[v][0] = bf_lo(xv[v].x), xs[v][1] = bf_hi(xv[v].x);
                xs[v][2] = bf_lo(xv[v].y), xs[v][3] = bf_hi(xv[v].y);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mx = fmaxf(mx, fabsf(xs[v][j]));
            }
            // 20 terms of at most mx mw each are below 2^(E + 1), E the exponent of 32 mx mw; 1.5 2^(E + 2)
            float seed[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float bound = __fmul_rn(__fmul_rn(mx, mw[e]), 32.0f);  // (mx may be near FP32's end)
                seed[e] = __fmul_rn(
                    __uint_as_float(max(__float_as_uint(bound) & 0x7f800000u, 0x01000000u)), 6.0f);
            }
            const f2 start = make_f2(seed[0], seed[1]);
            f2 acc = start, lo = splat(0.0f);
#pragma unroll
            for (int v = 0; v < kRouterVecs; ++v) {
                const f2 ws[4] = {make_f2(w[0][v].x, w[1][v].x), make_f2(w[0][v].y, w[1][v].y),
                                  make_f2(w[0][v].z, w[1][v].z), make_f2(w[0][v].w, w[1][v].w)};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f2 x2 = splat(xs[v][j]), next = fma2(x2, ws[j], acc);
                    lo = add2(lo, fma2(x2, ws[j], sub2(acc, next)));
                    acc = next;
                }
            }
            acc = sub2(acc, start);
            // a NaN or infinite term: seed or sum is not finite, and the logit is NaN
            total[t] = sum_merge(total[t], Sum2{lo_of(acc), lo_of(lo)});
            total[kRouterTokens + t] = sum_merge(total[kRouterTokens + t], Sum2{hi_of(acc), hi_of(lo)});
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

// For down a pass has up to 4 tokens, whose activations' two BF16 parts fill the 8 columns of its products.
constexpr int kDownTokens = 4;
constexpr int kMaxDownPasses = kExperts + 2 * kMaxTokens;  // sum over experts of ceil(pairs / 4)

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
    int32_t pass_of[kFusedTokens * kTopK];
};

struct DownPasses {
    int count;
    int info[kMaxDownPasses];               // expert, and the number of its tokens times 2^16
    uint2 pairs[kMaxDownPasses];            // 4 16-bit numbers
};

__host__ __device__ constexpr int most_down_passes(int T)
{
    return T * kTopK < kExperts + 2 * T ? T * kTopK : kExperts + 2 * T;
}

// Passes of up to 8 tokens as passes of up to 4, by one warp.
__device__ __forceinline__ void split_passes(DownPasses &to, const Passes &ps, int lane)
{
    int at = 0;
#pragma unroll 1
    for (int p0 = 0; p0 < ps.count; p0 += 32) {
        const int p = p0 + lane;
        const bool on = p < ps.count;
        const int tokens = on ? ps.tokens(p) : 0;
        const uint32_t two = __ballot_sync(0xffffffffu, tokens > kDownTokens), below = (1u << lane) - 1u;
        if (on) {
            const int i = at + lane + __popc(two & below);
            const uint4 pairs = ps.pairs[p];
            to.info[i] = ps.expert(p) | min(tokens, kDownTokens) << 16;
            to.pairs[i] = make_uint2(pairs.x, pairs.y);
            if (tokens > kDownTokens) {
                to.info[i + 1] = ps.expert(p) | (tokens - kDownTokens) << 16;
                to.pairs[i + 1] = make_uint2(pairs.z, pairs.w);
            }
        }
        at += min(ps.count - p0, 32) + __popc(two);
    }
    if (lane == 0)
        to.count = at;
}

// Passes of up to 128 pairs, whose experts stand in ps.ids, by pair: which earlier pairs have the same expert.
// Passes are in the order of their first pairs.  All threads; every block makes the same ones, since blocks share a
// pass's places.
__device__ __forceinline__ void build_few_passes(Passes &list, PassScratch &ps, int n, int first, int local)
{
    const int i = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = i < n ? ps.ids[i] : -1;
    const bool in = e >= first && e < first + local;
    int before = 0, lead = i;  // the pair that opens this one's pass
    if (in) {
#pragma unroll 1
        for (int j = 0; j < i; ++j)
            if (ps.ids[j] == e) {
                lead = before % kPassTokens == 0 ? j : lead;
                ++before;
            }
    }
    const bool opens = in && before % kPassTokens == 0;
    const uint32_t all = __ballot_sync(0xffffffffu, opens);
    if (lane == 0)
        ps.scan[warp] = __popc(all);
    __syncthreads();
    int pass = __popc(all & ((1u << lane) - 1u)), total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        pass += w < warp ? ps.scan[w] : 0;
        total += ps.scan[w];
    }
    if (opens) {
        ps.pass_of[i] = pass;
        list.info[pass] = 0;
    }
    if (i == 0)
        list.count = total;
    __syncthreads();
    if (in) {
        pass = ps.pass_of[opens ? i : lead];
        reinterpret_cast<int16_t *>(&list.pairs[pass])[before % kPassTokens] = (int16_t)i;
        // the last pair of the pass has the largest number
        atomicMax(&list.info[pass], (e - first) | (before % kPassTokens + 1) << 16);
    }
    __syncthreads();
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
// up and down: one kernel, since code that a kernel runs for the first time on an SM comes from far: the second run
// finds most of it there
// ---------------------------------------------------------------------------------------------

constexpr int kStages = 4;
constexpr int kRowBytes = kCols * 2;
constexpr int kStageBytes = (16 + 8) * kRowBytes;  // 16 rows of weights and 8 of tokens
constexpr int kAreaBytes = 2 * kWarps * 128 * 4;

// Where the 16 bytes `c` of row `row` of a stage stand: rows that eight neighbouring threads read together, 2r and
// 2r + 1, take different halves of the 128 bytes that a row has.
__device__ __forceinline__ uint32_t swizzled(int row, int c)
{
    return (uint32_t)(row * kRowBytes + ((c ^ (((row & 1) << 2) | ((row >> 1) & 3))) << 4));
}

// How a block's tiles are shared out: `parts` warps take a part of a tile's columns each.
struct Cut {
    int32_t K, steps, parts;  // columns, stages of a whole tile
};

Cut make_cut(int K)
{
    Cut c;
    c.K = K;
    c.steps = (K + kCols - 1) / kCols;
    c.parts = c.steps >= 16 ? 8 : (c.steps >= 8 ? 4 : (c.steps >= 4 ? 2 : 1));
    return c;
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
    DownPasses *passes;
    float *sums;               // [sum_rows][H]: a pair's share of the output, by part and pair
    int32_t sum_rows;
    int32_t first, local, T, H, F;
    float scaling;
    bool down;
    Cut cut;
};

// What is cut: up, the F places of each pass, in tiles of up to 8 (two rows of weights each); down, the H rows of each
// pass, in tiles of up to 16.
__device__ __forceinline__ uint32_t unit_of(const ShareArgs &a) { return (uint32_t)(a.down ? a.H : a.F); }
__device__ __forceinline__ int tile_shift(const ShareArgs &a) { return a.down ? 4 : 3; }

// Parts of a tile's columns for the down kernel: where blocks have few tiles, each warp gets some, while there is room
// for the parts' sums.
__device__ __forceinline__ int down_parts(const ShareArgs &a, int passes)
{
    const uint32_t tiles = ((uint32_t)passes * a.H + kSms * 16 - 1) / (kSms * 16);  // of a block
    int parts = 1;
    while (parts < kWarps && tiles * parts < 3 * kWarps && a.cut.steps >= 2 * parts &&
           2 * parts * a.T * kTopK <= a.sum_rows)
        parts *= 2;
    return parts;
}

// The tiles of a block's share [at, end) of all passes' places (rows), in order: runs inside a pass, each cut evenly, so
// that no tile is much smaller than the others.  A share is one stretch of memory but where it passes from expert to
// expert.
struct Tiles {
    int pass, from, n;  // the tile at hand: its pass, first place, and their number
    int i, tiles;       // its number in the run, the run's tiles
    uint32_t at, end;   // behind the run, behind all
    int start;          // first place of the run
    int base, more;     // tiles have base places, the first `more` of them one more

    __device__ __forceinline__ void open_run(uint32_t unit, int shift)
    {
        pass = (int)(at / unit);
        start = (int)(at - (uint32_t)pass * unit);
        const int size = min((int)(end - at), (int)unit - start);
        tiles = (size + (1 << shift) - 1) >> shift;
        base = size / tiles;
        more = size - base * tiles;
        at += size;
        i = 0;
    }
    // `by` tiles on; in front of the first at the beginning
    __device__ __forceinline__ void go(uint32_t unit, int shift, int by)
    {
#pragma unroll 1
        for (; by > 0; --by)
            if (++i >= tiles)
                open_run(unit, shift);
        from = start + i * base + min(i, more);
        n = base + (i < more ? 1 : 0);
    }
    __device__ __forceinline__ int count(uint32_t unit, int shift) const
    {
        const uint32_t t = (1u << shift) - 1, f0 = at % unit, all = end - at;
        const uint32_t n0 = min(all, unit - f0), rest = all - n0;  // the first run, and what is behind it
        return (int)(((n0 + t) >> shift) + rest / unit * ((unit + t) >> shift) + ((rest % unit + t) >> shift));
    }
};

// Two blocks' registers to an SM, so that one starts beside the router's.
__global__ void __launch_bounds__(kThreads, 2) moe_share_kernel(const ShareArgs a)
{
    extern __shared__ __align__(128) char smem[];
    __shared__ PassScratch scratch;
    __shared__ __align__(16) char lists[sizeof(Passes)];
    static_assert(sizeof(DownPasses) <= sizeof(Passes), "one place for either list");
    Passes &ps = *reinterpret_cast<Passes *>(lists);
    DownPasses &ds = *reinterpret_cast<DownPasses *>(lists);
    // the list at hand: count, info, and the pairs of pass p, token j
    const int &passes = a.down ? ds.count : ps.count;
    const int *info = a.down ? ds.info : ps.info;
    const int16_t *pair_of = a.down ? reinterpret_cast<const int16_t *>(ds.pairs)
                                    : reinterpret_cast<const int16_t *>(ps.pairs);
    const int per_pass = a.down ? kDownTokens : kPassTokens;
    float *area = reinterpret_cast<float *>(smem + kWarps * kStages * kStageBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const bool fused = !a.down && a.T <= kFusedTokens;
    const int pairs = a.T * kTopK;
    pdl_launch_dependents();
    // Twice: first without a pair and without touching memory, while the kernel before still runs, which fetches the
    // code; then in earnest.  The up kernel finds room beside the router's blocks; the down kernel, which starts as
    // the up kernel's blocks end, has its code from them.
#pragma unroll 1
    for (int dry = a.down ? 0 : 1; dry >= 0; --dry) {
        if (!dry)
            pdl_wait();
        // ---- routing and passes --------------------------------------------------------------------------
        if (a.down) {
            const int most = most_down_passes(a.T);
#pragma unroll 1
            for (int i = threadIdx.x; i < most; i += kThreads) {
                ds.info[i] = a.passes->info[i];
                ds.pairs[i] = a.passes->pairs[i];
            }
            if (threadIdx.x == 0)
                ds.count = a.passes->count;
            __syncthreads();
        } else if (fused) {
#pragma unroll 1
            for (int tok = warp; tok < (dry ? kWarps : a.T); tok += kWarps) {
                float4 z0 = make_float4(lane, 0.0f, 1.0f, 2.0f), z1 = z0;
                if (!dry) {
                    z0 = ld_stream_f4(a.logits + tok * kExperts + lane * kPerLane);
                    z1 = ld_stream_f4(a.logits + tok * kExperts + lane * kPerLane + 4);
                }
                const float4 b0 = *reinterpret_cast<const float4 *>(a.bias + lane * kPerLane);
                const float4 b1 = *reinterpret_cast<const float4 *>(a.bias + lane * kPerLane + 4);
                const float z[kPerLane] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
                const float bias[kPerLane] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
                const int id = route_ids(z, bias, lane);
                if (lane < kTopK)
                    scratch.ids[tok * kTopK + lane] = id;
            }
            __syncthreads();
            build_few_passes(ps, scratch, dry ? kTopK : pairs, dry ? 0 : a.first, dry ? kExperts : a.local);
        } else {
            build_passes(ps, scratch, a.ids, dry ? 0 : a.T, a.first, a.local);
        }
        if (!dry && !a.down && blockIdx.x == 0 && warp == kWarps - 1)
            split_passes(*a.passes, ps, lane);
        // ---- the block's tiles ------------------------------------------------------------------------------
        // block 0 of up, which also finishes the routing of few tokens, takes half a share then
        Cut cut = a.cut;
        Tiles ld;
        const uint32_t unit = unit_of(a);
        const int shift = tile_shift(a);
        {
            const uint64_t places = (uint64_t)((uint32_t)passes * unit);
            const uint32_t b = 2 * blockIdx.x;
            constexpr uint32_t kWhole = 2 * kSms;  // the grid's blocks, in halves
            ld.at = (uint32_t)(fused ? places * (b > 0 ? b - 1 : 0) / (kWhole - 1) : places * b / kWhole);
            ld.end = (uint32_t)(fused ? places * (b + 1) / (kWhole - 1) : places * (b + 2) / kWhole);
            ld.i = ld.tiles = 0;
        }
        if (a.down)
            cut.parts = down_parts(a, passes);
        if (dry) {
            ld.at = 0;
            ld.end = 1;
            cut.steps = cut.parts;
        }
        const int count = ld.count(unit, shift);
        Tiles cp = ld;
        // ---- the warps' streams ------------------------------------------------------------------------------
        // Up: `parts` warps take a part of a tile's columns each, and their sums meet behind a barrier, a round of
        // 8 / parts tiles at a time.  Down: warps go on by themselves.
        const int at_once = kWarps / cut.parts, rounds = (count + at_once - 1) / at_once;
        const int first = warp / cut.parts, part = warp - first * cut.parts;
        const int s0 = cut.steps * part / cut.parts, steps = cut.steps * (part + 1) / cut.parts - s0;
        const int mine = count > first ? (count - first + at_once - 1) / at_once : 0;
        const uint32_t base = smem_addr(smem) + warp * kStages * kStageBytes;
        const int chunk = lane & 7, row = lane >> 3;
        const int64_t n_act = (int64_t)pairs * a.F;

        const uint16_t *w[4], *x[2];  // rows lane / 8 + 4 i of the weights and of the tokens; nullptr: none
        int step = 0, left = mine * steps, put = 0, by = first + 1;
        auto open_tile = [&]() {
            ld.go(unit, shift, by);
            by = at_once;
            // past the last column nothing is read, and zeros take its place; rows that are not there are not
            // copied: what stands in their places reaches only their own sums, which nobody takes
            const int k = s0 * kCols + chunk * 8 < cut.K ? s0 * kCols + chunk * 8 : 0;
            const int what = info[ld.pass], e = what & 0xffff;
            const int tokens = dry ? 0 : what >> 16, n = dry ? 0 : ld.n;
            const int64_t pitch = a.down ? a.F : a.H;
            const uint16_t *from =
                (a.down ? a.w2 + ((int64_t)e * a.H + ld.from) * a.F
                        : a.w13 + ((int64_t)e * 2 * a.F + ld.from) * a.H) + k;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = row + 4 * i;  // up: 0-7 gate, 8-15 up
                const int64_t at = a.down ? r : (r & 7) + (r < 8 ? 0 : a.F);
                w[i] = (a.down ? r : r & 7) < n ? from + at * pitch : nullptr;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // up: tokens 0-3, 4-7; down: the first and second parts of tokens 0-3
                const int j = row + (a.down ? 0 : 4 * i);
                x[i] = nullptr;
                if (j < tokens) {
                    const int pair = pair_of[ld.pass * per_pass + j];
                    x[i] = (a.down ? a.act + i * n_act + (int64_t)pair * a.F
                                   : a.x + (pair / kTopK) * a.x_stride) + k;
                }
            }
        };
        auto copy_next = [&]() {
            if (left > 0) {
                if (step == 0)
                    open_tile();
                const uint32_t to = base + put * kStageBytes;
                // the two halves of the stage's columns
                const int k = (s0 + step) * kCols + chunk * 8;
                const int64_t off = k < cut.K ? step * kCols : 0;
                const int64_t off2 = k + 64 < cut.K ? step * kCols + 64 : 0;
                const uint32_t n1 = k < cut.K ? 16u : 0u, n2 = k + 64 < cut.K ? 16u : 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (w[i]) {
                        cp_async16(to + swizzled(i * 4 + row, chunk), w[i] + off, n1);
                        cp_async16(to + swizzled(i * 4 + row, chunk + 8), w[i] + off2, n2);
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (x[i]) {
                        cp_async16(to + swizzled(16 + i * 4 + row, chunk), x[i] + off, n1);
                        cp_async16(to + swizzled(16 + i * 4 + row, chunk + 8), x[i] + off2, n2);
                    }
                put = put + 1 == kStages ? 0 : put + 1;
                step = step + 1 == steps ? 0 : step + 1;
                --left;
            }
            cp_async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i)
            copy_next();

        int get = 0;
        bool drained = false;
#pragma unroll 1
        for (int round = 0; round < rounds; ++round) {
            float *meet = area + (round & 1) * kWarps * 128;
            const bool busy = round * at_once + first < count;
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (busy) {
#pragma unroll 1
                for (int s = 0; s < steps; ++s) {
                    cp_async_wait<kStages - 2>();
                    __syncwarp();
                    copy_next();
                    const uint32_t from = base + get * kStageBytes;
#pragma unroll
                    for (int h = 0; h < kCols / 32; ++h) {
                        const uint32_t at = from + swizzled(g, h * 4 + t);
                        const uint4 lo = lds128(at), hi = lds128(at + 8 * kRowBytes);
                        const uint4 y = lds128(at + 16 * kRowBytes);
                        const uint32_t f0[4] = {lo.x, hi.x, lo.y, hi.y}, f1[4] = {lo.z, hi.z, lo.w, hi.w};
                        mma16816<false>(acc, f0, y.x, y.y);
                        mma16816<false>(acc, f1, y.z, y.w);
                    }
                    get = get + 1 == kStages ? 0 : get + 1;
                }
            }
            if (a.down) {
                if (busy) {  // this warp's rows of the pairs' sums
                    cp.go(unit, shift, round == 0 ? first + 1 : at_once);
                    const int tokens = info[cp.pass] >> 16;
                    float *to = a.sums + (int64_t)part * pairs * a.H + cp.from + g;
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // both parts' products
                        acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 2);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (t < 2 && 2 * t + j < tokens) {
                            float *y = to + (int64_t)pair_of[cp.pass * kDownTokens + 2 * t + j] * a.H;
                            if (g < cp.n)
                                y[0] = acc[j];
                            if (g + 8 < cp.n)
                                y[8] = acc[2 + j];
                        }
                }
            } else {
                float *to = meet + warp * 128;
                *reinterpret_cast<float2 *>(to + g * 8 + 2 * t) = make_float2(acc[0], acc[1]);
                *reinterpret_cast<float2 *>(to + (8 + g) * 8 + 2 * t) = make_float2(acc[2], acc[3]);
                __syncthreads();
#pragma unroll 1
                for (int k = 0; k < at_once && round * at_once + k < count; ++k) {
                    cp.go(unit, shift, 1);
                    // places run fastest: neighbouring threads write neighbouring values
                    const int r = threadIdx.x & 7, j = (threadIdx.x >> 3) & 7;
                    if (threadIdx.x >> 6 != (k & 3) || r >= cp.n || j >= ps.tokens(cp.pass) || dry)
                        continue;
                    const float *from = meet + k * cut.parts * 128 + r * 8 + j;
                    float gate = 0.0f, up = 0.0f;
#pragma unroll 1
                    for (int i = 0; i < cut.parts; ++i) {
                        gate += from[i * 128];
                        up += from[i * 128 + 64];
                    }
                    const float v = __fdiv_rn(gate, 1.0f + expf(-gate)) * up;
                    const uint32_t hi = pack_bf16x2(v, 0.0f);
                    uint16_t *y = a.act + (int64_t)ps.pair(cp.pass, j) * a.F + cp.from + r;
                    y[0] = (uint16_t)hi;
                    y[n_act] = (uint16_t)pack_bf16x2(__fsub_rn(v, bf_lo(hi)), 0.0f);
                }
            }
            if (!drained && left == 0 && !dry && !a.down && warp == 0) {
                // The last weights are on their way.  The first ones that the down kernel's block here reads, up to
                // 192 KB of them, are brought to the L2 cache while that kernel starts.
                drained = true;
                const uint32_t at = (uint32_t)((uint64_t)((uint32_t)passes * a.H) * blockIdx.x / kSms);
                const uint32_t p = at / a.H, r = at - p * a.H;
                const int64_t rest = (int64_t)(a.H - r) * a.F * 2;  // of the pass
                const uint32_t bytes = (uint32_t)(rest < 192 * 1024 ? rest : 192 * 1024) / 32 / 16 * 16;
                if (bytes > 0 && passes > 0)
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                     (const char *)(a.w2 + ((int64_t)ps.expert(p) * a.H + r) * a.F) +
                                     lane * bytes),
                                 "r"(bytes)
                                 : "memory");
            }
        }
        cp_async_wait<0>();
        __syncthreads();
        if (fused && blockIdx.x == 0 && !dry) {
            // the choice's weights are of use to the last kernel only
#pragma unroll 1
            for (int tok = warp; tok < a.T; tok += kWarps) {
                const int id = lane < kTopK ? scratch.ids[tok * kTopK + lane] : 0;
                const float v = route_weight(lane < kTopK ? a.logits[tok * kExperts + id] : 0.0f);
                if (lane < kTopK) {
                    a.ids[tok * kTopK + lane] = id;
                    a.weights[tok * kTopK + lane] = v;
                }
            }
        }
    }
}

// out = sum over a token's pairs of scaling * weight * its share, in the order of k.  A thread takes four columns.  Its
// loads do not wait for one another: shares of pairs that are not here are read too (what the workspace holds there)
// and not taken.
__global__ void __launch_bounds__(kThreads) moe_sum_kernel(const ShareArgs a)
{
    const int pairs = a.T * kTopK, quads = a.H / 4;
    pdl_launch_dependents();
    pdl_wait();
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < a.T * quads; i += gridDim.x * kThreads) {
        const int tok = i / quads, col = (i - tok * quads) * 4;
        float4 v[kTopK];
        float c[kTopK];
        bool here[kTopK];
        const int passes = a.passes->count;
#pragma unroll
        for (int k = 0; k < kTopK; ++k) {
            v[k] = *reinterpret_cast<const float4 *>(a.sums + ((int64_t)tok * kTopK + k) * a.H + col);
            const int e = a.ids[tok * kTopK + k] - a.first;
            here[k] = e >= 0 && e < a.local;
            c[k] = a.scaling * a.weights[tok * kTopK + k];
        }
        const int parts = down_parts(a, passes);
#pragma unroll 1
        for (int p = 1; p < parts; ++p)
#pragma unroll
            for (int k = 0; k < kTopK; ++k)
                if (here[k]) {
                    const float4 y = *reinterpret_cast<const float4 *>(
                        a.sums + ((int64_t)p * pairs + tok * kTopK + k) * a.H + col);
                    v[k].x += y.x, v[k].y += y.y, v[k].z += y.z, v[k].w += y.w;
                }
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kTopK; ++k)
            if (here[k]) {
                sum.x = __fmaf_rn(c[k], v[k].x, sum.x);
                sum.y = __fmaf_rn(c[k], v[k].y, sum.y);
                sum.z = __fmaf_rn(c[k], v[k].z, sum.z);
                sum.w = __fmaf_rn(c[k], v[k].w, sum.w);
            }
        st_global_v2(a.out + tok * a.out_stride + col, pack_bf16x2(sum.x, sum.y),
                     pack_bf16x2(sum.z, sum.w));
    }
}

cudaError_t launch_share(const ShareArgs &s, int grid, cudaStream_t stream)
{
    constexpr int smem = kWarps * kStages * kStageBytes + kAreaBytes;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !done[dev])) {
        e = cudaFuncSetAttribute(moe_share_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && dev < 64)
            done[dev] = true;
    }
    return e == cudaSuccess
               ? launch_pdl(moe_share_kernel, dim3((unsigned)grid), dim3(kThreads), smem, stream, s)
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
    p.act = p.passes + (int64_t)(sizeof(DownPasses) + 15) / 16 * 16;
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
    s.passes = (DownPasses *)(a.workspace + p.passes);
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
    if (e == cudaSuccess) {
        s.cut = make_cut(a.H);
        e = launch_share(s, kSms, stream);
    }
    if (e == cudaSuccess) {
        s.cut = make_cut(a.F);
        s.down = true;
        e = launch_share(s, kSms, stream);
    }
    if (e == cudaSuccess) {
        const int64_t blocks = ((int64_t)a.T * (a.H / 4) + kThreads - 1) / kThreads;
        e = launch_pdl(moe_sum_kernel, dim3((unsigned)(blocks < 8 * kSms ? blocks : 8 * kSms)),
                       dim3(kThreads), 0, stream, s);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace beam
