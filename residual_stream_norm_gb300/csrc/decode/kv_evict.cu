// kv_evict.cu -- eviction from the slot cache by accumulated attention weight (sm_103a).
//
// The smallest weight that stays is found by radix selection on order-preserving integer keys: digits
// of 11, 11 and 10 bits from the top, each a histogram of the keys that still match, until what is left
// of the row is decided.  One ordered pass then moves what stays to the row's front and lists what
// leaves.  A block reads its weights once, into shared memory.
//
// What bounds it: 72 rows of ~100K entries take 57 us (3.1 TB/s; floor 26 us): a block reads,
// selects and moves one after the other, so memory waits while it selects.  In the histogram passes
// instructions count: a warp vote before the atomics took 81 us, joining equal digits 93, zeros counted
// apart and plain atomics 57.  One row of 2K takes 7.1 us: one block, barrier after barrier.
//
// One block a row; a cluster shares out long rows when there are few (histograms and counts meet in
// distributed shared memory).  Each warp counts what stays of a stretch of its own, and from the sums
// in front of it moves that stretch by itself.  A row that is compacted in place takes one block and
// goes in rounds instead, all of a round's reads before its writes: a stretch's front end is moved
// into the back of the stretch before it.

#include "decode_kernels.h"
#include "decode_mma.cuh"

namespace beam {
namespace {

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kBins = 2048;
constexpr int kPerThread = 4;                         // entries of a round, in place
constexpr int kRound = kPerThread * kEvictThreads;
constexpr int kList = 4096;                           // keys that the last digits are looked up in
constexpr int kMostCached = 50 * 1024;                // weights in shared memory

constexpr uint32_t kZeroKey = 0x80000000u;

// Counts of a round's warps, read four at a time.
struct alignas(16) WarpCounts {
    uint32_t of[kPerThread * kEvictWarps];
};
static_assert(alignof(WarpCounts) >= alignof(uint4) && sizeof(WarpCounts) == 4 * 32 * sizeof(uint32_t),
              "four counts a lane");

// Order-preserving key: larger weights, larger keys; -0 as +0; NaN below every number.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w)
        return 0u;
    const uint32_t u = w == 0.0f ? 0u : __float_as_uint(w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

// A word of another block of the cluster, at this block's shared address.
__device__ __forceinline__ uint32_t ld_cluster(const void *p, int rank)
{
    uint32_t v;
    asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
                 "ld.shared::cluster.u32 %0, [a];\n\t}"
                 : "=r"(v)
                 : "r"(smem_addr(p)), "r"(rank)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint2 ld_cluster2(const void *p, int rank)
{
    uint2 v;
    asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\t"
                 "ld.shared::cluster.v2.u32 {%0, %1}, [a];\n\t}"
                 : "=r"(v.x), "=r"(v.y)
                 : "r"(smem_addr(p)), "r"(rank)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane)  // inclusive
{
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, v, off);
        v += lane >= off ? o : 0u;
    }
    return v;
}

template <bool IN_PLACE>
__global__ void __launch_bounds__(kEvictThreads) kv_evict_kernel(const EvictArgs a, int split,
                                                                 int cached)
{
    extern __shared__ float s_weight[];  // [cached]
    __shared__ __align__(8) uint32_t s_hist[kBins];
    __shared__ uint32_t s_list[kList];
    __shared__ WarpCounts s_warp[2];
    __shared__ uint32_t s_pick[3];       // digit, still wanted of it, whether all of it stays
    __shared__ uint32_t s_count[2];      // of this block's entries: above the smallest, equal to it
    __shared__ uint32_t s_listed, s_zeros;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x % split;
    const int64_t row = blockIdx.x / split;
    pdl_launch_dependents();
    pdl_wait();
    int64_t n64 = a.len_in[row];
    n64 = n64 < 0 ? 0 : (n64 > a.width ? a.width : n64);
    const int n = (int)n64;
    const float *win = a.weight_in + row * a.width;
    const int64_t *tin = a.table_in + row * a.width;
    float *wout = a.weight_out + row * a.width;
    int64_t *tout = a.table_out + row * a.width;
    int64_t *freed = a.freed_out + row * a.freed_width;
    const bool over = n > a.budget;
    const int old = over ? n - (int)a.recent : 0;                   // entries that compete
    const int keep = over ? (int)(a.budget - a.recent) : 0;         // and how many of them stay
    const int per = (n + split - 1) / split;
    const int begin = min(n, rank * per), end = min(n, begin + per);  // this block's entries
    const int in_smem = min(end - begin, cached);
    const int compete = max(0, min(end, old) - begin);              // of them, the first ones
    // In place all weights that fit come first: a round's may be overwritten by the one before it.
    const int have = IN_PLACE || keep > 0 ? in_smem : 0;
    auto weight = [&](int j) { return j < have ? s_weight[j] : win[begin + j]; };

    // ---- the key above which all stay, and how many of those equal to it -------------------------------
    uint32_t thr = 0xffffffffu, ties = 0;
    if (keep > 0) {
        uint32_t prefix = 0, want = (uint32_t)keep;
        int shift = 32;
        bool listed = false;  // the keys that still match are in s_list
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int bits = pass < 2 ? 11 : 10;
            for (int i = tid; i < kBins; i += kEvictThreads)
                s_hist[i] = 0;
            if (tid == 0 && pass == 0)
                s_listed = s_zeros = 0;
            __syncthreads();
            const int above = shift;
            shift -= bits;
            const uint32_t digits = (1u << bits) - 1u;
            if (pass == 0) {
                // the weights arrive here; zeros, often many, are counted apart
                uint32_t zeros = 0;
#pragma unroll 1
                for (int j0 = tid; j0 < in_smem; j0 += 8 * kEvictThreads) {
                    float w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int j = j0 + k * kEvictThreads;
                        w[k] = j < in_smem ? win[begin + j] : 0.0f;
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int j = j0 + k * kEvictThreads;
                        if (j < in_smem)
                            s_weight[j] = w[k];
                        if (j < compete) {
                            if (w[k] == 0.0f)
                                ++zeros;
                            else
                                atomicAdd(&s_hist[weight_key(w[k]) >> 21], 1u);
                        }
                    }
                }
                for (int j = in_smem + tid; j < compete; j += kEvictThreads) {
                    const float w = win[begin + j];
                    if (w == 0.0f)
                        ++zeros;
                    else
                        atomicAdd(&s_hist[weight_key(w) >> 21], 1u);
                }
                zeros = __reduce_add_sync(0xffffffffu, zeros);
                if (lane == 0 && zeros) {
                    atomicAdd(&s_zeros, zeros);
                    atomicAdd(&s_hist[kZeroKey >> 21], zeros);
                }
            } else if (!listed) {
                // pass 1 keeps the keys that match the first digit, if they fit
                if (tid == 0 && kZeroKey >> above == prefix)
                    atomicAdd(&s_hist[(kZeroKey >> shift) & digits], s_zeros);
                const float *from = compete <= have ? s_weight : win + begin;
#pragma unroll 4
                for (int j = tid; j < compete; j += kEvictThreads) {
                    const uint32_t k = weight_key(from[j]);
                    if (k >> above == prefix && k != kZeroKey) {
                        atomicAdd(&s_hist[(k >> shift) & digits], 1u);
                        if (pass == 1) {
                            const uint32_t at = atomicAdd(&s_listed, 1u);
                            if (at < kList)
                                s_list[at] = k;
                        }
                    }
                }
            } else {
                if (tid == 0 && kZeroKey >> above == prefix)
                    atomicAdd(&s_hist[(kZeroKey >> shift) & digits], s_zeros);
                const int m = (int)s_listed;
                for (int j = tid; j < m; j += kEvictThreads) {
                    const uint32_t k = s_list[j];
                    if (k >> above == prefix)
                        atomicAdd(&s_hist[(k >> shift) & digits], 1u);
                }
            }
            __syncthreads();
            listed = pass == 1 && s_listed <= kList;
            uint32_t h[2];  // the bins from the top: 2047 - 2 tid, 2046 - 2 tid
            h[0] = s_hist[kBins - 1 - 2 * tid];
            h[1] = s_hist[kBins - 2 - 2 * tid];
            if (split > 1) {
                cluster_sync();
                h[0] = h[1] = 0;
                for (int q = 0; q < split; ++q) {
                    const uint2 v = ld_cluster2(&s_hist[kBins - 2 - 2 * tid], q);
                    h[0] += v.y;
                    h[1] += v.x;
                }
            }
            const uint32_t inc = warp_scan(h[0] + h[1], lane);
            if (lane == 31)
                s_warp[0].of[warp] = inc;
            __syncthreads();
            const uint32_t w = warp_scan(s_warp[0].of[lane], lane);
            const uint32_t before =
                (warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0u) + inc - h[0] - h[1];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t b = before + (i ? h[0] : 0u);
                if (b < want && want <= b + h[i]) {
                    s_pick[0] = kBins - 1 - 2 * tid - i;
                    s_pick[1] = want - b;
                    s_pick[2] = want - b == h[i];
                }
            }
            __syncthreads();
            prefix = (prefix << bits) | s_pick[0];
            want = s_pick[1];
            const bool decided = s_pick[2] != 0;
            if (split > 1)
                cluster_sync();  // the others have read this block's histogram
            if (decided && pass < 2) {  // all of the digit stays: everything from its first key on
                thr = (prefix << shift) - 1u;
                want = 0;
                break;
            }
            thr = prefix;
        }
        ties = want;
    } else if (IN_PLACE) {
        for (int j = tid; j < in_smem; j += kEvictThreads)
            s_weight[j] = win[begin + j];
    }
    const int64_t m = over ? a.budget : n;
    uint32_t gt_before = 0, eq_before = 0;  // of the competing entries in front
    if constexpr (!IN_PLACE) {
        // ---- each warp's stretch: count, sums in front, move ---------------------------------------
        const int len = ((end - begin + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
        const int s0 = min(end - begin, warp * len), s1 = min(end - begin, s0 + len);
        const float *from = s1 <= have ? s_weight : win + begin;
        if (keep > 0) {
            uint32_t gt = 0, eq = 0;
            const int c1 = min(s1, compete);
#pragma unroll 4
            for (int j = s0 + lane; j < c1; j += 32) {
                const uint32_t k = weight_key(from[j]);
                gt += k > thr;
                eq += k == thr;
            }
            gt = __reduce_add_sync(0xffffffffu, gt);
            eq = __reduce_add_sync(0xffffffffu, eq);
            __syncthreads();  // s_warp is free
            if (lane == 0) {
                s_warp[0].of[warp] = gt;
                s_warp[1].of[warp] = eq;
            }
            __syncthreads();
            const uint32_t g = warp_scan(s_warp[0].of[lane], lane);
            const uint32_t e = warp_scan(s_warp[1].of[lane], lane);
            gt_before = warp > 0 ? __shfl_sync(0xffffffffu, g, warp - 1) : 0u;
            eq_before = warp > 0 ? __shfl_sync(0xffffffffu, e, warp - 1) : 0u;
            if (split > 1) {
                if (tid == 31) {
                    s_count[0] = g;
                    s_count[1] = e;
                }
                cluster_sync();
                for (int q = 0; q < rank; ++q) {
                    gt_before += ld_cluster(&s_count[0], q);
                    eq_before += ld_cluster(&s_count[1], q);
                }
                cluster_sync();
            }
        }
        constexpr int kAhead = 4;
        const uint32_t low = (1u << lane) - 1u;
        int64_t slot[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int j = s0 + 32 * k + lane;
            slot[k] = j < s1 ? tin[begin + j] : -1;
        }
        for (int base = s0; base < s1; base += 32 * kAhead) {
            float w[kAhead];
            int64_t next[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int j = base + 32 * k + lane, jn = j + 32 * kAhead;
                w[k] = j < s1 ? from[j] : 0.0f;
                next[k] = jn < s1 ? tin[begin + jn] : -1;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int j = base + 32 * k + lane;
                const uint32_t key = weight_key(w[k]);
                const bool c = j < compete && keep > 0;
                const uint32_t above = __ballot_sync(0xffffffffu, c && key > thr);
                const uint32_t equal = __ballot_sync(0xffffffffu, c && key == thr);
                const uint32_t gt = gt_before + __popc(above & low);
                const uint32_t eq = eq_before + __popc(equal & low);
                if (j < s1) {
                    const int at = begin + j;
                    const bool stay =
                        at >= old || (c && (key > thr || (key == thr && eq < ties)));
                    // entries in front that stay
                    const int to = at >= old ? at - old + keep : (int)(gt + min(eq, ties));
                    if (stay) {
                        wout[to] = w[k];
                        tout[to] = slot[k];
                    } else {
                        freed[at - to] = slot[k];
                    }
                }
                gt_before += __popc(above);
                eq_before += __popc(equal);
                slot[k] = next[k];
            }
        }
    } else {
    __syncthreads();
    // ---- move: rounds in order; a round's reads are complete before its writes ---------------------------
    int64_t slot[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int j = begin + k * kEvictThreads + tid;
        slot[k] = j < end ? tin[j] : -1;
    }
    for (int base = begin, round = 0; base < end; base += kRound, round ^= 1) {
        float w[kPerThread];
        int64_t next[kPerThread];
        uint32_t above[kPerThread], equal[kPerThread];
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) {
            const int j = base + k * kEvictThreads + tid;
            w[k] = j < end ? weight(j - begin) : 0.0f;
            const int jn = j + kRound;
            next[k] = jn < end ? tin[jn] : -1;
            const uint32_t key = weight_key(w[k]);
            const bool c = j < old && j < end && keep > 0;
            above[k] = __ballot_sync(0xffffffffu, c && key > thr);
            equal[k] = __ballot_sync(0xffffffffu, c && key == thr);
            if (lane == 0)
                s_warp[round].of[k * kEvictWarps + warp] =
                    (uint32_t)__popc(above[k]) | (uint32_t)__popc(equal[k]) << 16;
        }
        __syncthreads();
        // running counts over the 128 (k, warp): four a lane
        const uint4 c4 = *reinterpret_cast<const uint4 *>(&s_warp[round].of[4 * lane]);
        const uint32_t sum = c4.x + c4.y + c4.z + c4.w, inc = warp_scan(sum, lane);
        const uint32_t all = __shfl_sync(0xffffffffu, inc, 31);
        uint32_t mine = inc - sum;  // exclusive, at this warp's place among the lane's four
        mine += (warp & 3) > 0 ? c4.x : 0u;
        mine += (warp & 3) > 1 ? c4.y : 0u;
        mine += (warp & 3) > 2 ? c4.z : 0u;
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) {
            const int j = base + k * kEvictThreads + tid;
            const uint32_t front = __shfl_sync(0xffffffffu, mine, 8 * k + warp / 4);
            const uint32_t low = (1u << lane) - 1u;
            const uint32_t gt = gt_before + (front & 0xffffu) + __popc(above[k] & low);
            const uint32_t eq = eq_before + (front >> 16) + __popc(equal[k] & low);
            if (j < end) {
                const bool is_gt = (above[k] >> lane) & 1u, is_eq = (equal[k] >> lane) & 1u;
                const bool stay = j >= old || is_gt || (is_eq && eq < ties);
                // entries in front that stay
                const int to = j >= old ? (over ? keep + j - old : j) : (int)(gt + min(eq, ties));
                if (stay) {
                    wout[to] = w[k];
                    tout[to] = slot[k];
                } else {
                    freed[j - to] = slot[k];
                }
            }
            slot[k] = next[k];
        }
        gt_before += all & 0xffffu;
        eq_before += all >> 16;
    }
    }
    // ---- behind what stays -------------------------------------------------------------------------
    const int64_t stride = (int64_t)split * kEvictThreads;
    __syncthreads();  // in place: the others' reads are complete
    for (int64_t j = m + rank * kEvictThreads + tid; j < a.width; j += stride) {
        wout[j] = 0.0f;
        tout[j] = -1;
    }
    for (int64_t j = n - m + rank * kEvictThreads + tid; j < a.freed_width; j += stride)
        freed[j] = -1;
    if (tid == 0 && rank == 0)
        a.len_out[row] = (int32_t)m;
}

// How many clusters of `split` blocks the device holds at a time (a cluster stays within one of its groups
// of SMs, so fewer than the SMs would give); the same for all calls.
int resident_clusters(int split)
{
    static int known[64][4] = {};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 0;
    int *at = dev < 64 ? &known[dev][split / 4] : nullptr;
    if (at && *at)
        return *at;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = kMostCached * 4;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)split;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kv_evict_kernel<false>, &cfg) != cudaSuccess)
        return 0;
    if (at)
        *at = n;
    return n;
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs &a, cudaStream_t stream)
{
    const bool in_place = (a.width > 0) && (a.table_in == a.table_out || a.weight_in == a.weight_out ||
                                            a.len_in == a.len_out);
    cudaError_t e = in_place ? allow_smem<kv_evict_kernel<true>>(kMostCached * 4)
                             : allow_smem<kv_evict_kernel<false>>(kMostCached * 4);
    if (e != cudaSuccess)
        return e;
    // Blocks of a cluster per row, as many as make long rows shorter, while all rows' clusters are resident at
    // once.  1, 2, 4 and 8 blocks for 8 rows, us: of 9K 11.9, 12.8, 13.0, 17.6; of 12.5K 14.1, 13.5, 13.6, 17.9; of
    // 16K 15.4, 14.5, 14.0, 18.3; of 80K 63, 33, 23.5, 23.2; of 200K 150, 85, 41, 32.  More clusters than fit
    // take a second round: 15 and 16 rows of 100K in eights 25.5 and 47 (in fours 27), 36 and 37 in fours 29.5 and
    // 54 (in pairs 45), 76 and 77 rows of 40K in pairs 22.7 and 42 (single blocks 31).
    int split = 1;
    if (!in_place) {
        constexpr struct {
            int split, width;
        } kinds[] = {{8, 81920}, {4, 16384}, {2, 12288}};
        for (const auto &k : kinds)
            if (split == 1 && a.width >= k.width && a.rows <= resident_clusters(k.split))
                split = k.split;
    }
    const int64_t per = (a.width + split - 1) / split;
    const int cached = (int)(per < kMostCached ? per : kMostCached);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = (size_t)cached * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    // at most 2^30 blocks a launch
    const int64_t most = ((int64_t)1 << 30) / split;
    for (int64_t r = 0; r < a.rows; r += most) {
        EvictArgs b = a;
        b.rows = a.rows - r < most ? a.rows - r : most;
        b.table_out = a.table_out + r * a.width;
        b.table_in = a.table_in + r * a.width;
        b.weight_out = a.weight_out + r * a.width;
        b.weight_in = a.weight_in + r * a.width;
        b.freed_out = a.freed_out + r * a.freed_width;
        b.len_in = a.len_in + r;
        b.len_out = a.len_out + r;
        cfg.gridDim = dim3((unsigned)(b.rows * split));
        e = cudaLaunchKernelEx(&cfg, in_place ? kv_evict_kernel<true> : kv_evict_kernel<false>, b,
                               split, cached);
        if (e != cudaSuccess)
            return e;
    }
    return cudaGetLastError();
}

}  // namespace beam
