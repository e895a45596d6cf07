// kv_evict.cu -- eviction from the slot cache by accumulated attention weight (sm_103a).
//
// The k-th largest weight of a row is found by radix selection on order-preserving integer keys: four
// passes of eight bits, each a histogram of the keys that still match.  One ordered pass then moves
// what stays to the row's front and lists what leaves.

#include "decode_kernels.h"
#include "decode_mma.cuh"

namespace beam {
namespace {

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;

// Order-preserving key: larger weights, larger keys; -0 as +0; NaN below every number.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w)
        return 0u;
    const uint32_t u = w == 0.0f ? 0u : __float_as_uint(w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kEvictThreads) kv_evict_kernel(const EvictArgs a)
{
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_prefix, s_want;
    __shared__ int s_cnt[2][kEvictWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        int64_t n = a.len_in[row];
        n = n < 0 ? 0 : (n > a.width ? a.width : n);
        const float *win = a.weight_in + row * a.width;
        const int64_t *tin = a.table_in + row * a.width;
        float *wout = a.weight_out + row * a.width;
        int64_t *tout = a.table_out + row * a.width;
        int64_t *freed = a.freed_out + row * a.freed_width;
        const bool over = n > a.budget;
        const int64_t old = over ? n - a.recent : 0;  // entries that compete
        const int64_t keep = over ? a.budget - a.recent : 0;
        // ---- the smallest key that stays, and how many of the entries that have it -----------------
        uint32_t thr = 0xffffffffu, ties = 0;
        if (keep > 0) {
            if (tid == 0) {
                s_prefix = 0;
                s_want = (uint32_t)keep;
            }
            for (int shift = 24; shift >= 0; shift -= 8) {
                if (tid < 256)
                    hist[tid] = 0;
                __syncthreads();
                const uint32_t prefix = s_prefix;
                for (int64_t j = tid; j < old; j += kEvictThreads) {
                    const uint32_t k = weight_key(win[j]);
                    if (shift == 24 || (k >> (shift + 8)) == prefix)
                        atomicAdd(&hist[(k >> shift) & 255u], 1u);
                }
                __syncthreads();
                if (tid == 0) {
                    uint32_t want = s_want;
                    int d = 255;
                    while (hist[d] < want)
                        want -= hist[d--];
                    s_want = want;
                    s_prefix = (prefix << 8) | (uint32_t)d;
                }
                __syncthreads();
            }
            thr = s_prefix;
            ties = s_want;
        }
        // ---- move ----------------------------------------------------------------------------------
        int64_t kept_before = 0, eq_before = 0;
        for (int64_t base = 0; base < n; base += kEvictThreads) {
            const int64_t j = base + tid;
            const bool in = j < n;
            const float w = in ? win[j] : 0.0f;
            const int64_t slot = in ? tin[j] : -1;
            const uint32_t k = weight_key(w);
            const bool compete = in && j < old;
            const bool eq = compete && keep > 0 && k == thr;
            const uint32_t eqb = __ballot_sync(0xffffffffu, eq);
            if (lane == 0)
                s_cnt[0][warp] = __popc(eqb);
            __syncthreads();
            int before = 0, all = 0;
            for (int x = 0; x < kEvictWarps; ++x) {
                before += x < warp ? s_cnt[0][x] : 0;
                all += s_cnt[0][x];
            }
            const int64_t eq_rank = eq_before + before + __popc(eqb & ((1u << lane) - 1u));
            const bool stay =
                in && (!compete || (keep > 0 && (k > thr || (eq && eq_rank < (int64_t)ties))));
            eq_before += all;
            const uint32_t sb = __ballot_sync(0xffffffffu, stay);
            if (lane == 0)
                s_cnt[1][warp] = __popc(sb);
            __syncthreads();
            before = all = 0;
            for (int x = 0; x < kEvictWarps; ++x) {
                before += x < warp ? s_cnt[1][x] : 0;
                all += s_cnt[1][x];
            }
            const int64_t to = kept_before + before + __popc(sb & ((1u << lane) - 1u));
            if (stay) {
                wout[to] = w;
                tout[to] = slot;
            } else if (in) {
                freed[j - to] = slot;
            }
            kept_before += all;
            __syncthreads();
        }
        for (int64_t j = kept_before + tid; j < a.width; j += kEvictThreads) {
            wout[j] = 0.0f;
            tout[j] = -1;
        }
        for (int64_t j = n - kept_before + tid; j < a.freed_width; j += kEvictThreads)
            freed[j] = -1;
        if (tid == 0)
            a.len_out[row] = (int32_t)kept_before;
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs &a, cudaStream_t stream)
{
    const unsigned grid = (unsigned)(a.rows < (1 << 20) ? a.rows : (1 << 20));
    const cudaError_t e =
        launch_pdl(kv_evict_kernel, dim3(grid), dim3(kEvictThreads), 0, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace beam
