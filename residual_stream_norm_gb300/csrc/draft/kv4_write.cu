// kv4_write.cu -- keys and values into a cache held in 4 bits (sm_103a).
//
// A group of 32, 64 or 128 columns is held as codes 0..15 on the line minimum + scale * code.  Half a warp
// takes one row of a KV head: each lane 8 columns (16 bytes in, 4 bytes of codes out), the group's smallest
// and largest value by shuffles of a BF16 pair (minimum, -maximum) among its 4, 8 or 16 lanes.  For a prefill
// chunk the kernel is bound by its instructions rather than by memory, so a half-warp's place in a token is worked out
// once, and codes are rounded and packed with FP32 additions and fused multiply-adds.

#include "beam_device.cuh"
#include "beam_f32x2.cuh"
#include "draft_kernels.h"

namespace beam {
namespace {

constexpr int kThreads = 256;
constexpr int kHalves = kThreads / 16;

__device__ __forceinline__ uint32_t min_nan_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// x / 15, rounded as by IEEE division: the rounded product with the rounded reciprocal, and Markstein's correction by
// the exact remainder (which is exact above 2^-100).
__device__ __forceinline__ float fifteenth(float x)
{
    constexpr float kInv = 0.06666667014360428f;  // RN(1 / 15)
    const float q = __fmul_rn(x, kInv);
    const float y = __fmaf_rn(__fmaf_rn(-q, 15.0f, x), kInv, q);
    return x < 7.888609052210118e-31f || x > 1.0e38f ? __fdiv_rn(x, 15.0f) : y;
}

// The codes rint(d / scale) of 8 values x of one group, d = x - lo, with the quotient of IEEE division: the rounded
// product with the rounded reciprocal, corrected by the exact remainder.  (Tried for every FP32 mantissa of d and every
// BF16 mantissa of a scale.  A division where the product stands near a half instead, which values of eight bits often
// do exactly: 30 us for 16,384 tokens of 8 heads, 24 this way; all by division 61.)
__device__ __forceinline__ uint32_t codes_of(const uint4 &v, float lo, float scale)
{
    constexpr float kMagic = 12582912.0f;  // 1.5 2^23: a sum with it is rounded to a whole number
    const float inv = __frcp_rn(scale);
    const f2 lo2 = splat(lo), inv2 = splat(inv), minus = splat(-scale), magic = splat(kMagic);
    float n[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f2 d = sub2(widen(word(v, i)), lo2), q = mul2(d, inv2);
        const f2 x = sub2(add2(fma2(fma2(q, minus, d), inv2, q), magic), magic);
        n[2 * i] = lo_of(x);
        n[2 * i + 1] = hi_of(x);
    }
    // where a remainder would not be exact; there a scale may also be far from span / 15
    if (scale < 7.888609052210118e-31f) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const uint32_t w = i < 4 ? (i < 2 ? v.x : v.y) : (i < 6 ? v.z : v.w);
            const float d = __fsub_rn(i & 1 ? bf_hi(w) : bf_lo(w), lo);
            const float x = fminf(rintf(__fdiv_rn(d, scale)), 15.0f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                n[j] = j == i ? x : n[j];
        }
    }
    // four codes a number below 2^16: exact
    const float a = __fmaf_rn(__fmaf_rn(__fmaf_rn(n[3], 16.0f, n[2]), 16.0f, n[1]), 16.0f, n[0]);
    const float b = __fmaf_rn(__fmaf_rn(__fmaf_rn(n[7], 16.0f, n[6]), 16.0f, n[5]), 16.0f, n[4]);
    return __byte_perm(__float_as_uint(__fadd_rn(a, kMagic)), __float_as_uint(__fadd_rn(b, kMagic)),
                       0x5410);
}

template <int Group>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const Kv4WriteArgs a)
{
    constexpr int kLanes = Group / 8;   // lanes of a group
    constexpr int kGroups = 128 / Group;
    pdl_launch_dependents();
    const int lane = threadIdx.x & 15, half = threadIdx.x >> 4;
    const int per = 2 * a.n_kv;                          // rows of a token: its K heads, then its V heads
    const int at_once = per < kHalves ? kHalves / per : 1;  // tokens of a block
    const int tt = per < kHalves ? half / per : 0;
    const int64_t step = (int64_t)gridDim.x * at_once;
    pdl_wait();
    // every bound is the same for both halves of a warp, or a half without a row goes along: shuffles are the warp's
    for (int j0 = 0; j0 < per; j0 += kHalves) {
        const int j = per < kHalves ? half - tt * per : j0 + half;
        const bool on = j < per && tt < at_once;
        const bool value = j >= a.n_kv;
        const int head = value ? j - a.n_kv : j;
        const uint16_t *src = (const uint16_t *)(value ? a.src[1] : a.src[0]) + head * 128 + lane * 8;
        const int64_t stride = value ? a.src_stride[1] : a.src_stride[0];
        uint32_t *codes = reinterpret_cast<uint32_t *>(value ? a.cache[1] : a.cache[0]) + head * 16 + lane;
        uint32_t *scales = reinterpret_cast<uint32_t *>(value ? a.scales[1] : a.scales[0]) +
                           head * kGroups + lane / kLanes;
        // the row after this one, and the slot after that, are on their way
        int64_t slot = -1, next_slot;
        uint4 next = make_uint4(0, 0, 0, 0);
        auto load_slot = [&](int64_t t) { next_slot = on && t < a.T ? a.slot[t] : -1; };
        auto load_row = [&](int64_t t) {
            slot = next_slot < a.num_slots ? next_slot : -1;
            if (slot >= 0)
                next = ld_stream(src + t * stride);
        };
        int64_t t0 = (int64_t)blockIdx.x * at_once;
        load_slot(t0 + tt);
        load_row(t0 + tt);
        load_slot(t0 + step + tt);
        for (; t0 < a.T; t0 += step) {
            const uint4 v = next;
            const int64_t at = slot;
            load_row(t0 + step + tt);
            load_slot(t0 + 2 * step + tt);
            constexpr uint32_t kSign = 0x80008000u;
            const uint32_t lo2 = min_nan_bf16x2(min_nan_bf16x2(v.x, v.y),
                                                min_nan_bf16x2(v.z, v.w));
            const uint32_t hi2 = min_nan_bf16x2(
                min_nan_bf16x2(v.x ^ kSign, v.y ^ kSign),
                min_nan_bf16x2(v.z ^ kSign, v.w ^ kSign));
            // (minimum, -maximum)
            uint32_t ends = min_nan_bf16x2(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
#pragma unroll
            for (int off = 1; off < kLanes; off <<= 1)
                ends = min_nan_bf16x2(ends, __shfl_xor_sync(0xffffffffu, ends, off));
            const float lo = bf_lo(ends);
            const float span = -__fadd_rn(bf_hi(ends), lo);  // NaN or infinite: as the values are
            const uint32_t held = pack_bf16x2(fifteenth(span), lo);
            const float scale = bf_lo(held);
            const bool bad = !isfinite(span) || !isfinite(lo);
            const uint32_t code = bad || !(scale > 0.0f) ? 0u : codes_of(v, lo, scale);
            if (at >= 0) {
                codes[at * a.n_kv * 16] = code;
                if (lane % kLanes == 0)
                    scales[at * a.n_kv * kGroups] = bad ? 0x7fc0u : held;
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4WriteArgs &a, cudaStream_t stream)
{
    const int at_once = 2 * a.n_kv < kHalves ? kHalves / (2 * a.n_kv) : 1;
    const int64_t blocks = (a.T + at_once - 1) / at_once;
    const unsigned grid = (unsigned)(blocks < 152 * 8 ? blocks : 152 * 8);
    cudaError_t e;
    if (a.group == 32)
        e = launch_pdl(kv4_write_kernel<32>, dim3(grid), dim3(kThreads), 0, stream, a);
    else if (a.group == 64)
        e = launch_pdl(kv4_write_kernel<64>, dim3(grid), dim3(kThreads), 0, stream, a);
    else
        e = launch_pdl(kv4_write_kernel<128>, dim3(grid), dim3(kThreads), 0, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace beam
