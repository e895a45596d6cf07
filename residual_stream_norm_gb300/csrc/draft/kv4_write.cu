// kv4_write.cu -- keys and values into a cache held in 4 bits (sm_103a).
//
// A group of 32, 64 or 128 columns is held as codes 0..15 on the line minimum + scale * code.  Half a warp
// takes one row of a KV head: each lane 8 columns (16 bytes in, 4 bytes of codes out), the group's smallest
// and largest value by shuffles of a BF16 pair (minimum, -maximum) among its 4, 8 or 16 lanes.  For a prefill
// chunk the kernel is bound by its instructions rather than by memory (16,384 tokens of 8 heads 21 us, 67 MB read and 19
// written in 13 at the measured copy rate), so a half-warp's place in a token is worked out once, codes are rounded with
// packed FP32 additions, whose bits are packed with whole-number multiply-adds.

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

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// x / 15, rounded as by IEEE division: the rounded product with the rounded reciprocal, and Markstein's correction by
// the exact remainder (which is exact above 2^-100).
__device__ __forceinline__ float fifteenth(float x)
{
    constexpr float kInv = 0.06666667014360428f;  // RN(1 / 15)
    const float q = __fmul_rn(x, kInv);
    const float y = __fmaf_rn(__fmaf_rn(-q, 15.0f, x), kInv, q);
    return x < 7.888609052210118e-31f ? __fdiv_rn(x, 15.0f) : y;  // (infinite and NaN x: what it gives is not used)
}

// The codes rint(d / scale) of 8 values x of one group, d = x - lo, with the quotient of IEEE division: the rounded
// product with the rounded reciprocal, corrected by the exact remainder.  (A host test compares them for every FP32 mantissa of d
// and every BF16 mantissa of a scale.  A division where the product stands near a half instead, which values of eight bits often
// do exactly: 30 us for 16,384 tokens of 8 heads at that step, 24 this way; all by division 61.)
__device__ __forceinline__ uint32_t codes_of(const uint4 &v, float lo, float scale)
{
    // 1.5 2^23: a sum with it is rounded to a whole number, in the lowest bits
    constexpr float kMagic = 12582912.0f;
    constexpr uint32_t kMagicBits = 0x4b400000u;
    const float inv = __frcp_rn(scale);
    const f2 lo2 = splat(lo), inv2 = splat(inv), minus = splat(-scale), magic = splat(kMagic);
    uint32_t n[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f2 d = sub2(widen(word(v, i)), lo2), q = mul2(d, inv2);
        const f2 x = add2(fma2(fma2(q, minus, d), inv2, q), magic);
        n[2 * i] = __float_as_uint(lo_of(x));
        n[2 * i + 1] = __float_as_uint(hi_of(x));
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
                n[j] = j == i ? __float_as_uint(__fadd_rn(x, kMagic)) : n[j];
        }
    }
    // sum of 16^i n_i modulo 2^32, and what the upper bits add to it
    uint32_t w = n[7];
#pragma unroll
    for (int i = 6; i >= 0; --i)
        w = w * 16u + n[i];
    return w - kMagicBits * 0x11111111u;
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
    const uint32_t step = gridDim.x * (uint32_t)at_once, T = (uint32_t)a.T;  // T < 2^31: two steps behind it is in 32 bits
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
        int64_t next_slot;
        int slot = -1;  // -1: not written
        uint4 next = make_uint4(0, 0, 0, 0);
        uint32_t t0 = blockIdx.x * (uint32_t)at_once;
        const uint16_t *row = src + (t0 + tt) * stride;
        const int64_t row_step = step * stride;
        auto load_slot = [&](uint32_t t) { next_slot = on && t < T ? a.slot[t] : -1; };
        auto load_row = [&]() {
            slot = (uint64_t)next_slot < (uint64_t)a.num_slots ? (int)next_slot : -1;
            if (slot >= 0)
                next = ld_stream(row);
            row += row_step;
        };
        load_slot(t0 + tt);
        load_row();
        load_slot(t0 + step + tt);
        for (; t0 < T; t0 += step) {
            const uint4 v = next;
            const int at = slot;
            load_row();
            load_slot(t0 + 2 * step + tt);
            constexpr uint32_t kSign = 0x80008000u;
            const uint32_t lo2 = min_nan_bf16x2(min_nan_bf16x2(v.x, v.y),
                                                min_nan_bf16x2(v.z, v.w));
            const uint32_t hi2 = max_nan_bf16x2(max_nan_bf16x2(v.x, v.y),
                                                max_nan_bf16x2(v.z, v.w)) ^ kSign;
            // (minimum, -maximum)
            uint32_t ends = min_nan_bf16x2(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
#pragma unroll
            for (int off = 1; off < kLanes; off <<= 1)
                ends = min_nan_bf16x2(ends, __shfl_xor_sync(0xffffffffu, ends, off));
            const float lo = bf_lo(ends);
            const float span = -__fadd_rn(bf_hi(ends), lo);  // NaN or infinite: as the values are
            const uint32_t held = pack_bf16x2(fifteenth(span), lo);
            const float scale = bf_lo(held);
            const bool bad = !isfinite(span);  // as it is for an infinite minimum
            const uint32_t code = bad || !(scale > 0.0f) ? 0u : codes_of(v, lo, scale);
            if (at >= 0) {
                codes[(uint64_t)(uint32_t)at * (uint32_t)(a.n_kv * 16)] = code;
                if (lane % kLanes == 0)
                    scales[(uint64_t)(uint32_t)at * (uint32_t)(a.n_kv * kGroups)] = bad ? 0x7fc0u : held;
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4WriteArgs &a, cudaStream_t stream)
{
    const int at_once = 2 * a.n_kv < kHalves ? kHalves / (2 * a.n_kv) : 1;
    const int64_t blocks = (a.T + at_once - 1) / at_once;
    // as many blocks as fit (four an SM at 63 registers): 21.0 us for 16,384 tokens, with twice as many 21.8
    const unsigned grid = (unsigned)(blocks < 152 * 4 ? blocks : 152 * 4);
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
