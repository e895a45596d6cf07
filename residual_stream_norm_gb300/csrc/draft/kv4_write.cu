// kv4_write.cu -- keys and values into a cache held in 4 bits (sm_103a).
//
// A group of 32, 64 or 128 columns is held as codes 0..15 on the line minimum + scale * code.  Half a warp
// takes one row of a KV head: each lane 8 columns (16 bytes in, 4 bytes of codes out), the group's smallest
// and largest value by shuffles among its 4, 8 or 16 lanes.

#include "beam_device.cuh"
#include "draft_kernels.h"

namespace beam {
namespace {

constexpr int kThreads = 256;

template <int Group>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const Kv4WriteArgs a)
{
    constexpr int kLanes = Group / 8;   // lanes of a group
    constexpr int kGroups = 128 / Group;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 15;
    const int64_t rows = a.T * 2 * a.n_kv;  // of a token: its K heads, then its V heads
    const int64_t step = (int64_t)gridDim.x * (kThreads / 16);
    const uint32_t per = 2 * a.n_kv;
    // both halves of a warp take part in every shuffle: the loop runs for as long as either has a row
    for (int64_t r = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
         (r & ~(int64_t)1) < rows; r += step) {
        const int64_t t = r < rows ? r / per : 0;
        const int j = (int)(r - t * per);
        const int which = j >= a.n_kv;
        const int head = which ? j - a.n_kv : j;
        const int64_t slot = r < rows ? a.slot[t] : -1;
        const bool on = slot >= 0 && slot < a.num_slots;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (on)
            v = ld_stream((const uint16_t *)(which ? a.src[1] : a.src[0]) +
                          t * (which ? a.src_stride[1] : a.src_stride[0]) + head * 128 + lane * 8);
        float x[8];
        float lo = __uint_as_float(0x7f800000u), hi = -lo;
        bool finite = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf_lo(word(v, i));
            x[2 * i + 1] = bf_hi(word(v, i));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, x[i]);
            hi = fmaxf(hi, x[i]);
            finite = finite && isfinite(x[i]);
        }
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
            finite = __shfl_xor_sync(0xffffffffu, (int)finite, off) && finite;
        }
        const float span = __fsub_rn(hi, lo);
        const uint32_t held = pack_bf16x2(__fdiv_rn(span, 15.0f), lo);
        float scale = bf_lo(held);
        const bool bad = !finite || !isfinite(span);
        const bool flat = bad || !(scale > 0.0f);
        if (flat)
            scale = 1.0f;
        uint32_t code = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = fminf(rintf(__fdiv_rn(__fsub_rn(x[i], lo), scale)), 15.0f);
            code |= (flat ? 0u : (uint32_t)q) << (4 * i);
        }
        if (on) {
            const int64_t row = slot * a.n_kv + head;
            reinterpret_cast<uint32_t *>((which ? a.cache[1] : a.cache[0]) + row * 64)[lane] = code;
            if (lane % kLanes == 0)
                reinterpret_cast<uint32_t *>(which ? a.scales[1]
                                                     : a.scales[0])[row * kGroups + lane / kLanes] =
                    bad ? 0x7fc0u : held;
        }
    }
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4WriteArgs &a, cudaStream_t stream)
{
    const int64_t rows = a.T * 2 * a.n_kv;
    const int64_t blocks = (rows + kThreads / 16 - 1) / (kThreads / 16);
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
