// w4_matvec.cu -- products of a few tokens with a matrix of 4-bit weights (sm_103a).
//
// y[t, n] = sum_g scale[n, g] * ( sum_{k in g} x[t, k] (w[n, k] - z[n, g]) ).  w - z is a whole number of
// at most five bits, exact in BF16, so the inner sum is a BF16 matrix product with FP32 sums.  A warp
// takes 16 rows of w as the 16 rows of the matrix instruction and eight tokens as its columns; the
// warps of a block share out k and join their sums at the end, in order.

#include "decode_kernels.h"
#include "decode_mma.cuh"

namespace beam {
namespace {

constexpr int kW4Warps = 4;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4Step = 256;                    // k of a warp's step
constexpr int kW4Pitch = kW4Step / 2 + 16;      // bytes of a row in shared memory: no bank conflicts
constexpr int kW4Stages = 5;
constexpr int kW4StageBytes = 16 * kW4Pitch;
constexpr int kW4Smem = kW4Warps * kW4Stages * kW4StageBytes;

// a - b of two BF16 pairs; exact here.
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <int NT>
__global__ void __launch_bounds__(kW4Threads) w4_matvec_kernel(const W4Args a)
{
    extern __shared__ __align__(128) char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int64_t row0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.y * (8 * NT);
    const uint32_t buf = smem_addr(smem) + warp * kW4Stages * kW4StageBytes;
    const int64_t all = (a.K + kW4Step - 1) / kW4Step;
    const int steps = (int)((all - warp + kW4Warps - 1) / kW4Warps);
    const int64_t kbytes = a.K / 2, groups = a.K / a.group;
    pdl_launch_dependents();
    auto issue = [&](int s) {
        if (s < steps) {
            const int64_t b0 = (int64_t)(s * kW4Warps + warp) * (kW4Step / 2);
            const uint32_t dst = buf + (s % kW4Stages) * kW4StageBytes;
            const int ch = lane & 7;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 4 * j + (lane >> 3);
                const bool in = row0 + r < a.N && b0 + 16 * ch < kbytes;
                const char *src =
                    (const char *)a.w + (in ? (row0 + r) * kbytes + b0 + 16 * ch : 0);
                cp_async16(dst + r * kW4Pitch + 16 * ch, src, in ? 16u : 0u);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kW4Stages - 1; ++s)
        issue(s);
    pdl_wait();  // the weights are parameters; x is not
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
    const bool r0 = row0 + g < a.N, r1 = row0 + g + 8 < a.N;
    const uint16_t *sc = (const uint16_t *)a.scales;
    for (int s = 0; s < steps; ++s) {
        cp_async_wait<kW4Stages - 2>();
        __syncwarp();
        issue(s + kW4Stages - 1);
        const uint32_t st = buf + (s % kW4Stages) * kW4StageBytes;
        const int64_t k0 = (int64_t)(s * kW4Warps + warp) * kW4Step;
        const int blocks = (int)((a.K - k0 < kW4Step ? a.K - k0 : kW4Step) / 32);
        float part[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0.0f;
        for (int j = 0; j < blocks; ++j) {
            const int64_t k = k0 + 32 * j, grp = k / a.group;
            const uint32_t z0 =
                (128u + (a.zeros ? (r0 ? a.zeros[(row0 + g) * groups + grp] & 15u : 0u) : 8u));
            const uint32_t z1 =
                (128u + (a.zeros ? (r1 ? a.zeros[(row0 + g + 8) * groups + grp] & 15u : 0u) : 8u));
            // 128 + z in BF16: 0x4300 + z
            const uint32_t zz0 = (0x4280u + z0) * 0x10001u, zz1 = (0x4280u + z1) * 0x10001u;
            uint32_t w0, w1;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w0) : "r"(st + g * kW4Pitch + 16 * j + 4 * t));
            asm volatile("ld.shared.u32 %0, [%1];"
                         : "=r"(w1)
                         : "r"(st + (g + 8) * kW4Pitch + 16 * j + 4 * t));
            uint32_t f0[4], f1[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // nibbles i and i + 4
                f0[i] = sub_bf16x2(((w0 >> (4 * i)) & 0x000f000fu) | 0x43004300u, zz0);
                f1[i] = sub_bf16x2(((w1 >> (4 * i)) & 0x000f000fu) | 0x43004300u, zz1);
            }
            const uint32_t a0[4] = {f0[0], f1[0], f0[1], f1[1]};
            const uint32_t a1[4] = {f0[2], f1[2], f0[3], f1[3]};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int64_t tok = t0 + 8 * n + g;
                const uint4 x = tok < a.T ? ld_cached((const char *)a.x +
                                                      2 * (tok * a.x_stride + k + 8 * t))
                                          : make_uint4(0u, 0u, 0u, 0u);
                mma16816<false>(part[n], a0, __byte_perm(x.x, x.z, 0x5410),
                                __byte_perm(x.x, x.z, 0x7632));
                mma16816<false>(part[n], a1, __byte_perm(x.y, x.w, 0x5410),
                                __byte_perm(x.y, x.w, 0x7632));
            }
            if ((k + 32) % a.group == 0 || j + 1 == blocks) {  // the group's end, or the step's
                const float s0 = r0 ? bf_lo(sc[(row0 + g) * groups + grp]) : 0.0f;
                const float s1 = r1 ? bf_lo(sc[(row0 + g + 8) * groups + grp]) : 0.0f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[n][e] = __fmaf_rn(e < 2 ? s0 : s1, part[n][e], acc[n][e]);
                        part[n][e] = 0.0f;
                    }
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);  // [warp][token][16 rows]
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            red[(warp * 8 * NT + 8 * n + 2 * t + (e & 1)) * 16 + g + 8 * (e >> 1)] = acc[n][e];
    __syncthreads();
    for (int x = tid; x < 8 * NT * 16; x += kW4Threads) {
        const int64_t tok = t0 + x / 16, n = row0 + x % 16;
        if (tok < a.T && n < a.N) {
            float v = red[x];
#pragma unroll
            for (int w = 1; w < kW4Warps; ++w)
                v = __fadd_rn(v, red[w * 8 * NT * 16 + x]);
            reinterpret_cast<uint16_t *>(a.y)[tok * a.y_stride + n] =
                (uint16_t)pack_bf16x2(v, 0.0f);
        }
    }
}

template <int NT>
cudaError_t launch(const W4Args &a, cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(
        w4_matvec_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kW4Smem);
    if (e != cudaSuccess)
        return e;
    W4Args b = a;
    const int64_t tiles = (a.T + 8 * NT - 1) / (8 * NT);
    for (int64_t at = 0; at < tiles; at += 65535) {
        const int64_t here = tiles - at < 65535 ? tiles - at : 65535;
        b.T = a.T - at * 8 * NT;
        b.x = (const char *)a.x + 2 * at * 8 * NT * a.x_stride;
        b.y = (char *)a.y + 2 * at * 8 * NT * a.y_stride;
        const cudaError_t f =
            launch_pdl(w4_matvec_kernel<NT>, dim3((unsigned)((a.N + 15) / 16), (unsigned)here),
                       dim3(kW4Threads), kW4Smem, stream, b);
        if (f != cudaSuccess)
            return f;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_w4_matvec(const W4Args &a, cudaStream_t stream)
{
    if (a.T <= 8)
        return launch<1>(a, stream);
    if (a.T <= 16)
        return launch<2>(a, stream);
    return launch<4>(a, stream);
}

}  // namespace beam
