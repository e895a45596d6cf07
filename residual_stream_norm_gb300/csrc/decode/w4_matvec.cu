// w4_matvec.cu -- products of a few tokens with a matrix of 4-bit weights (sm_103a).
//
// y[t, n] = sum_g scale[n, g] * ( sum_{k in g} x[t, k] (w[n, k] - z[n, g]) ).  w - z is a whole number of
// at most five bits, exact in BF16, so the inner sum is a BF16 matrix product with FP32 sums: 16 rows of
// w are the 16 rows of the matrix instruction, eight tokens its columns.
//
// A block takes R rows and steps of 256 k through shared memory (cp.async, several stages); its warps
// share out the rows (WN) and each step's k (8 / WN).  With few rows a cluster of blocks shares out k as
// well and joins its sums through distributed shared memory, in order, so no workspace is needed and
// results do not depend on timing.
//
// Measured: 1 token, 6144 x 5120: 10.2 us (floor 2.4 us; six steps a block, then two cluster barriers:
// latency); 8 tokens, 5120 x 14336: 15.2 us with the weights in the L2
// cache, 19.0 from memory; 16 tokens 25.8; 32 tokens, 5120 x 40960, groups of 32: 77.5 us.
// What bounds the larger ones is not the weights' bytes but instructions (53 to 58% of the issue slots,
// warps held up by the arithmetic pipe): unpacking takes 2.75
// instructions a pair of weights (shift, mask with the 128 that makes it a BF16 number, exact
// subtraction of 128 + z), and 32 tokens add the fragments of x and the scaling of each group's sums.
// Rows a block: 1 token 64: 10.2, 32: 11.4, 128: 11.2 us; 8 tokens 15.1, 16.4, 21.0; 32 tokens 128: 77.5,
// 64: 85, 256: 118.  Copies further ahead: equal or slower.

#include "beam_f32x2.cuh"
#include "decode_kernels.h"
#include "decode_mma.cuh"

namespace beam {
namespace {

constexpr int kW4Threads = 256;
constexpr int kStep = 256;          // k of a stage: 128 bytes of each row
constexpr int kWindow = 1024;       // k whose scales and zeros are held at a time

template <int NT, int MTW, int WN, int GROUP>
struct W4Config {
    static constexpr int kTok = 8 * NT;
    static constexpr int kRows = 16 * MTW * WN;
    static constexpr int kWk = 8 / WN;
    static constexpr int kStages = NT >= 4 ? 2 : 4;
    static constexpr int kStageBytes = kRows * 128 + kTok * 512;
    static constexpr int kRed = kWk * kTok * kRows * 4;
    static constexpr int kMain = kStages * kStageBytes > kRed ? kStages * kStageBytes : kRed;
    // then the window's scales and zeros: as copied, and as used (one word each)
    static constexpr int kParams = kMain + kRows * (kWindow / GROUP) * 3;
    static constexpr int kBytes = kParams + kRows * (kWindow / GROUP + 1) * 4;
};

// a - b of two BF16 pairs; exact here.
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

// A float of another block of the cluster, at this block's shared address.
__device__ __forceinline__ float ld_cluster(uint32_t addr, int rank)
{
    float v;
    asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
                 "ld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

// C = A B, without a sum to start from.
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// x: which 16-byte chunk of a token's 128 bytes a chunk is kept at.  A quarter of a warp reads four
// neighbouring chunks of an even and of the next token: no bank conflicts.
__device__ __forceinline__ int x_place(int tok, int chunk)
{
    return chunk ^ (((tok & 1) << 2) | ((tok >> 1) & 3));
}

template <int NT, int MTW, int WN, int GROUP>
__global__ void __launch_bounds__(kW4Threads, NT >= 4 ? 2 : 3)
    w4_matvec_kernel(const W4Args a, int split)
{
    using C = W4Config<NT, MTW, WN, GROUP>;
    constexpr int R = C::kRows, kTok = C::kTok, WK = C::kWk, ST = C::kStages;
    constexpr int kWin = kWindow / GROUP, kPitch = kWin + 1;
    extern __shared__ __align__(128) char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3, wn = warp % WN, wk = warp / WN;
    const int rank = blockIdx.x % split;
    const int64_t row0 = (int64_t)(blockIdx.x / split) * R, t0 = (int64_t)blockIdx.y * kTok;
    const int all = (int)((a.K + kStep - 1) / kStep);
    const int s0 = (int)((int64_t)all * rank / split), s1 = (int)((int64_t)all * (rank + 1) / split);
    const int64_t kbytes = a.K / 2, groups = a.K / GROUP;
    const uint32_t base = smem_addr(smem);
    uint32_t *params = reinterpret_cast<uint32_t *>(smem + C::kParams);  // [R][kPitch]: scale, 128 + zero
    const int toks = (int)(a.T - t0 < kTok ? a.T - t0 : kTok);
    pdl_launch_dependents();

    // weights of step s: rows of 128 bytes, chunk c of row r at c ^ (r % 8)
    const char *w_src = (const char *)a.w + row0 * kbytes + (tid >> 3) * kbytes + 16 * (tid & 7);
    const uint32_t w_dst = base + (tid >> 3) * 128 + 16 * ((tid & 7) ^ ((tid >> 3) & 7));
    const int64_t w_left = kbytes - 16 * (tid & 7);  // > 0: this thread's chunk of step 0 exists
    auto copy_w = [&](int s, int stage) {
        const int64_t at = (int64_t)s * (kStep / 2);
        const uint32_t dst = w_dst + stage * C::kStageBytes;
#pragma unroll
        for (int j = 0; j < R / 32; ++j) {
            const bool in = row0 + 32 * j + (tid >> 3) < a.N && at < w_left;
            cp_async16(dst + 32 * j * 128, in ? w_src + at + 32 * j * kbytes : (const char *)a.w,
                       in ? 16u : 0u);
        }
    };
    // x of step s: four blocks of 64 k, each of rows of 128 bytes
    const char *x_src = (const char *)a.x + 2 * ((t0 + (tid >> 5)) * a.x_stride + 8 * (tid & 31));
    const uint32_t x_dst = base + R * 128 + ((tid & 31) >> 3) * kTok * 128 + (tid >> 5) * 128 +
                           16 * x_place(tid >> 5, tid & 7);
    auto copy_x = [&](int s, int stage) {
        const int64_t k = (int64_t)s * kStep;
        const uint32_t dst = x_dst + stage * C::kStageBytes;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const bool in = 8 * j + (tid >> 5) < toks && k + 8 * (tid & 31) < a.K;
            cp_async16(dst + 8 * j * 128,
                       in ? x_src + 2 * (k + 8 * j * a.x_stride) : (const char *)a.x,
                       in ? 16u : 0u);
        }
    };
    // Scales and zeros of the window that starts with step s (a multiple of four).  Rows that start on 16
    // bytes are copied while the window before is worked on and then unpacked; others are loaded when
    // they are needed, which costs their latency once a window.
    const bool ahead_ok = groups % 16 == 0 && (uint64_t)a.scales % 16 == 0 &&
                          (!a.zeros || (uint64_t)a.zeros % 16 == 0);
    const uint32_t raw_s = base + C::kMain, raw_z = raw_s + R * kWin * 2;
    auto copy_params = [&](int s) {
        constexpr int kChunksS = kWin * 2 / 16;           // of a row's scales: 16 bytes each
        constexpr int kZ = kWin < 16 ? kWin : 16;         // bytes of a copy of zeros
        const int64_t g0 = (int64_t)s * (kStep / GROUP);
        for (int x = tid; x < R * kChunksS; x += kW4Threads) {
            const int r = x / kChunksS, c = x % kChunksS;
            const bool in = row0 + r < a.N && g0 + 8 * c < groups;
            cp_async16(raw_s + 16 * x,
                       (const char *)a.scales + (in ? 2 * ((row0 + r) * groups + g0 + 8 * c) : 0),
                       in ? 16u : 0u);
        }
        if (a.zeros)
            for (int x = tid; x < R * (kWin / kZ); x += kW4Threads) {
                const int r = x / (kWin / kZ), c = x % (kWin / kZ);
                const bool in = row0 + r < a.N && g0 + kZ * c < groups;
                const uint8_t *src = a.zeros + (in ? (row0 + r) * groups + g0 + kZ * c : 0);
                if constexpr (kZ == 16)
                    cp_async16(raw_z + 16 * x, src, in ? 16u : 0u);
                else
                    cp_async8(raw_z + 8 * x, src, in ? 8u : 0u);
            }
    };
    auto load_params = [&](int s) {
        if (ahead_ok) {
            const uint16_t *rs = reinterpret_cast<const uint16_t *>(smem + C::kMain);
            const uint8_t *rz = reinterpret_cast<const uint8_t *>(smem + C::kMain + R * kWin * 2);
#pragma unroll 4
            for (int x = 2 * tid; x < R * kWin; x += 2 * kW4Threads) {  // two groups at a time
                const uint32_t sc = *reinterpret_cast<const uint32_t *>(rs + x);
                const uint32_t z =
                    a.zeros ? *reinterpret_cast<const uint16_t *>(rz + x) & 0x0f0fu : 0x0808u;
                uint32_t *dst = params + x / kWin * kPitch + x % kWin;
                dst[0] = sc << 16 | (0x4300u + (z & 15u));  // 128 + z in BF16
                dst[1] = (sc & 0xffff0000u) | (0x4300u + (z >> 8));
            }
            return;
        }
        const int64_t g0 = (int64_t)s * (kStep / GROUP);
        const int gn = (int)(groups - g0 < kWin ? groups - g0 : kWin);
#pragma unroll 4
        for (int x = tid; x < R * kWin; x += kW4Threads) {
            const int r = x / kWin, i = x % kWin;
            uint32_t v = 0u;
            if (i < gn && row0 + r < a.N) {
                const int64_t at = (row0 + r) * groups + g0 + i;
                v = (uint32_t)((const uint16_t *)a.scales)[at] << 16;
                v |= 0x4300u + (a.zeros ? a.zeros[at] & 15u : 8u);  // 128 + z in BF16
            }
            params[r * kPitch + i] = v;
        }
    };
    int win = s0 & ~(kWindow / kStep - 1);
    if (ahead_ok)
        copy_params(win);
#pragma unroll
    for (int s = 0; s < ST - 1; ++s)  // the weights are parameters: they need not wait
        if (s0 + s < s1)
            copy_w(s0 + s, s);
    if (!ahead_ok)
        load_params(win);
    pdl_wait();
#pragma unroll
    for (int s = 0; s < ST - 1; ++s) {
        if (s0 + s < s1)
            copy_x(s0 + s, s);
        cp_async_commit();  // the first group holds every weight copy so far too
    }

    f2 acc[MTW][NT][2];  // pairs of neighbouring tokens: rows g and g + 8
#pragma unroll
    for (int m = 0; m < MTW; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            acc[m][n][0] = acc[m][n][1] = 0ull;
    int stage = 0, ahead = ST - 1;
    bool fresh = ahead_ok;  // the window's parameters are there, but not unpacked
    for (int s = s0; s < s1; ++s) {
        // Step i of the block (from 0) finds ST - 1 + i groups committed and needs the first i + 1, the
        // weights' and x's of its own: all but the newest ST - 2.  The second window's scales and
        // zeros are in group ST - 1 (from 0), with the copies that step 0 issues.  A block whose
        // share starts on step s0 % 4 of a window needs them in step 4 - s0 % 4, which with four
        // stages covers group 4 for s0 % 4 = 0 and 3 for 1, but only 2 for 2 and 1 for 3: there
        // everything is waited for.  Later windows are copied four steps ahead.  (A second buffer
        // instead of the wait: equal times, but 9 to 16 tokens in groups of 64 then fit one block an SM,
        // 5120 -> 14336 25.6 -> 35.2 us.)
        if (ST > 2 && s - win == kWindow / kStep && s - s0 < ST - 1)
            cp_async_wait<0>();
        else
            cp_async_wait<ST - 2>();
        __syncthreads();
        if (s - win == kWindow / kStep)
            win = s, fresh = true;
        if (fresh) {
            load_params(win);
            __syncthreads();
            if (ahead_ok && win + kWindow / kStep < s1)
                copy_params(win + kWindow / kStep);
            fresh = false;
        }
        if (s + ST - 1 < s1) {
            copy_w(s + ST - 1, ahead);
            copy_x(s + ST - 1, ahead);
        }
        ahead = ahead + 1 == ST ? 0 : ahead + 1;
        cp_async_commit();
        const char *ws = smem + stage * C::kStageBytes, *xs = ws + R * 128;
        stage = stage + 1 == ST ? 0 : stage + 1;
        // this warp's part of the step, a group or a part of one at a time: BLK blocks of 32 k
        constexpr int kMine = 8 / WK, kMost = NT >= 8 ? 1 : (NT >= 4 ? 2 : 4);
        constexpr int kInGroup = GROUP / 32 < kMine ? GROUP / 32 : kMine;
        constexpr int BLK = kInGroup < kMost ? kInGroup : kMost;
#pragma unroll
        for (int jg = 0; jg < kMine / BLK; ++jg) {
            const int j0 = wk * kMine + jg * BLK;
            uint32_t b[BLK][NT][4];
#pragma unroll
            for (int jj = 0; jj < BLK; ++jj)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int j = j0 + jj;
                    const uint4 x = *reinterpret_cast<const uint4 *>(
                        xs + (j >> 1) * kTok * 128 + (8 * n + g) * 128 +
                        16 * x_place(g, 4 * (j & 1) + t));
                    b[jj][n][0] = __byte_perm(x.x, x.z, 0x5410);
                    b[jj][n][1] = __byte_perm(x.x, x.z, 0x7632);
                    b[jj][n][2] = __byte_perm(x.y, x.w, 0x5410);
                    b[jj][n][3] = __byte_perm(x.y, x.w, 0x7632);
                }
            const uint32_t *pp = params + (wn * MTW * 16 + g) * kPitch +
                                 (s - win) * (kStep / GROUP) + 32 * j0 / GROUP;
#pragma unroll
            for (int m = 0; m < MTW; ++m) {
                const uint32_t p0 = pp[16 * m * kPitch], p1 = pp[(16 * m + 8) * kPitch];
                const uint32_t z0 = __byte_perm(p0, p0, 0x1010), z1 = __byte_perm(p1, p1, 0x1010);
                float part[NT][4];
#pragma unroll
                for (int jj = 0; jj < BLK; ++jj) {
                    const char *at = ws + (wn * MTW * 16 + g) * 128 + 16 * ((j0 + jj) ^ g) + 4 * t;
                    const uint32_t w0 = *reinterpret_cast<const uint32_t *>(at + 16 * m * 128);
                    const uint32_t w1 =
                        *reinterpret_cast<const uint32_t *>(at + (16 * m + 8) * 128);
                    uint32_t f0[4], f1[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // values i and i + 4 of the eight
                        f0[i] = sub_bf16x2(((w0 >> (4 * i)) & 0x000f000fu) | 0x43004300u, z0);
                        f1[i] = sub_bf16x2(((w1 >> (4 * i)) & 0x000f000fu) | 0x43004300u, z1);
                    }
                    const uint32_t a0[4] = {f0[0], f1[0], f0[1], f1[1]};
                    const uint32_t a1[4] = {f0[2], f1[2], f0[3], f1[3]};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (jj == 0)
                            mma16816_first(part[n], a0, b[jj][n][0], b[jj][n][1]);
                        else
                            mma16816<false>(part[n], a0, b[jj][n][0], b[jj][n][1]);
                        mma16816<false>(part[n], a1, b[jj][n][2], b[jj][n][3]);
                    }
                }
                const f2 c0 = splat(__uint_as_float(p0 & 0xffff0000u));
                const f2 c1 = splat(__uint_as_float(p1 & 0xffff0000u));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[m][n][0] = fma2(c0, make_f2(part[n][0], part[n][1]), acc[m][n][0]);
                    acc[m][n][1] = fma2(c1, make_f2(part[n][2], part[n][3]), acc[m][n][1]);
                }
            }
        }
    }
    // ---- the warps' sums over k, then the cluster's, in order ------------------------------------------
    cp_async_wait<0>();
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);  // [WK][kTok][R]
#pragma unroll
    for (int m = 0; m < MTW; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(wk * kTok + 8 * n + 2 * t + (e & 1)) * R + (wn * MTW + m) * 16 + g +
                    8 * (e >> 1)] = e & 1 ? hi_of(acc[m][n][e >> 1]) : lo_of(acc[m][n][e >> 1]);
    __syncthreads();
    constexpr int kOut = kTok * R;
    const int first = kOut / split * rank, end = kOut / split * (rank + 1);
    if (split > 1) {
        for (int x = tid; x < toks * R; x += kW4Threads) {
            float v = red[x];
#pragma unroll
            for (int w = 1; w < WK; ++w)
                v = __fadd_rn(v, red[w * kOut + x]);
            red[x] = v;
        }
        cluster_sync();
    }
    for (int x = first + tid; x < end; x += kW4Threads) {
        const int64_t tok = x / R, n = row0 + x % R;
        if (tok >= toks || n >= a.N)
            continue;
        float v;
        if (split > 1) {
            v = ld_cluster(base + 4 * x, 0);
            for (int q = 1; q < split; ++q)
                v = __fadd_rn(v, ld_cluster(base + 4 * x, q));
        } else {
            v = red[x];
#pragma unroll
            for (int w = 1; w < WK; ++w)
                v = __fadd_rn(v, red[w * kOut + x]);
        }
        reinterpret_cast<uint16_t *>(a.y)[(t0 + tok) * a.y_stride + n] =
            (uint16_t)pack_bf16x2(v, 0.0f);
    }
    if (split > 1)
        cluster_sync();  // the others may still read this block's sums
}

template <int NT, int MTW, int WN, int GROUP>
cudaError_t launch(const W4Args &a, cudaStream_t stream)
{
    using C = W4Config<NT, MTW, WN, GROUP>;
    constexpr int bytes = C::kBytes;
    cudaError_t e = allow_smem<w4_matvec_kernel<NT, MTW, WN, GROUP>>(bytes);
    if (e != cudaSuccess)
        return e;
    const int64_t tiles = (a.N + C::kRows - 1) / C::kRows;
    const int64_t steps = (a.K + kStep - 1) / kStep;
    const int64_t ttiles = (a.T + C::kTok - 1) / C::kTok;
    // How many blocks of a cluster share out k: what makes the rounds of blocks on the SMs shortest, a
    // block costing about three steps besides its own.
    const int64_t slots = kPlanSms * (NT >= 4 ? 2 : 3);
    int split = 1;
    int64_t best = INT64_MAX;
    for (int q = 1; q <= 8 && q <= steps; q *= 2) {
        const int64_t cost =
            (tiles * ttiles * q + slots - 1) / slots * ((steps + q - 1) / q + 3);
        if (cost < best)
            best = cost, split = q;
    }
    W4Args b = a;
    for (int64_t at = 0; at < ttiles; at += 65535) {
        const int64_t here = ttiles - at < 65535 ? ttiles - at : 65535;
        b.T = a.T - at * C::kTok;
        b.x = (const char *)a.x + 2 * at * C::kTok * a.x_stride;
        b.y = (char *)a.y + 2 * at * C::kTok * a.y_stride;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(tiles * split), (unsigned)here);
        cfg.blockDim = dim3(kW4Threads);
        cfg.dynamicSmemBytes = bytes;
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
        e = cudaLaunchKernelEx(&cfg, w4_matvec_kernel<NT, MTW, WN, GROUP>, b, split);
        if (e != cudaSuccess)
            return e;
    }
    return cudaGetLastError();
}

template <int NT, int MTW, int WN>
cudaError_t launch_group(const W4Args &a, cudaStream_t stream)
{
    return a.group == 32   ? launch<NT, MTW, WN, 32>(a, stream)
           : a.group == 64 ? launch<NT, MTW, WN, 64>(a, stream)
                           : launch<NT, MTW, WN, 128>(a, stream);
}

}  // namespace

cudaError_t launch_w4_matvec(const W4Args &a, cudaStream_t stream)
{
    if (a.T <= 8)
        return launch_group<1, 2, 2>(a, stream);
    if (a.T <= 16)
        return launch_group<2, 2, 4>(a, stream);
    if (a.T <= 32)
        return launch_group<4, 2, 4>(a, stream);
    return launch_group<8, 1, 8>(a, stream);
}

}  // namespace beam
