// attn_prefix_tc.cu -- the shared prefix's part of the attention for many query rows (sm_103a).
//
// All query rows that share a KV head see the same keys, so S = Q K^T and O = P V are products of
// 128 x 128 tiles: tcgen05, sums in tensor memory.  A block takes two tiles of 128 rows (or, when there
// are no more than 128 rows, two streams of key tiles for the one tile) and works on them in turn:
// while one half's four warps turn scores into weights, a row a thread, the tensor cores work for the
// other.  The weights go back to tensor memory in the place of the scores' second half, in 16 bits,
// as the A operand of the second product.
//
// What bounds it: for 768 rows and 32K keys it takes 80 us (1.29 PFLOP/s, tensor pipe 52% busy).  A step
// (two products of 128 x 128 x 128 for each half) takes about 3450 cycles, of which the products need
// 2180 at the full rate.  In a trace Q K^T's eight instructions take 890 of them and P V's 540; the likely
// reason is that the former read both operands from shared memory, which the copies write as well; and
// a half's next scores must wait until its weights, which lie in their place, have been used.  FP8: the
// expansion to FP16 shares the shared memory too (3900 cycles a step).  Alone, a block costs about
// 11 us to set up and write out, so few rows or keys go to the rows kernel.
//
// The reference m of a row is raised (and O scaled, in tensor memory) only when a score exceeds what it was
// raised to by more than 8, a published way to leave out nearly all scaling of an online softmax.  A BF16
// cache's weights 2^(s - m) then stay below 2^8, which BF16 and FP32 hold as well as those below 1.  For an FP8
// cache they are FP16, so m is raised to 7 below the largest score: they reach 2^7 at least and 2^15 at most,
// are within 2^-11 of themselves down to 2^-21 of the largest, and below that within 2^-32 of it.
//
// A window cuts the prefix row by row.  A weight of zero does not hide an infinite or NaN value from the
// matrix product, so where some row does not see a key of a tile the softmax warps first look the
// tile's values over, and put zeros in the place of such values; the rows that do see them get them
// back at the end.
//
// Roles: warps 0-7 softmax; 8 issues the products; 9 copies keys and 10 values (TMA, by slot; one warp
// for both took longer to issue a tile's copies than the products took); for an FP8 cache warps 11-14
// expand the copied bytes to FP16 (exact) in the layout of the products.

#include "attn_common.cuh"
#include "beam_f32x2.cuh"
#include "decode_mma.cuh"
#include "decode_tc.cuh"
#include "decode_tma.cuh"

namespace beam {
namespace {

__device__ unsigned int g_tc_fault_word = 0u;

constexpr int kTile = 128 * 128 * 2;  // bytes of a 128 x 128 tile of 16-bit values: two halves
constexpr int kHalfTile = kTile / 2;  // 64 values of each row
constexpr int kRawTile = 128 * 128;   // FP8
constexpr float kRaise = 8.0f;
constexpr float kBelow = 7.0f;  // FP8

template <bool FP8, bool SPLIT>
struct TcConfig {
    static constexpr int kThreads = FP8 ? 480 : 352;
    static constexpr int kQTiles = SPLIT ? 1 : 2;
    static constexpr int kRaw = FP8 ? (SPLIT ? 4 : 2) : 0;  // half of them keys, half values
    static constexpr int kRing = kRaw > 0 ? kRaw / 2 : 1;
    static constexpr int kK = kQTiles * kTile;        // two stages
    static constexpr int kV = kK + 2 * kTile;         // two stages
    static constexpr int kRawAt = kV + 2 * kTile;
    static constexpr int kMask = kRawAt + kRaw * kRawTile;  // uint32_t [8][4]
    static constexpr int kBars = kMask + 128;
    static constexpr int kNumBars = 1 + 8 + 8 + 2 + 2 + 1 + 8;
    static constexpr int kMisc = kBars + 8 * kNumBars;      // tensor memory address, fail
    static constexpr int kBytes = kMisc + 16;                // + largest first key, values left out
    static_assert(kBytes <= 232448, "shared memory of a block");
};

// 64 columns of this thread's row, complete on return.
__device__ __forceinline__ void load64(uint32_t addr, float (&r)[64])
{
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
          "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
          "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
          "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31]),
          "=r"(u[32]), "=r"(u[33]), "=r"(u[34]), "=r"(u[35]), "=r"(u[36]), "=r"(u[37]),
          "=r"(u[38]), "=r"(u[39]), "=r"(u[40]), "=r"(u[41]), "=r"(u[42]), "=r"(u[43]),
          "=r"(u[44]), "=r"(u[45]), "=r"(u[46]), "=r"(u[47]), "=r"(u[48]), "=r"(u[49]),
          "=r"(u[50]), "=r"(u[51]), "=r"(u[52]), "=r"(u[53]), "=r"(u[54]), "=r"(u[55]),
          "=r"(u[56]), "=r"(u[57]), "=r"(u[58]), "=r"(u[59]), "=r"(u[60]), "=r"(u[61]),
          "=r"(u[62]), "=r"(u[63])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Puts zeros in the place of the infinite and NaN values of a tile; 128 threads.  Whether this thread
// found one.
template <bool F16>
__device__ __forceinline__ bool leave_out(uint32_t tile, int t)
{
    constexpr uint32_t kExp = F16 ? 0x7c007c00u : 0x7f807f80u;
    bool found = false;
#pragma unroll 4
    for (int i = 0; i < kTile / 16 / 128; ++i) {
        const uint32_t at = tile + (i * 128 + t) * 16;
        uint4 v = lds128(at);
        uint32_t bad = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t x = __vcmpeq2(word(v, k) & kExp, kExp);
            word(v, k) &= ~x;
            bad |= x;
        }
        if (bad) {
            sts128(at, v);
            found = true;
        }
    }
    return found;
}

// Adds to a row's sums, in shared memory (chunk c at c ^ (lane % 8)), the infinite and NaN values of the
// keys it sees.
template <bool FP8>
__device__ __noinline__ void put_back(const AttnArgs &a, uint32_t row, int lane, int kvh, int64_t key,
                                      int64_t key_end)
{
    for (; key < key_end; ++key) {
        const int64_t slot = a.prefix[key];
        if (slot < 0 || slot >= a.num_slots)
            continue;
        const int64_t at = (slot * a.n_kv + kvh) * kD;
        for (int d = 0; d < kD; ++d) {
            float v;
            if constexpr (FP8)
                v = (((const uint8_t *)a.v_cache)[at + d] & 0x7fu) == 0x7fu
                        ? __uint_as_float(0x7fc00000u)
                        : 0.0f;
            else
                v = __uint_as_float((uint32_t)((const uint16_t *)a.v_cache)[at + d] << 16);
            if (!isfinite(v)) {
                const uint32_t p = row + 16 * ((d >> 2) ^ (lane & 7)) + 4 * (d & 3);
                float o;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(o) : "r"(p) : "memory");
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(p), "f"(__fadd_rn(o, v)) : "memory");
            }
        }
    }
}

// One product of 128 x 128 x 128: eight steps of 16.
__device__ __forceinline__ void scores_product(uint32_t d, uint32_t q, uint32_t k, uint32_t desc)
{
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        const uint32_t off = (ks >> 2) * kHalfTile + (ks & 3) * 32;
        tc_mma_ss(d, operand_desc(q + off, 16), operand_desc(k + off, 16), desc, ks > 0);
    }
}

__device__ __forceinline__ void values_product(uint32_t d, uint32_t p, uint32_t v, uint32_t desc,
                                               bool add)
{
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
        tc_mma_ts(d, p + 8 * ks, operand_desc(v + ks * 2048, kHalfTile), desc, add || ks > 0);
}

template <bool FP8, bool SPLIT, bool WINDOW>
__global__ void __launch_bounds__(TcConfig<FP8, SPLIT>::kThreads, 1)
    attn_tc_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnPlan p,
                   const __grid_constant__ CacheMaps maps)
{
    using C = TcConfig<FP8, SPLIT>;
    extern __shared__ __align__(1024) char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = smem_addr(smem);
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(smem + C::kMask);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBars);
    uint64_t *q_full = bars, *k_full = bars + 1, *k_empty = bars + 3, *v_full = bars + 5,
             *v_empty = bars + 7, *m_full = bars + 9, *s_full = bars + 17, *p_full = bars + 19,
             *o_full = bars + 21, *r_full = bars + 22, *r_empty = bars + 26;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::kMisc);
    volatile int *s_fail = reinterpret_cast<int *>(smem + C::kMisc + 4);
    int *s_first = reinterpret_cast<int *>(smem + C::kMisc + 8);
    volatile int *s_left_out = reinterpret_cast<int *>(smem + C::kMisc + 12);

    const int kvh = blockIdx.y;
    const int64_t row0 = (int64_t)blockIdx.x * (SPLIT ? 128 : 256);
    const int64_t key0 = p.p_first + (int64_t)blockIdx.z * p.tc_steps * (SPLIT ? 256 : 128);
    const int64_t key_end = min(a.n_prefix, key0 + (int64_t)p.tc_steps * (SPLIT ? 256 : 128));
    const int N = (int)((key_end - key0 + 127) / 128);          // key tiles
    const int halves = SPLIT ? 2 : (p.rows - row0 > 128 ? 2 : 1);  // that have rows

    if (tid == 0) {
        *s_fail = base % 1024 != 0;
        *s_first = 0;
        *s_left_out = 0;
        mbar_init(q_full, SPLIT ? 128 : 128 * halves);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], FP8 ? 128 : 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], FP8 ? 128 : 1);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
        }
        mbar_init(o_full, 1);
        for (int i = 0; i < 8; ++i)
            mbar_init(&m_full[i], 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&r_full[i], 1);
            mbar_init(&r_empty[i], 128);
        }
        fence_mbar_init();
    }
    // Tensor memory is asked for behind the kernels before, and the next one may start only when every block here has it:
    // a block that held columns while it waits for another kernel's end could keep that kernel's blocks from theirs.
    pdl_wait();
    if (warp == 8)
        tmem_alloc_all(s_tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    pdl_launch_dependents();

    if (warp < 8 && !*s_fail) {
        // ---- softmax: a row a thread -------------------------------------------------------------
        const int half = warp >> 2;
        const int64_t rr = row0 + (SPLIT ? 0 : 128 * half) + (tid & 127);
        const bool act = rr < p.rows;
        bool seen = false;
        int first = 0;  // first key that the row sees, counted from key0
        float scale = 0.0f;
        if (half < halves) {
            int i = 0, hg = 0;
            const int64_t tok = act ? row_token(a, p, rr, i, hg) : 0;
            if (act) {
                const int64_t pos = seq_len(a, (uint32_t)rr / (uint32_t)p.R) - a.q_len + i;
                seen = pos >= 0;
                if (WINDOW && seen)
                    first = (int)max((int64_t)0, min(key_end, a.n_prefix + pos + 1 - a.window) - key0);
            }
            if constexpr (WINDOW) {
                const int most = __reduce_max_sync(0xffffffffu, first);
                if (lane == 0)
                    atomicMax(s_first, most);
                named_sync(1, 128 * (SPLIT ? 2 : halves));
            }
            // The warp loads its 32 rows two at a time, half a warp a row, all of them in flight;
            // FP8: a row's largest magnitude gives the factor that takes it to FP16.
            const int64_t off =
                act ? 2 * (tok * a.q_stride + (int64_t)(kvh * p.group + hg) * kD) : -1;
            uint4 row[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int64_t o = __shfl_sync(0xffffffffu, off, 2 * k + (lane >> 4));
                row[k] = o >= 0 ? ld_cached((const char *)a.q + o + 16 * (lane & 15))
                                : make_uint4(0u, 0u, 0u, 0u);
            }
            float inv = 1.0f;
            if constexpr (FP8) {
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    uint32_t mx = 0u;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t w = word(row[k], j);
                        mx = max(mx, max((w << 16) & 0x7fffffffu, w & 0x7fff0000u));
                    }
#pragma unroll
                    for (int x = 1; x < 16; x <<= 1)
                        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                    float f, back;
                    f16_row_factor(mx, f, back);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        word(row[k], j) = pack_f16x2(__fmul_rn(bf_lo(word(row[k], j)), f),
                                                     __fmul_rn(bf_hi(word(row[k], j)), f));
                    back = __shfl_sync(0xffffffffu, back, 16 * (lane & 1));
                    inv = lane >> 1 == k ? back : inv;  // of this thread's row
                }
            }
            scale = __fmul_rn(__fmul_rn(a.sm_scale * a.k_scale, kLog2e), inv);
            if (!SPLIT || half == 0) {
                const uint32_t dst = base + (SPLIT ? 0 : half) * kTile + (lane >> 3 & 1) * kHalfTile;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int r = 32 * (warp & 3) + 2 * k + (lane >> 4);
                    sts128(dst + r * 128 + 16 * ((lane & 7) ^ (r & 7)), row[k]);
                }
                fence_async_shared();
                mbar_arrive(q_full);
            }
        }
        const int tiles = half >= halves ? 0 : (SPLIT ? (N + 1 - half) / 2 : N);
        const uint32_t s_at = tmem + half * 128 + ((uint32_t)(warp & 3) << 21);
        const uint32_t o_at = s_at - half * 128 + 256 + half * 128;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        const int most_first = WINDOW ? *s_first : 0;
        // scores of 64 columns from c0 on: -inf where there is no key or the row does not see it
        bool all = true, cut = false;  // whether the tile has all keys; whether the window cuts it
        auto hide = [&](float (&r)[64], uint32_t m0, uint32_t m1, int c0, int from) {
            if (!all) {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    r[c] = ((c < 32 ? m0 : m1) >> (c & 31)) & 1u ? r[c] : -INFINITY;
            }
            if (WINDOW && cut) {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    r[c] = c0 + c >= from ? r[c] : -INFINITY;
            }
        };
        for (int j = 0; j < tiles; ++j) {
            const int i = SPLIT ? 2 * j + half : j;
            ok = mbar_wait_or_fail(&m_full[i & 7], (i >> 3) & 1, s_fail) &&
                 mbar_wait_or_fail(&s_full[half], j & 1, s_fail);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t mask[4];
#pragma unroll
            for (int w = 0; w < 4; ++w)
                mask[w] = s_mask[4 * (i & 7) + w];
            const int from = first - 128 * i;  // the row's first column
            all = (mask[0] & mask[1] & mask[2] & mask[3]) == 0xffffffffu;
            cut = WINDOW && most_first > 128 * i;
            float r[64];
            float mx0 = -INFINITY, mx1 = -INFINITY;
            load64(s_at, r);
            hide(r, mask[0], mask[1], 0, from);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                mx0 = max3(mx0, r[c], r[c + 1]);
                mx1 = max3(mx1, r[c + 2], r[c + 3]);
            }
            load64(s_at + 64, r);
            hide(r, mask[2], mask[3], 64, from);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                mx0 = max3(mx0, r[c], r[c + 1]);
                mx1 = max3(mx1, r[c + 2], r[c + 3]);
            }
            // rounded so that no weight passes its bound
            constexpr float below = FP8 ? kBelow : 0.0f;
            const float mx = __fmul_ru(fmaxf(mx0, mx1), scale);
            const bool raise = mx > __fadd_rd(m, below + kRaise);
            if (__any_sync(0xffffffffu, raise)) {
                const float mn = raise ? __fsub_ru(mx, below) : m;
                const float f = m == mn ? 1.0f : exp2_fast(__fsub_rn(m, mn));
                l = __fmul_rn(l, f);
                m = mn;
                if (j > 0) {  // the last product with the values is complete: s_full came after it
                    float o[64];
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        // keep the scores in r: they are read again below
                        load64(o_at + 64 * h, o);
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            o[c] = __fmul_rn(o[c], f);
                        tmem_st32(o_at + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(&o[0]));
                        tmem_st32(o_at + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(&o[32]));
                    }
                    load64(s_at + 64, r);
                    hide(r, mask[2], mask[3], 64, from);
                }
            }
            const float neg = m == -INFINITY ? 0.0f : -m;
            const f2 scale2 = splat(scale), neg2 = splat(neg);
            f2 sum = 0ull;
#pragma unroll
            for (int h = 1; h >= 0; --h) {  // the second half is in registers and makes room first
                if (h == 0) {
                    load64(s_at, r);
                    hide(r, mask[0], mask[1], 0, from);
                }
                uint32_t w[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const f2 x = fma2(make_f2(r[2 * c], r[2 * c + 1]), scale2, neg2);
                    const float e0 = exp2_fast(lo_of(x)), e1 = exp2_fast(hi_of(x));
                    sum = add2(sum, make_f2(e0, e1));
                    w[c] = FP8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
                }
                tmem_st32(s_at + 64 + 32 * h, w);
            }
            l = __fadd_rn(l, __fadd_rn(lo_of(sum), hi_of(sum)));
            if (cut) {
                ok = mbar_wait_or_fail(&v_full[i & 1], (i >> 1) & 1, s_fail);
                if (ok && leave_out<FP8>(base + C::kV + (i & 1) * kTile, tid & 127))
                    *s_left_out = 1;
                fence_async_shared();
                __syncwarp();  // the warp is whole again before its tensor-memory instructions
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_full[half]);
        }
        // ---- the part ----------------------------------------------------------------------------
        // (by whole warps, also where a wait runs out for some lanes only)
        if (half < halves &&
            __all_sync(0xffffffffu, ok && mbar_wait_or_fail(o_full, 0, s_fail))) {
            tc_fence_after();
            const int part = SPLIT ? 2 * blockIdx.z + half : blockIdx.z;
            const int64_t at = ((int64_t)kvh * p.rows + rr) * p.tc_parts + part;
            if (tiles > 0) {
                // The stages are free now (every copy has arrived, every product is complete): a warp's
                // 32 rows go through them, so that rows are written whole.  Chunk c of row r lies at
                // c ^ (r % 8).
                const uint32_t stage = base + (half ? C::kV : C::kK) + (warp & 3) * 16384;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    float r[64];
                    load64(o_at + 64 * h, r);
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        sts128(stage + lane * 512 + 16 * ((16 * h + c) ^ (lane & 7)),
                               make_uint4(__float_as_uint(r[4 * c]), __float_as_uint(r[4 * c + 1]),
                                          __float_as_uint(r[4 * c + 2]),
                                          __float_as_uint(r[4 * c + 3])));
                }
                if constexpr (WINDOW) {
                    if (act && *s_left_out)
                        put_back<FP8>(a, stage + lane * 512, lane, kvh, key0 + first, key_end);
                }
                __syncwarp();
                const int64_t rr0 = rr - lane;
                const int rows = (int)min((int64_t)32, p.rows - rr0);
                const int64_t step = (int64_t)p.tc_parts * kD;
                float *po = reinterpret_cast<float *>(a.workspace + p.tc_o_off) +
                            ((int64_t)kvh * p.rows + rr0) * step + part * kD + 4 * lane;
#pragma unroll
                for (int x0 = 0; x0 < 32; x0 += 8) {
                    uint4 v[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        v[x] = lds128(stage + (x0 + x) * 512 + 16 * (lane ^ x));
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (x0 + x < rows)
                            st_global(po + (x0 + x) * step, v[x]);
                }
            }
            if (act)
                reinterpret_cast<float2 *>(a.workspace + p.tc_ml_off)[at] =
                    make_float2(seen ? m : -INFINITY, seen ? l : 0.0f);
        }
    } else if (warp == 8 && !*s_fail) {
        // ---- the products: the whole warp waits, one lane issues (descriptors then stay uniform) -------
        {
            const bool one = elect_one();
            constexpr uint32_t dqk = mma_desc(FP8, false), dpv = mma_desc(FP8, true);
            const uint32_t kt = base + C::kK, vt = base + C::kV;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait_or_fail(bar, parity, s_fail));
                return ok;
            };
            wait(q_full, 0);
            auto wait_k = [&](int i) { wait(&k_full[i & 1], (i >> 1) & 1); };
            auto qk = [&](int half, int i) {
                tc_fence_after();
                if (one) {
                    scores_product(tmem + half * 128, base + (SPLIT ? 0 : half) * kTile,
                                   kt + (i & 1) * kTile, dqk);
                    tc_commit(&s_full[half]);
                }
                __syncwarp();
            };
            auto pv = [&](int half, int j, int i) {
                tc_fence_after();
                if (one)
                    values_product(tmem + 256 + half * 128, tmem + half * 128 + 64,
                                   vt + (i & 1) * kTile, dpv, j > 0);
                __syncwarp();
            };
            auto commit = [&](uint64_t *bar) {
                if (one)
                    tc_commit(bar);
                __syncwarp();
            };
            if constexpr (SPLIT) {
                for (int i = 0; i < 2 && i < N && ok; ++i) {
                    wait_k(i);
                    if (!ok)
                        break;
                    qk(i, i);
                    commit(&k_empty[i]);
                }
                for (int i = 0; i < N && ok; ++i) {
                    const int half = i & 1, j = i >> 1;
                    if (!wait(&v_full[i & 1], (i >> 1) & 1) || !wait(&p_full[half], j & 1))
                        break;
                    pv(half, j, i);
                    commit(&v_empty[i & 1]);
                    if (i + 2 < N) {
                        wait_k(i + 2);
                        if (!ok)
                            break;
                        qk(half, i + 2);
                        commit(&k_empty[i & 1]);
                    }
                }
            } else {
                wait_k(0);
                if (ok) {
                    for (int h = 0; h < halves; ++h)
                        qk(h, 0);
                    commit(&k_empty[0]);
                }
                for (int i = 0; i < N && ok; ++i)
                    for (int h = 0; h < halves && ok; ++h) {
                        if (h == 0)
                            wait(&v_full[i & 1], (i >> 1) & 1);
                        if (!wait(&p_full[h], i & 1))
                            break;
                        pv(h, i, i);
                        if (h == halves - 1)
                            commit(&v_empty[i & 1]);
                        if (i + 1 < N) {
                            if (h == 0)
                                wait_k(i + 1);
                            if (!ok)
                                break;
                            qk(h, i + 1);
                            if (h == halves - 1)
                                commit(&k_empty[(i + 1) & 1]);
                        }
                    }
            }
            if (ok)
                commit(o_full);
        }
        __syncwarp();
    } else if ((warp == 9 || warp == 10) && !*s_fail) {
        // ---- copies: keys (warp 9, with the masks of which exist) or values (warp 10) -----------------
        const bool v = warp == 10;
        const CUtensorMap *run = v ? &maps.v_run : &maps.k_run, *four = v ? &maps.v : &maps.k;
        auto fetch = [&](int i, int64_t (&x)[4]) {  // this lane's four keys of tile i
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t key = key0 + (int64_t)i * 128 + 4 * lane + j;
                x[j] = i < N && key < key_end ? a.prefix[key] : -1;
            }
        };
        bool ok = true;
        int64_t x[4], ahead[4];
        fetch(0, x);
        for (int i = 0; i < N; ++i) {
            fetch(i + 1, ahead);  // arrives while this tile's copies wait and are issued
            int s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[j] = x[j] >= 0 && x[j] < a.num_slots ? (int)x[j] : -1;
            // runs of 16 slots go as one copy, others four by four
            const int s0 = __shfl_sync(0xffffffffu, s[0], lane & ~3);
            const bool in = s0 >= 0 && s0 + 15 < a.num_slots && s[0] == s0 + 4 * (lane & 3) &&
                            s[1] == s[0] + 1 && s[2] == s[0] + 2 && s[3] == s[0] + 3;
            const bool whole =
                ((__ballot_sync(0xffffffffu, in) >> (lane & ~3)) & 15u) == 15u;
            uint64_t *full, *empty;
            uint32_t dst, parity;
            if constexpr (FP8) {
                const int st = i % C::kRing;
                full = &r_full[2 * v + st];
                empty = &r_empty[2 * v + st];
                parity = ((i / C::kRing) & 1) ^ 1;
                dst = base + C::kRawAt + (v * C::kRing + st) * kRawTile;
            } else {
                full = v ? &v_full[i & 1] : &k_full[i & 1];
                empty = v ? &v_empty[i & 1] : &k_empty[i & 1];
                parity = ((i >> 1) & 1) ^ 1;
                dst = base + (v ? C::kV : C::kK) + (i & 1) * kTile;
            }
            ok = __all_sync(0xffffffffu, mbar_wait_or_fail(empty, parity, s_fail));
            if (!ok)
                break;
            if (lane == 0)
                mbar_arrive_expect_tx(full, FP8 ? kRawTile : kTile);
            __syncwarp();
            if (whole) {
                // a lane of each four for each half of the head
                if ((lane & 3) < (FP8 ? 1 : 2))
                    copy_run(dst + (lane & 3) * kHalfTile + (lane >> 2) * 2048, run,
                             kvh * kD + 64 * (lane & 3), s0, full);
            } else {
                gather4(dst + lane * 512, four, kvh * kD, s[0], s[1], s[2], s[3], full);
                if (!FP8)
                    gather4(dst + kHalfTile + lane * 512, four, kvh * kD + 64, s[0], s[1], s[2],
                            s[3], full);
            }
            if (!v) {
                // The tile's mask.  Its place was last used by tile i - 8: this copy waited for the
                // scores of tile i - 4 or a later one, so the softmax warps have left tile i - 6.
                uint32_t bits = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    bits |= s[j] >= 0 ? 1u << (4 * (lane & 7) + j) : 0u;
                bits |= __shfl_xor_sync(0xffffffffu, bits, 1);
                bits |= __shfl_xor_sync(0xffffffffu, bits, 2);
                bits |= __shfl_xor_sync(0xffffffffu, bits, 4);
                if ((lane & 7) == 0)
                    s_mask[4 * (i & 7) + (lane >> 3)] = bits;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&m_full[i & 7]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = ahead[j];
        }
    } else if (FP8 && warp >= 11 && !*s_fail) {
        // ---- FP8 to FP16, in the products' order ----------------------------------------------------
        constexpr int ahead = SPLIT ? 2 : 1;
        const int ct = tid - 352;
        bool ok = true;
        auto expand = [&](bool v, int i) {
            const int st = i % C::kRing;
            ok = ok && mbar_wait_or_fail(&r_full[2 * v + st], (i / C::kRing) & 1, s_fail) &&
                 mbar_wait_or_fail(v ? &v_empty[i & 1] : &k_empty[i & 1], ((i >> 1) & 1) ^ 1, s_fail);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                return;
            const uint32_t src = base + C::kRawAt + (v * C::kRing + st) * kRawTile;
            const uint32_t dst = base + (v ? C::kV : C::kK) + (i & 1) * kTile;
#pragma unroll 4
            for (int x = 0; x < 8; ++x) {
                // eight lanes: four chunks of an even and of the next row (stores without conflicts)
                const int idx = x * 128 + ct;
                const int c = (idx & 3) + 4 * ((idx >> 9) & 1), r = (idx >> 2) & 127;
                const uint4 b = lds128(src + r * 128 + 16 * (c ^ (r & 7)));
                const uint4 lo = make_uint4(e4m3x2_to_f16x2(b.x), e4m3x2_to_f16x2(b.x >> 16),
                                            e4m3x2_to_f16x2(b.y), e4m3x2_to_f16x2(b.y >> 16));
                const uint4 hi = make_uint4(e4m3x2_to_f16x2(b.z), e4m3x2_to_f16x2(b.z >> 16),
                                            e4m3x2_to_f16x2(b.w), e4m3x2_to_f16x2(b.w >> 16));
                const uint32_t at = dst + (c >> 2) * kHalfTile + r * 128;
                sts128(at + 16 * ((2 * (c & 3)) ^ (r & 7)), lo);
                sts128(at + 16 * ((2 * (c & 3) + 1) ^ (r & 7)), hi);
            }
            fence_async_shared();
            mbar_arrive(v ? &v_full[i & 1] : &k_full[i & 1]);
            mbar_arrive(&r_empty[2 * v + st]);
        };
        for (int i = 0; i < ahead && i < N && ok; ++i)
            expand(false, i);
        for (int i = 0; i < N && ok; ++i) {
            expand(true, i);
            if (i + ahead < N && ok)
                expand(false, i + ahead);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*s_fail) {
        // a wait ran out: what is in flight ends before the block does (a bounded wait)
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < kWaitLimitNs / 4) {
        }
        if (tid == 0)
            atomicOr(&g_tc_fault_word, kFaultCopyTimeout);
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 8)
        tmem_free_all(tmem);
}

template <bool FP8, bool SPLIT, bool WINDOW>
cudaError_t launch(const AttnArgs &a, const AttnPlan &p, const CacheMaps &maps, cudaStream_t stream)
{
    constexpr int bytes = TcConfig<FP8, SPLIT>::kBytes;
    const cudaError_t e = allow_smem<attn_tc_kernel<FP8, SPLIT, WINDOW>>(bytes);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(attn_tc_kernel<FP8, SPLIT, WINDOW>,
                      dim3((unsigned)p.tc_rtiles, (unsigned)a.n_kv, (unsigned)p.tc_blocks),
                      dim3(TcConfig<FP8, SPLIT>::kThreads), bytes, stream, a, p, maps);
}

template <bool FP8, bool SPLIT>
cudaError_t launch_window(const AttnArgs &a, const AttnPlan &p, const CacheMaps &maps,
                          cudaStream_t stream)
{
    return a.window > 0 ? launch<FP8, SPLIT, true>(a, p, maps, stream)
                        : launch<FP8, SPLIT, false>(a, p, maps, stream);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs &a, const AttnPlan &p, const CacheMaps &maps,
                           cudaStream_t stream)
{
    if (a.fp8)
        return p.tc_split ? launch_window<true, true>(a, p, maps, stream)
                          : launch_window<true, false>(a, p, maps, stream);
    return p.tc_split ? launch_window<false, true>(a, p, maps, stream)
                      : launch_window<false, false>(a, p, maps, stream);
}

cudaError_t read_attn_tc_fault_word(unsigned int *value, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(value, g_tc_fault_word, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0u;
        e = cudaMemcpyToSymbol(g_tc_fault_word, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace beam
