// kv4_attn.cu -- attention of a decode batch over a KV cache held in 4 bits (sm_103a).
//
// A key is 64 bytes of codes and 4 to 16 of scales for its 128 columns, so the kernel is bound by memory only
// if a code costs next to nothing to unpack.  Two things see to that.
//  - A 16-bit word whose low bits are a code c is the FP16 value c 2^-24 (or 16 c 2^-24 for a code in bits
//    4-7): masking a 32-bit word of eight codes, once as it stands and once shifted by 8, gives the four
//    register pairs that a matrix instruction takes, exactly.  The factor 16 of every second pair goes into
//    the query (scaled by 1/16 there) and out of the result's rows.
//  - Codes multiply first and scales after: s = scale <q, c> + minimum sum q, with FP32 sums of exact
//    products, and out = sum (p scale) c + sum p minimum.  The products' sums over 32 keys are added to the
//    output outside the matrix instruction, which cuts off where FP32 rounds: codes are all positive, and what it cuts
//    off over 100,000 keys showed beside values that average out (error 0.0026 instead of 0.0017).
// Both products take the cache as the left operand, whose rows are keys (Q K^T) or columns (V^T P^T), and up
// to 24 query rows of a KV head as the right one, so that few rows waste little: ldmatrix hands out the keys'
// words, and with a transpose the values' (a 16-bit unit is four columns of a key).
//
// Every warp works alone: it copies tiles of 32 keys with cp.async one or two ahead into its own part of shared memory,
// each with a note of where it stands, and carries the running maximum and sum of the unit at hand in registers, its
// output in tensor memory.  A unit is a sequence, a KV head and a tile of query rows.  All sequences' tiles, one after the
// other, are cut into even shares, and a share is walked by a team of neighbouring warps, one for each KV head and row
// tile: the heads' rows of a slot are neighbours in memory, and what one warp's access brings besides is in the L2 cache
// for the others (with shares of single heads instead, at that step, 8 contexts of 100K keys in groups of 32 read 2.6
// times their bytes: 365 us, and 301 so).  A unit that is cut between teams leaves parts (FP32 maximum, sum, output) that
// a second kernel joins in order; short ones are taken whole (see draft_plan.h).
//
// What bounds it: instructions and their latency (8 contexts of 100K keys in groups of 128: 138 us for 720 MB, 0.77 of
// the measured copy rate, in groups of 32 186 us for 847 MB; 24 rows of 32 sequences in groups of 64 163 us for 371 MB at
// about 1,100 instructions a tile).

#include <cuda_fp16.h>

#include "beam_device.cuh"
#include "beam_f32x2.cuh"
#include "beam_tma.cuh"
#include "decode/decode_mma.cuh"
#include "decode/decode_tc.cuh"
#include "draft_kernels.h"

namespace beam {
namespace {

using kv4::kScan;
using kv4::kSms;
using kv4::kTile;
using kv4::warps_of;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMinExp = -100;
constexpr int kReach = 7;

struct Sizes {
    int32_t heads, R, rtiles;
    uint32_t team, teams;   // warps of a team: KV heads * rtiles
    uint32_t gang;          // 0: shares; else the warps that take a unit whole
    uint32_t crew;          // warps that join a row
    uint32_t per;           // sequences that a thread counts
    float *part_o;          // [teams][team][2][8 * NT][128]
    float *part_ml;         // [teams][team][2][8 * NT][2]
};

// What stands behind a tile's codes and scales: where it is from.
struct Note {
    uint32_t valid;          // keys to be seen
    int b, hr;               // sequence; KV head * rtiles + row tile
    int tile, tiles;         // of the unit
    int n, ns, skip;         // keys of the sequence; see Keys
};

__host__ __device__ constexpr int scales_at() { return 2 * kTile * 64; }
__host__ __device__ constexpr int note_at(int NG) { return scales_at() + 2 * kTile * 4 * NG; }
__host__ __device__ constexpr int stage_bytes(int NG) { return note_at(NG) + (int)sizeof(Note); }
constexpr int kSmem = 225 * 1024;
__host__ __device__ constexpr int rows_at(int NT) { return NT * 4 * 32 * 16; }  // behind a query
__host__ __device__ constexpr int query_bytes(int NT) { return NT > 1 ? rows_at(NT) + NT * 8 * 4 * 5 : 0; }
__host__ __device__ constexpr int stages_of(int NT, int NG)
{
    const int fit = (kSmem / warps_of(NT, NG) - query_bytes(NT)) / stage_bytes(NG);
    return fit < 6 ? fit : 6;
}
__host__ __device__ constexpr int warp_bytes(int NT, int NG)
{
    return stages_of(NT, NG) * stage_bytes(NG) + query_bytes(NT);
}

// The keys that any row of a sequence sees, in a list of its own: first the `ns` sinks, then those from
// ns + skip on.
struct Keys {
    int n, ns, skip, count;
    __device__ __forceinline__ int tiles() const { return (count + kTile - 1) / kTile; }
};

__device__ __forceinline__ Keys keys_of(const Kv4AttnArgs &a, uint32_t b)
{
    Keys k;
    const int w = (int)a.width;
    k.n = a.len[b];
    k.n = k.n < 0 ? 0 : (k.n > w ? w : k.n);
    const int first_p = k.n > a.q_len ? k.n - a.q_len : 0;
    const int lo = a.window > 0 && first_p + 1 > a.window ? first_p + 1 - (int)a.window : 0;
    k.ns = lo < a.n_sink ? lo : (int)a.n_sink;
    k.skip = lo - k.ns;
    k.count = k.n - k.skip;
    return k;
}

// Tiles in front of each thread's run of sequences (s_before), and of all sequences.  Fewer than 2^31 in all (the
// entry point's checks).
__device__ __forceinline__ uint32_t scan_tiles(const Kv4AttnArgs &a, const Sizes &z, uint32_t *s_before,
                                               uint32_t *s_warp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t own = 0, s = 0;
    if (threadIdx.x < kScan) {
        const uint32_t first = threadIdx.x * z.per;
#pragma unroll 1
        for (uint32_t b = first; b < first + z.per && b < (uint32_t)a.B; ++b)
            own += (uint32_t)keys_of(a, b).tiles();
        s = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off)
                s += o;
        }
        if (lane == 31)
            s_warp[warp] = s;
    }
    __syncthreads();
    uint32_t total = 0, before = s - own;
#pragma unroll
    for (int i = 0; i < kScan / 32; ++i) {
        before += i < warp ? s_warp[i] : 0;
        total += s_warp[i];
    }
    if (threadIdx.x < kScan)
        s_before[threadIdx.x] = before;
    __syncthreads();
    return total;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

template <int NG>
__device__ __forceinline__ void lds_scales(uint32_t (&w)[NG], uint32_t addr)
{
    if constexpr (NG == 1)
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
    else if constexpr (NG == 2)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr)
                     : "memory");
}

// Columns that hold n: a power of two from 32 on.
__device__ __forceinline__ uint32_t tmem_columns(uint32_t n) { return n <= 32 ? 32 : 1u << (32 - __clz(n - 1)); }

// By one whole warp.
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns) : "memory");
}

// 8 columns of tensor memory, of this thread's lane.  A load's values may be used behind the wait below.
__device__ __forceinline__ void tmem_ld8(uint32_t addr, float (&x)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t addr, const float (&x)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(x[0]),
                 "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "r"(addr)
                 : "memory");
}

// Waits for all loads; the values named are behind it for the compiler too.
template <int N>
__device__ __forceinline__ void tmem_loaded(float (&x)[N][8])
{
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile(""
                     : "+f"(x[i][0]), "+f"(x[i][1]), "+f"(x[i][2]), "+f"(x[i][3]), "+f"(x[i][4]), "+f"(x[i][5]),
                       "+f"(x[i][6]), "+f"(x[i][7]));
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Byte offset of chunk c (16 bytes, 32 columns) of key `key` of a tile: eight keys' chunks take all banks.
__device__ __forceinline__ uint32_t chunk_at(int key, int c)
{
    return (uint32_t)(key * 64 + ((c ^ ((key >> 1) & 3)) << 4));
}

__device__ __forceinline__ void sts_f32(uint32_t at, float x)
{
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
}
__device__ __forceinline__ float2 lds_f32x2(uint32_t at)
{
    float2 x;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(at) : "memory");
    return x;
}

template <int NT, int NG>
struct Unit {
    // query, FP16: columns c*32 + t*8 + {j, j + 4} of row g, j = 0..3 (odd j: a sixteenth); of more than one row tile
    // in shared memory, where it leaves room in the registers
    uint32_t q[1][4][4];
    // rows 2t, 2t+1: with t = scale (sum of products) + minimum qsum, the scores are fac t in powers of two
    // (of more than one row tile in shared memory too, behind the query: [1 + NG][NT * 8])
    float fac[2], qsum[2][NG];
    float m[NT][2], l[NT][2], omin[NT][2][NG];  // of the scaled scores
    int e[NT][2];            // scales seen are below 2^e, the largest of them by no more than 2^(kReach + 1)
    uint32_t raised;         // a bit for each row whose e may be more than its own scales ask for
    bool one_e;              // the same one for all rows
    uint32_t tmem;           // the output: 8 columns for each (chunk, row tile), [2][4] of a product's places
};

// Row `row` of a sequence and KV head: its query's index and place in the sequence.
template <int NT, int NG>
__device__ __forceinline__ void begin_unit(Unit<NT, NG> &u, const Kv4AttnArgs &a, const Sizes &z,
                                           const Note &at, uint32_t qb, int lane)
{
    const int g = lane >> 2, t = lane & 3;
    const int kv = at.hr / z.rtiles, r0 = (at.hr - kv * z.rtiles) * NT * 8;
    uint4 v[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + nt * 8 + g, i = r / z.heads;
        const uint16_t *from = (const uint16_t *)a.q + ((int64_t)at.b * a.q_len + i) * a.q_stride +
                               (kv * z.heads + r - i * z.heads) * 128 + t * 8;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            v[nt][c] = r < z.R ? ld_plain(from + c * 32) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        // the row's power of two: its largest element to [2^14, 2^15)
        uint32_t mx = 0u;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int w = 0; w < 4; ++w)
                mx = max(mx, max(word(v[nt][c], w) & 0x7fffu, (word(v[nt][c], w) >> 16) & 0x7fffu));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        int k = mx >= 0x7f80u || mx == 0u ? 0 : 141 - (int)(mx >> 7);
        k = min(k, 60);
        // a negative scale of the scores turns the query around, none takes it out
        const float f = a.sm_scale == 0.0f ? 0.0f : (a.sm_scale < 0.0f ? -pow2i(k) : pow2i(k));
        float gs[NG];
#pragma unroll
        for (int j = 0; j < NG; ++j)
            gs[j] = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float x[8];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                x[2 * w] = bf_lo(word(v[nt][c], w)) * f;
                x[2 * w + 1] = bf_hi(word(v[nt][c], w)) * f;
                gs[c * NG / 4] += x[2 * w] + x[2 * w + 1];
            }
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float h = j & 1 ? 0.0625f : 1.0f;
                q[j] = pack_f16x2(x[j] * h, x[j + 4] * h);
                if (NT == 1)
                    u.q[0][c][j] = q[j];
            }
            if (NT > 1)  // read by this lane alone
                sts128(qb + ((nt * 4 + c) * 32 + lane) * 16, make_uint4(q[0], q[1], q[2], q[3]));
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            gs[j] += __shfl_xor_sync(0xffffffffu, gs[j], 1);
            gs[j] += __shfl_xor_sync(0xffffffffu, gs[j], 2);
            gs[j] *= 5.9604644775390625e-08f;  // 2^-24, as the codes' products
        }
        // (not 0, which would make NaN of what is masked)
        const float fac = a.sm_scale == 0.0f ? 1.0f
                                             : fmaxf(fabsf(a.sm_scale) * kLog2e * pow2i(-k) * 16777216.0f,
                                                     1.1754943508222875e-38f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int from = (2 * t + e) * 4;  // a lane whose g is this row
            const uint32_t at_row = qb + rows_at(NT) + (nt * 8 + 2 * t + e) * 4;
            const float row_fac = __shfl_sync(0xffffffffu, fac, from);
            if (NT == 1)
                u.fac[e] = row_fac;
            else if (g == 0)
                sts_f32(at_row, row_fac);
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const float row_sum = __shfl_sync(0xffffffffu, gs[j], from);
                if (NT == 1)
                    u.qsum[e][j] = row_sum;
                else if (g == 0)
                    sts_f32(at_row + (j + 1) * NT * 32, row_sum);
                u.omin[nt][e][j] = 0.0f;
            }
            u.m[nt][e] = __uint_as_float(0xff800000u);
            u.l[nt][e] = 0.0f;
            u.e[nt][e] = kMinExp;
        }
    }
    u.raised = 0u;
    u.one_e = true;
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float zero[8] = {};
            tmem_st8(u.tmem + (c * NT + nt) * 8, zero);
        }
}

// A tile of 32 keys.  Thread (g, t) holds scores of keys 16 mt + g (i < 2) and 16 mt + 8 + g (i >= 2) for
// rows 2t (i even) and 2t + 1.
template <int NT, int NG>
__device__ __forceinline__ void take_tile(Unit<NT, NG> &u, const Kv4AttnArgs &a, const Sizes &z, const Note &at,
                                          uint32_t kb, uint32_t qb, int lane)
{
    const int g = lane >> 2, t = lane & 3;
    const uint32_t vb = kb + kTile * 64, ksb = kb + scales_at(), vsb = ksb + kTile * 4 * NG;
    const float ninf = __uint_as_float(0xff800000u);
    // every row sees every key of the tile: the last key for the first row, the first for the last
    const int v0 = at.tile * kTile, v1 = v0 + kTile - 1;
    const int p0 = v0 < at.ns ? v0 : v0 + at.skip, p1 = v1 < at.ns ? v1 : v1 + at.skip;
    const bool all = at.valid == 0xffffffffu && p1 <= at.n - a.q_len &&
                     (a.window == 0 || p1 < a.n_sink ||
                      at.n - 1 - (p0 < a.n_sink ? (int)a.n_sink : p0) < a.window);
    const bool plain = all && u.one_e;
    float s[NT][2][4];
    // ---- scores, but for fac -----------------------------------------------------------------------
    {
        uint32_t sc[2][2][NG], lo[2][4], hi[2][4];  // words of chunk c of keys g and g + 8
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            const uint32_t from = kb + chunk_at(mt * 16 + (lane & 7), lane >> 3);
            ldmatrix_x4(lo[mt], from);
            ldmatrix_x4(hi[mt], from + 8 * 64);
            lds_scales<NG>(sc[mt][0], ksb + (mt * 16 + g) * 4 * NG);
            lds_scales<NG>(sc[mt][1], ksb + (mt * 16 + g + 8) * 4 * NG);
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            float acc[NT][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[nt][mt][i] = 0.0f;
#pragma unroll
            for (int c = j * (4 / NG); c < (j + 1) * (4 / NG); ++c) {
                uint32_t q[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if constexpr (NT == 1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            q[nt][i] = u.q[0][c][i];
                    } else {
                        const uint4 w = lds128(qb + ((nt * 4 + c) * 32 + lane) * 16);
                        q[nt][0] = w.x, q[nt][1] = w.y, q[nt][2] = w.z, q[nt][3] = w.w;
                    }
                }
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t wl = lo[mt][c] >> (8 * h), wh = hi[mt][c] >> (8 * h);
                        const uint32_t f[4] = {wl & 0x000f000fu, wh & 0x000f000fu, wl & 0x00f000f0u,
                                               wh & 0x00f000f0u};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<true>(acc[nt][mt], f, q[nt][2 * h], q[nt][2 * h + 1]);
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float2 qs = make_float2(u.qsum[0][j], u.qsum[1][j]);
                if (NT > 1)
                    qs = lds_f32x2(qb + rows_at(NT) + (((j + 1) * NT + nt) * 8 + 2 * t) * 4);
                const f2 sum = make_f2(qs.x, qs.y);  // of a key's two rows
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t w = sc[mt][h][j];
                        float *x = &s[nt][mt][2 * h];
                        const float *y = &acc[nt][mt][2 * h];
                        const f2 m = splat(bf_hi(w));
                        const f2 z2 = j == 0 ? mul2(m, sum) : fma2(m, sum, make_f2(x[0], x[1]));
                        const f2 r = fma2(splat(bf_lo(w)), make_f2(y[0], y[1]), z2);
                        x[0] = lo_of(r);
                        x[1] = hi_of(r);
                    }
            }
        }
    }
    // ---- what a row does not see; the largest of the values' scales --------------------------------
    // (not of NaN and infinite ones, which show in the output)
    int e_new[NT][2];
    uint32_t sees = 0u;  // of this thread's scores; not used where all are seen
    if (plain) {
        uint32_t w[NG];
        lds_scales<NG>(w, vsb + lane * 4 * NG);
        int top = 0;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int x = (int)(w[j] & 0x7fffu);
            top = max(top, x >= 0x7f80 ? 0 : x);
        }
        top = max(u.e[0][0], (__reduce_max_sync(0xffffffffu, top) >> 7) - 126);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            e_new[nt][0] = e_new[nt][1] = top;
    } else {
        const int kv = at.hr / z.rtiles, r0 = (at.hr - kv * z.rtiles) * NT * 8;
        int highest = kMinExp;
        bool pad[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = r0 + nt * 8 + 2 * t + e;
                const int p = row < z.R ? at.n - a.q_len + row / z.heads : -1;
                pad[nt][e] = p < 0;
                int top = 0;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key = mt * 16 + g + 8 * h, v = v0 + key;
                        const int pos = v < at.ns ? v : v + at.skip;
                        const bool seen = ((at.valid >> key) & 1) && pos <= p &&
                                          (a.window == 0 || p - pos < a.window || pos < a.n_sink);
                        float &x = s[nt][mt][e + 2 * h];
                        x = seen ? x : ninf;
                        sees |= seen ? 1u << (nt * 8 + mt * 4 + e + 2 * h) : 0u;
                        uint32_t w[NG];
                        lds_scales<NG>(w, vsb + key * 4 * NG);
#pragma unroll
                        for (int j = 0; j < NG; ++j) {
                            const int b = (int)(w[j] & 0x7fffu);
                            top = max(top, b >= 0x7f80 || !seen ? 0 : b);
                        }
                    }
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
                // what the row's own scales ask for, at least
                e_new[nt][e] = max(u.e[nt][e] - ((u.raised >> (nt * 2 + e)) & 1u ? kReach : 0), (top >> 7) - 126);
                highest = max(highest, max(u.e[nt][e], e_new[nt][e]));
            }
        // Rows go by the largest of all rows' where that is no more than kReach above what their own scales ask for: a
        // weight has 2^40 in hand, half a step of FP16's smallest being 2^-25 and weights scaled up to 2^15.  (By
        // another row's scales alone an e could rise tile by tile.)
        highest = __reduce_max_sync(0xffffffffu, highest);
        bool one = true;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int least = e_new[nt][e];
                e_new[nt][e] = pad[nt][e] || highest - least <= kReach ? highest : max(u.e[nt][e], least);
                const uint32_t bit = 1u << (nt * 2 + e);
                u.raised = e_new[nt][e] > least ? u.raised | bit : u.raised & ~bit;
                one = one && e_new[nt][e] == highest;
            }
        u.one_e = __all_sync(0xffffffffu, one);
    }
    // ---- maxima and weights -------------------------------------------------------------------------
    float up[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float2 fac = make_float2(u.fac[0], u.fac[1]);
        if (NT > 1)
            fac = lds_f32x2(qb + rows_at(NT) + (nt * 8 + 2 * t) * 4);
        float ref[2], alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(fmaxf(s[nt][0][e], s[nt][0][e + 2]), fmaxf(s[nt][1][e], s[nt][1][e + 2]));
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float mn = fmaxf(u.m[nt][e], mx * (e ? fac.y : fac.x));
            ref[e] = mn == ninf ? 0.0f : mn;
            alpha[e] = exp2_fast(u.m[nt][e] - ref[e]);  // 0 at the first tile
            up[nt][e] = alpha[e] * pow2i(max(u.e[nt][e] - e_new[nt][e], -126));
            u.e[nt][e] = e_new[nt][e];
            u.m[nt][e] = mn;
        }
        const f2 fac2 = make_f2(fac.x, fac.y), ref2 = make_f2(-ref[0], -ref[1]);
        const f2 alpha2 = make_f2(alpha[0], alpha[1]);
        f2 sum = splat(0.0f);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float *x = &s[nt][mt][2 * h];
                const f2 y = fma2(make_f2(x[0], x[1]), fac2, ref2);
                x[0] = exp2_fast(lo_of(y));
                x[1] = exp2_fast(hi_of(y));
                const f2 p = make_f2(x[0], x[1]);
                sum = mt + h == 0 ? p : add2(sum, p);
            }
        sum = fma2(make_f2(u.l[nt][0], u.l[nt][1]), alpha2, sum);
        u.l[nt][0] = lo_of(sum);
        u.l[nt][1] = hi_of(sum);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const f2 x = mul2(make_f2(u.omin[nt][0][j], u.omin[nt][1][j]), alpha2);
            u.omin[nt][0][j] = lo_of(x);
            u.omin[nt][1][j] = hi_of(x);
        }
    }
    uint32_t b[NT][2][NG][2];
    const float vinv = pow2i(15 - u.e[0][0]);
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
        uint32_t sc[2][NG];
        lds_scales<NG>(sc[0], vsb + (mt * 16 + g) * 4 * NG);
        lds_scales<NG>(sc[1], vsb + (mt * 16 + g + 8) * 4 * NG);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const float vs[2] = {bf_lo(sc[0][j]) * vinv, bf_lo(sc[1][j]) * vinv};
            const float vm[2] = {bf_hi(sc[0][j]), bf_hi(sc[1][j])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
                const float(&p)[4] = s[nt][mt];
                if (plain) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const f2 p2 = make_f2(p[2 * h], p[2 * h + 1]), x = mul2(p2, splat(vs[h]));
                        const f2 y = fma2(p2, splat(vm[h]),
                                          make_f2(u.omin[nt][0][j], u.omin[nt][1][j]));
                        w[2 * h] = lo_of(x);
                        w[2 * h + 1] = hi_of(x);
                        u.omin[nt][0][j] = lo_of(y);
                        u.omin[nt][1][j] = hi_of(y);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // a key that is not seen leaves nothing, whatever it holds; NaN in one that is seen shows, also
                        // where its weight is 0 in FP32
                        const bool seen = (sees >> (nt * 8 + mt * 4 + i)) & 1u;
                        w[i] = seen ? p[i] * (bf_lo(sc[i >> 1][j]) * pow2i(15 - u.e[nt][i & 1])) : 0.0f;
                        u.omin[nt][i & 1][j] = seen ? __fmaf_rn(p[i], vm[i >> 1], u.omin[nt][i & 1][j])
                                                    : u.omin[nt][i & 1][j];
                    }
                }
                b[nt][mt][j][0] = movmatrix_trans(pack_f16x2(w[0], w[1]));
                b[nt][mt][j][1] = movmatrix_trans(pack_f16x2(w[2], w[3]));
            }
        }
    }
    // ---- output ------------------------------------------------------------------------------------
    tmem_wait_st();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float o[NT][8];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            tmem_ld8(u.tmem + (c * NT + nt) * 8, o[nt]);
        uint32_t v[4];  // units of chunk c: keys 0-7, 8-15, 16-23, 24-31
        ldmatrix_x4_trans(v, vb + chunk_at(lane, c));
        float acc[NT][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[nt][jj][i] = 0.0f;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const uint32_t wl = v[2 * mt] >> (8 * jj), wh = v[2 * mt + 1] >> (8 * jj);
                const uint32_t f[4] = {wl & 0x000f000fu, wl & 0x00f000f0u, wh & 0x000f000fu,
                                       wh & 0x00f000f0u};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16816<true>(acc[nt][jj], f, b[nt][mt][c * NG / 4][0], b[nt][mt][c * NG / 4][1]);
            }
        tmem_loaded(o);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float *x = &acc[nt][i >> 2][i & 3];
                const f2 y = fma2(make_f2(o[nt][i], o[nt][i + 1]), make_f2(up[nt][0], up[nt][1]),
                                  make_f2(x[0], x[1]));
                o[nt][i] = lo_of(y);
                o[nt][i + 1] = hi_of(y);
            }
            tmem_st8(u.tmem + (c * NT + nt) * 8, o[nt]);
        }
    }
}

// Results of a whole unit, or the part of a cut one.
template <int NT, int NG>
__device__ __forceinline__ void end_unit(Unit<NT, NG> &u, const Kv4AttnArgs &a, const Sizes &z,
                                         const Note &at, bool whole, float *part_o, float *part_ml, int lane)
{
    const int g = lane >> 2, t = lane & 3;
    const int kv = at.hr / z.rtiles, r0 = (at.hr - kv * z.rtiles) * NT * 8;
    tmem_wait_st();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float o[4][8];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            tmem_ld8(u.tmem + (c * NT + nt) * 8, o[c]);
        tmem_loaded(o);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = u.l[nt][e], om[NG];
#pragma unroll
            for (int j = 0; j < NG; ++j)
                om[j] = u.omin[nt][e][j];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
                for (int j = 0; j < NG; ++j)
                    om[j] += __shfl_xor_sync(0xffffffffu, om[j], off);
            }
            const int in_tile = nt * 8 + 2 * t + e, r = r0 + in_tile;
            const bool none = l == 0.0f;
            const float inv = whole ? __fdiv_rn(1.0f, l) : 1.0f;
            const float back = pow2i(u.e[nt][e] - 1);  // (e: up to 128) and 2^(1 + 24 - 15): codes' unit over weights'
            const int i = r / z.heads, head = kv * z.heads + r - i * z.heads;
            const int64_t row = (int64_t)at.b * a.q_len + i;
            uint16_t *out = (uint16_t *)a.out + row * a.out_stride + head * 128 + 4 * g;
            float *po = part_o + in_tile * 128 + 4 * g;
            if (r < z.R) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float d[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = o[c][(j >> 1) * 4 + e + 2 * (j & 1)] * (j & 1 ? 64.0f : 1024.0f);
                        d[j] = none ? 0.0f : __fmaf_rn(x, back, om[c * NG / 4]) * inv;
                    }
                    if (whole)
                        st_global_v2(out + c * 32, pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]));
                    else
                        *reinterpret_cast<float4 *>(po + c * 32) = make_float4(d[0], d[1], d[2], d[3]);
                }
                if (g == 0) {
                    if (!whole)
                        *reinterpret_cast<float2 *>(part_ml + in_tile * 2) =
                            make_float2(u.m[nt][e], l);
                    else if (a.lse)
                        a.lse[row * a.n_q + head] =
                            none ? __uint_as_float(0xff800000u) : (u.m[nt][e] + log2f(l)) * kLn2;
                }
            }
            __syncwarp();
        }
    }
}

// One warp's tiles: `todo` of them from the note `ld` on, every `stride`-th.  Shares: the team's `mine`-th one, units one
// after the other.  A gang (z.gang): some tiles of one unit, left as a part at the warp's own place in shared memory.
template <int NT, int NG>
__device__ __forceinline__ void take_tiles(const Kv4AttnArgs &a, const Sizes &z, uint32_t base, char *own,
                                           Note ld, uint32_t todo, int stride, uint32_t mine, uint32_t tmem, int lane)
{
    constexpr int kStages = stages_of(NT, NG);
    const uint32_t qb = base + kStages * stage_bytes(NG);
    const int kv = ld.hr / z.rtiles;
    // ---- copies --------------------------------------------------------------------------------------
    int64_t entry;
    // table entry of key `lane` of the tile; -1: none.  Nothing is done with it before the tile's copies, a tile later.
    auto load_slot = [&]() {
        const int v = ld.tile * kTile + lane;
        entry = -1;
        if (v < ld.n - ld.skip)
            entry = a.table[ld.b * a.table_stride + (v < ld.ns ? v : v + ld.skip)];
    };
    if (todo > 0)
        load_slot();
    // of a slot: the lane's 16 bytes of one of eight rows, and its scales
    const uint32_t slot_bytes = (uint32_t)a.n_kv * 64u, slot_scales = (uint32_t)a.n_kv * 4u * NG;
    const uint64_t own_bytes = (uint32_t)(kv * 64 + (lane & 3) * 16), own_scales = (uint32_t)(kv * 4 * NG);
    const uint32_t lane_at = chunk_at(lane >> 2, lane & 3);
    auto load_tile = [&](uint32_t j, int put) {  // tile number j
        if (j < todo) {
            const uint32_t to = base + put * stage_bytes(NG);
            const int slot = entry >= 0 && entry < a.num_slots ? (int)entry : -1;  // -1: not to be seen
            ld.valid = __ballot_sync(0xffffffffu, slot >= 0);
#pragma unroll
            for (int i = 0; i < kTile / 8; ++i) {
                const int at_key = __shfl_sync(0xffffffffu, slot, i * 8 + (lane >> 2));
                const uint64_t off = (uint64_t)(uint32_t)max(at_key, 0) * slot_bytes + own_bytes;
                const uint32_t n = at_key >= 0 ? 16u : 0u;
                cp_async16(to + lane_at + i * 512, (const char *)a.cache[0] + off, n);
                cp_async16(to + lane_at + i * 512 + kTile * 64, (const char *)a.cache[1] + off, n);
            }
            const uint64_t off = (uint64_t)(uint32_t)max(slot, 0) * slot_scales + own_scales;
            const uint32_t at = to + scales_at() + lane * 4 * NG, n = slot >= 0 ? 4u * NG : 0u;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if constexpr (NG == 1)
                    cp_async4(at + x * kTile * 4, (const char *)a.scales[x] + off, n);
                else if constexpr (NG == 2)
                    cp_async8(at + x * kTile * 8, (const char *)a.scales[x] + off, n);
                else
                    cp_async16(at + x * kTile * 16, (const char *)a.scales[x] + off, n);
            }
            if (lane == 0) {
                sts128(to + note_at(NG), make_uint4(ld.valid, (uint32_t)ld.b, (uint32_t)ld.hr,
                                                    (uint32_t)ld.tile));
                sts128(to + note_at(NG) + 16, make_uint4((uint32_t)ld.tiles, (uint32_t)ld.n,
                                                         (uint32_t)ld.ns, (uint32_t)ld.skip));
            }
            if (j + 1 < todo) {
                ld.tile += stride;
                if (ld.tile >= ld.tiles) {
                    ld.tile = 0;
                    Keys k;
                    do
                        k = keys_of(a, (uint32_t)++ld.b);
                    while (k.count == 0);  // tiles are left, so keys are
                    ld.n = k.n;
                    ld.ns = k.ns;
                    ld.skip = k.skip;
                    ld.tiles = k.tiles();
                }
                load_slot();
            }
        }
        cp_async_commit();
    };
#pragma unroll 1
    for (int s = 0; s < kStages - 1; ++s)
        load_tile((uint32_t)s, s);
    // ---- tiles ----------------------------------------------------------------------------------------
    Unit<NT, NG> u;
    u.tmem = tmem;
    bool fresh = true, from_start = false;
    int get = 0;
#pragma unroll 1
    for (uint32_t j = 0; j < todo; ++j) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        load_tile(j + kStages - 1, get == 0 ? kStages - 1 : get - 1);
        const uint32_t from = base + get * stage_bytes(NG);
        const uint4 n0 = lds128(from + note_at(NG)), n1 = lds128(from + note_at(NG) + 16);
        const Note at{n0.x, (int)n0.y, (int)n0.z, (int)n0.w, (int)n1.x, (int)n1.y, (int)n1.z, (int)n1.w};
        if (fresh) {
            begin_unit(u, a, z, at, qb, lane);
            from_start = at.tile == 0;
            fresh = false;
        }
        take_tile(u, a, z, at, from, qb, lane);
        const bool last = at.tile + 1 == at.tiles;
        if (j + 1 == todo || (last && !z.gang)) {
            // the share's first unit leaves its part in place 0, a later one in place 1
            const bool first_unit = j <= (uint32_t)at.tile;
            const int64_t part = (int64_t)((mine * z.team + (uint32_t)at.hr) * 2 + (first_unit ? 0 : 1)) * NT * 8;
            float *po = z.gang ? reinterpret_cast<float *>(own) : z.part_o + part * 128;
            float *pm = z.gang ? reinterpret_cast<float *>(own + NT * 8 * 512) : z.part_ml + part * 2;
            if (z.gang) {  // the part takes the place of the tiles
                cp_async_wait<0>();
                __syncwarp();
            }
            end_unit(u, a, z, at, from_start && last && z.gang < 2, po, pm, lane);
            fresh = true;
        }
        get = get + 1 == kStages ? 0 : get + 1;
    }
    cp_async_wait<0>();
    __syncwarp();
}

// A joined row: row r of sequence b and KV head kv, its lane's four columns of the sum o, reference m, sum l.
__device__ __forceinline__ void write_row(const Kv4AttnArgs &a, const Sizes &z, int b, int kv, int r, float m,
                                          float l, const float4 &o, int lane)
{
    const int i = r / z.heads, head = kv * z.heads + r - i * z.heads;
    const int64_t row = (int64_t)b * a.q_len + i;
    const bool none = l == 0.0f;
    const float inv = none ? 0.0f : __fdiv_rn(1.0f, l);
    st_global_v2((uint16_t *)a.out + row * a.out_stride + head * 128 + lane * 4,
                 pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (a.lse && lane == 0)
        a.lse[row * a.n_q + head] = none ? __uint_as_float(0xff800000u) : (m + log2f(l)) * kLn2;
}

template <int NT, int NG>
__global__ void __launch_bounds__(warps_of(NT, NG) * 32, 1) kv4_attn_kernel(const Kv4AttnArgs a, const Sizes z)
{
    extern __shared__ __align__(128) char smem[];
    __shared__ uint32_t s_before[kScan];
    __shared__ uint32_t s_warp[kScan / 32];
    __shared__ uint32_t s_tmem;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // Tensor memory is asked for behind the kernels before: a block that held columns while it waits for their end could
    // keep one of their blocks from its own, and both would wait for ever.  The next kernel may start only when every
    // block here has its columns, for the same reason.  No more than the warps use, since blocks of few warps, and those
    // of the next call, may share an SM.
    pdl_wait();
    const uint32_t columns = tmem_columns((blockDim.x / 32 + 3) / 4 * NT * 32);
    if (warp == 0)
        tmem_alloc(&s_tmem, columns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // a warp reaches 32 lanes, by its number; those with the same lanes have columns next to each other
    const uint32_t tmem = s_tmem + ((uint32_t)(warp & 3) << 21) + (uint32_t)(warp >> 2) * NT * 32;
    pdl_launch_dependents();
    const uint32_t warps = blockDim.x / 32;
    char *own = smem + warp * warp_bytes(NT, NG);
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(own);
    // Gangs: each `gang` warps of a block take a unit whole, every gang-th tile a warp.  Shares: `active` of the teams
    // have one, and as many teams' warps work at a time as there are; few teams are spread over all places.
    uint32_t total = 0, share = 1, active = 0;
    if (!z.gang) {
        total = scan_tiles(a, z, s_before, s_warp);
        share = (total + z.teams - 1) / z.teams;
        active = total > 0 ? (total + share - 1) / share : 0;
    }
    const uint32_t gang = z.gang ? z.gang : 1, in_block = warp / gang, i = warp - in_block * gang;
    const uint32_t at_once = warps / gang, all = z.gang ? (uint32_t)a.B * z.team : z.teams * z.team;
    auto meet = [&]() {
        if (gang > 1)
            named_sync(1 + (int)in_block, (int)gang * 32);
        else
            __syncwarp();
    };
#pragma unroll 1
    for (uint32_t v = blockIdx.x * at_once + in_block; v < all; v += gridDim.x * at_once) {
        const uint32_t place = v / z.team;
        Note ld;
        ld.hr = (int)(v - place * z.team);
        uint32_t b = place, mine = 0, start = 0, cum = 0, todo = 0;
        if (!z.gang) {
            mine = (place * active + z.teams - 1) / z.teams;
            if (mine >= active || mine * z.teams / active != place)
                continue;
            start = mine * share;
            todo = min(share, total - start);
            uint32_t lo = 0;  // the last thread's run that starts at or before `start`
#pragma unroll 1
            for (int step = kScan / 2; step > 0; step /= 2)
                if (s_before[lo + step] <= start)
                    lo += step;
            cum = s_before[lo];
            b = lo * z.per;
        }
        Keys k = keys_of(a, b);
#pragma unroll 1
        while (!z.gang && start >= cum + (uint32_t)k.tiles()) {
            cum += (uint32_t)k.tiles();
            k = keys_of(a, ++b);
        }
        ld.b = (int)b;
        ld.n = k.n;
        ld.ns = k.ns;
        ld.skip = k.skip;
        ld.tiles = k.tiles();
        ld.tile = z.gang ? (int)i : (int)(start - cum);
        if (z.gang)
            todo = (uint32_t)ld.tiles > i ? ((uint32_t)ld.tiles - i + gang - 1) / gang : 0;
        take_tiles<NT, NG>(a, z, base, own, ld, todo, (int)gang, mine, tmem, lane);
        if (!z.gang || (gang == 1 && todo > 0))
            continue;  // written, as a whole or as parts
        // ---- a gang's parts; a warp without tiles leaves an empty one ------------------------------------------
        float *ml = reinterpret_cast<float *>(own + NT * 8 * 512);
        if (todo == 0)
            for (int r = lane; r < NT * 8; r += 32)
                *reinterpret_cast<float2 *>(ml + r * 2) = make_float2(__uint_as_float(0xff800000u), 0.0f);
        meet();
        const int kv = ld.hr / z.rtiles, r0 = (ld.hr - kv * z.rtiles) * NT * 8;
        const char *first = own - i * warp_bytes(NT, NG);
#pragma unroll 1
        for (int r = (int)i; r < NT * 8 && r0 + r < z.R; r += (int)gang) {
            const float ninf = __uint_as_float(0xff800000u);
            float2 part = make_float2(ninf, 0.0f);
            if (lane < (int)gang)
                part = *reinterpret_cast<const float2 *>(first + lane * warp_bytes(NT, NG) + NT * 8 * 512 + r * 8);
            float m = part.x;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            const float f = part.y == 0.0f ? 0.0f : exp2_fast(part.x - (m == ninf ? 0.0f : m));
            float l = part.y * f;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                l += __shfl_xor_sync(0xffffffffu, l, off);
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
            for (int p = 0; p < (int)gang; ++p) {
                const float fp = __shfl_sync(0xffffffffu, f, p);
                if (__shfl_sync(0xffffffffu, part.y, p) == 0.0f)  // an empty part, whose sums need not be there
                    continue;
                const float4 x = *reinterpret_cast<const float4 *>(first + p * warp_bytes(NT, NG) + r * 512 +
                                                                   lane * 16);
                o.x = __fmaf_rn(x.x, fp, o.x);
                o.y = __fmaf_rn(x.y, fp, o.y);
                o.z = __fmaf_rn(x.z, fp, o.z);
                o.w = __fmaf_rn(x.w, fp, o.w);
            }
            write_row(a, z, ld.b, kv, r0 + r, m, l, o, lane);
        }
        meet();  // the parts have been read
    }
    __syncwarp();
    tmem_wait_st();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        tmem_free(s_tmem, columns);
}

// Rows of units that were cut, from their parts; rows of sequences without keys.  z.crew warps (a power of two, up to the
// block's 8) take a row: each every crew-th part, in order, and the crew's sums meet in shared memory, in order.
template <int NT>
__global__ void __launch_bounds__(kScan)
    kv4_join_kernel(const Kv4AttnArgs a, const Sizes z)
{
    __shared__ uint32_t s_before[kScan];
    __shared__ uint32_t s_warp[kScan / 32];
    __shared__ float4 s_o[kScan];
    __shared__ float2 s_ml[kScan / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t crew = z.crew, at_once = kScan / 32 / crew, i_row = warp / crew, i = warp - i_row * crew;
    const float ninf = __uint_as_float(0xff800000u);
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t total = scan_tiles(a, z, s_before, s_warp);
    const uint32_t share = (total + z.teams - 1) / z.teams;
    const uint32_t rows = (uint32_t)a.B * a.q_len * a.n_q;
#pragma unroll 1
    for (uint32_t w = blockIdx.x * at_once; w < rows; w += gridDim.x * at_once) {
        const uint32_t me = w + i_row, row = me / (uint32_t)a.n_q, b = row / (uint32_t)a.q_len;
        const int head = (int)(me - row * a.n_q), kv = head / z.heads;
        const int r = (int)(row - b * a.q_len) * z.heads + head - kv * z.heads;
        const int rt = r / (NT * 8), in_tile = r - rt * NT * 8;
        uint32_t tiles = 0, t0 = 0, w0 = 0, w1 = 0;
        if (me < rows) {
            tiles = (uint32_t)keys_of(a, b).tiles();
            const uint32_t run = b / z.per;
            t0 = s_before[run];
#pragma unroll 1
            for (uint32_t j = run * z.per; j < b; ++j)
                t0 += (uint32_t)keys_of(a, j).tiles();
            if (tiles > 0) {
                w0 = t0 / share;
                w1 = (t0 + tiles - 1) / share;
            }
        }
        const bool cut = w0 != w1;  // the others were written whole, or have no keys
        // part of share n: its place 0 if the unit is the share's first, which all but share w0 have for sure
        auto part = [&](uint32_t n) {
            return (int64_t)((n * z.team + kv * z.rtiles + rt) * 2 + (n * share >= t0 ? 0 : 1)) * NT * 8 +
                   in_tile;
        };
        // running maximum over 32 parts at a time
        float m = ninf, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
        for (uint32_t n0 = w0 + i; cut && n0 <= w1; n0 += 32 * crew) {
            float2 ml = make_float2(ninf, 0.0f);
            if (n0 + lane * crew <= w1)
                ml = *reinterpret_cast<const float2 *>(z.part_ml + part(n0 + lane * crew) * 2);
            float mx = ml.x;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float mn = fmaxf(m, mx), ref = mn == ninf ? 0.0f : mn, alpha = exp2_fast(m - ref);
            m = mn;
            const float f = exp2_fast(ml.x - ref);
            float lf = ml.y * f;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                lf += __shfl_xor_sync(0xffffffffu, lf, off);
            l = __fmaf_rn(l, alpha, lf);
            o.x *= alpha, o.y *= alpha, o.z *= alpha, o.w *= alpha;
            const int n = (int)min((w1 - n0) / crew + 1, 32u);
#pragma unroll 1
            for (int i1 = 0; i1 < n; i1 += 8) {
                float4 x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (i1 + j < n)
                        x[j] = *reinterpret_cast<const float4 *>(z.part_o + part(n0 + (i1 + j) * crew) * 128 +
                                                                 lane * 4);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float fj = __shfl_sync(0xffffffffu, f, i1 + j);
                    o.x = __fmaf_rn(x[j].x, fj, o.x);
                    o.y = __fmaf_rn(x[j].y, fj, o.y);
                    o.z = __fmaf_rn(x[j].z, fj, o.z);
                    o.w = __fmaf_rn(x[j].w, fj, o.w);
                }
            }
        }
        if (crew > 1) {
            s_o[threadIdx.x] = o;
            if (lane == 0)
                s_ml[warp] = make_float2(m, l);
            __syncthreads();
            if (i == 0) {
#pragma unroll 1
                for (uint32_t j = 1; j < crew; ++j) {
                    const float2 ml = s_ml[warp + j];
                    const float4 x = s_o[threadIdx.x + 32 * j];
                    const float mn = fmaxf(m, ml.x), ref = mn == ninf ? 0.0f : mn;
                    const float fa = exp2_fast(m - ref), fb = exp2_fast(ml.x - ref);
                    m = mn;
                    l = __fmaf_rn(l, fa, ml.y * fb);
                    o.x = __fmaf_rn(o.x, fa, x.x * fb);
                    o.y = __fmaf_rn(o.y, fa, x.y * fb);
                    o.z = __fmaf_rn(o.z, fa, x.z * fb);
                    o.w = __fmaf_rn(o.w, fa, x.w * fb);
                }
            }
            __syncthreads();
        }
        if (i == 0 && me < rows && (cut || tiles == 0))
            write_row(a, z, (int)b, kv, r, m, l, o, lane);
    }
}

template <int NT, int NG>
cudaError_t launch(Kv4AttnArgs a, const Kv4AttnPlan &p, cudaStream_t stream)
{
    if (a.num_slots == 0)  // nothing is read: any address does
        a.cache[0] = a.cache[1] = (const uint8_t *)a.workspace,
        a.scales[0] = a.scales[1] = a.workspace;
    Sizes z;
    z.heads = p.heads;
    z.R = p.R;
    z.rtiles = p.rtiles;
    z.team = (uint32_t)(a.n_kv * p.rtiles);
    z.teams = (uint32_t)p.teams;
    z.gang = (uint32_t)p.gang;
    z.per = ((uint32_t)a.B + kScan - 1) / kScan;
    z.part_o = (float *)a.workspace;
    z.part_ml = z.part_o + (int64_t)z.teams * z.team * 2 * NT * 8 * 128;
    constexpr int smem = warps_of(NT, NG) * warp_bytes(NT, NG);
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !done[dev])) {
        e = cudaFuncSetAttribute(kv4_attn_kernel<NT, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 smem);
        if (e == cudaSuccess && dev < 64)
            done[dev] = true;
    }
    if (e == cudaSuccess)
        e = launch_pdl(kv4_attn_kernel<NT, NG>, dim3(p.ctas), dim3(p.warps * 32),
                       (size_t)p.warps * warp_bytes(NT, NG), stream, a, z);
    if (e == cudaSuccess && p.gang == 0) {
        // few rows, which may have many parts: a block each
        const int64_t rows = (int64_t)a.B * a.q_len * a.n_q;
        z.crew = rows <= 4 * kSms ? 8 : (rows <= 16 * kSms ? 2 : 1);
        const int64_t at_once = kScan / 32 / z.crew, blocks = (rows + at_once - 1) / at_once;
        e = launch_pdl(kv4_join_kernel<NT>, dim3((unsigned)(blocks < kSms * 8 ? blocks : kSms * 8)),
                       dim3(kScan), 0, stream, a, z);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int NT>
cudaError_t launch_groups(const Kv4AttnArgs &a, const Kv4AttnPlan &p, cudaStream_t stream)
{
    return a.group == 128  ? launch<NT, 1>(a, p, stream)
           : a.group == 64 ? launch<NT, 2>(a, p, stream)
                           : launch<NT, 4>(a, p, stream);
}

}  // namespace

cudaError_t launch_kv4_attn(const Kv4AttnArgs &a, const Kv4AttnPlan &p, cudaStream_t stream)
{
    return p.nt == 1   ? launch_groups<1>(a, p, stream)
           : p.nt == 2 ? launch_groups<2>(a, p, stream)
                       : launch_groups<3>(a, p, stream);
}

}  // namespace beam
