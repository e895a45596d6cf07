// kv4_attn.cu -- attention of a decode batch over a KV cache held in 4 bits (sm_103a).
//
// A key is 64 bytes of codes and 4 to 16 of scales for its 128 columns, so the kernel is bound by memory only
// if a code costs next to nothing to unpack.  Two things see to that.
//  - A 16-bit word whose low bits are a code c is the FP16 value c 2^-24 (or 16 c 2^-24 for a code in bits
//    4-7): masking a 32-bit word of eight codes, once as it stands and once shifted by 8, gives the four
//    register pairs that a matrix instruction takes, exactly.  The factor 16 of every second pair goes into
//    the query (scaled by 1/16 there) and out of the result's rows.
//  - Codes multiply first and scales after: s = scale <q, c> + minimum sum q, with FP32 sums of exact
//    products, and out = sum (p scale) c + sum p minimum.
// Both products take the cache as the left operand, whose rows are keys (Q K^T) or columns (V^T P^T), and up
// to 24 query rows of a KV head as the right one, so that few rows waste little: ldmatrix hands out the keys'
// words, and with a transpose the values' (a 16-bit unit is four columns of a key).
//
// Every warp works alone: it owns an even share of all units' tiles of 64 keys, one after the other, copies
// them with cp.async a few tiles ahead into its own part of shared memory, and carries the running maximum,
// sum and output of the unit at hand.  A unit is a sequence, a KV head and a tile of query rows; one that is
// cut between warps leaves parts (FP32 maximum, sum, output) that a second kernel joins in order.

#include <cuda_fp16.h>

#include "beam_device.cuh"
#include "decode/decode_mma.cuh"
#include "draft_kernels.h"

namespace beam {
namespace {

constexpr int kSms = 152;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 64;  // keys
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMinExp = -100;

struct Sizes {
    int32_t heads, R, rtiles;
    int32_t warps;          // of the first kernel
    float *part_o;          // [warps][2][8 * NT][128]
    float *part_ml;         // [warps][2][8 * NT][2]
};

__host__ __device__ constexpr int stages_of(int NG) { return NG == 4 ? 2 : 3; }
__host__ __device__ constexpr int stage_bytes(int NG) { return 2 * kTile * 64 + 2 * kTile * 4 * NG + 16; }

// The keys that any row of a sequence sees, in a list of its own: first the `ns` sinks, then those from
// ns + skip on.
struct Keys {
    int n, ns, skip, count;
};

__device__ __forceinline__ Keys keys_of(const Kv4AttnArgs &a, int64_t b)
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

__device__ __forceinline__ int64_t tiles_of(const Keys &k) { return (k.count + (int64_t)kTile - 1) / kTile; }

// Tiles of all units in front of each thread's run of sequences, and of all.  `per` sequences a thread.
__device__ __forceinline__ int64_t scan_tiles(const Kv4AttnArgs &a, const Sizes &z, int64_t *s_before,
                                              int64_t *s_warp, int64_t per)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t own = 0;
    for (int64_t b = threadIdx.x * per; b < (threadIdx.x + 1) * per && b < a.B; ++b)
        own += tiles_of(keys_of(a, b));
    own *= (int64_t)a.n_kv * z.rtiles;
    int64_t s = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off)
            s += o;
    }
    if (lane == 31)
        s_warp[warp] = s;
    __syncthreads();
    int64_t total = 0, before = s - own;
    for (int i = 0; i < kWarps; ++i) {
        before += i < warp ? s_warp[i] : 0;
        total += s_warp[i];
    }
    s_before[threadIdx.x] = before;
    __syncthreads();
    return total;
}

// Where a warp stands: a tile of a unit.
struct At {
    int64_t b;
    int hr;    // KV head * rtiles + row tile
    int tile, tiles;
    Keys k;
};

__device__ __forceinline__ void advance(At &p, const Kv4AttnArgs &a, int hrs)
{
    if (++p.tile < p.tiles)
        return;
    p.tile = 0;
    if (++p.hr < hrs)
        return;
    p.hr = 0;
    do {
        if (++p.b >= a.B)
            return;
        p.k = keys_of(a, p.b);
        p.tiles = (int)tiles_of(p.k);
    } while (p.tiles == 0);
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

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

template <int NT, int NG>
struct Unit {
    // query, FP16: columns c*32 + t*8 + {j, j + 4} of row g, j = 0..3 (odd j: a sixteenth)
    uint32_t q[NT][4][4];
    float fac[NT][2];        // rows 2t, 2t+1: what a sum of products is scaled by
    float qsum[NT][2][NG];   // sums of the query's columns by group, scaled
    int p[NT][2];            // places of the rows in the sequence (-1: padding)
    float m[NT][2], l[NT][2], omin[NT][2][NG];
    int e[NT][2];            // scales seen are below 2^e
    float o[NT][4][2][4];
};

template <int NT, int NG>
__device__ __forceinline__ void begin_unit(Unit<NT, NG> &u, const Kv4AttnArgs &a, const Sizes &z,
                                           const At &at, int lane)
{
    const int g = lane >> 2, t = lane & 3;
    const int kv = at.hr / z.rtiles, r0 = (at.hr - kv * z.rtiles) * NT * 8;
    const float sm = a.sm_scale * kLog2e;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + nt * 8 + g;
        const int i = r / z.heads;
        uint4 v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            v[c] = r < z.R ? ld_plain((const uint16_t *)a.q + (at.b * a.q_len + i) * a.q_stride +
                                      (kv * z.heads + r - i * z.heads) * 128 + c * 32 + t * 8)
                           : make_uint4(0, 0, 0, 0);
        uint32_t mx = 0u;
        float sum[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            sum[c] = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float x = bf_lo(word(v[c], w)), y = bf_hi(word(v[c], w));
                mx = max(mx, max(__float_as_uint(x) & 0x7fffffffu, __float_as_uint(y) & 0x7fffffffu));
                sum[c] += x + y;
            }
        }
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, off));
#pragma unroll
            for (int c = 0; c < 4; ++c)
                sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], off);
        }
        // the row's power of two: its largest element to [2^14, 2^15)
        int k = (mx >> 23) == 255u || mx == 0u ? 0 : 141 - (int)(mx >> 23);
        k = min(k, 60);
        const float f = pow2i(k);
        // a sum of products of q 2^k and c 2^-24, back
        const float inv = pow2i(-k);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float x[8];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                x[2 * w] = bf_lo(word(v[c], w)) * f;
                x[2 * w + 1] = bf_hi(word(v[c], w)) * f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float h = j & 1 ? 0.0625f : 1.0f;
                u.q[nt][c][j] = pack_f16x2(x[j] * h, x[j + 4] * h);
            }
        }
        float gs[NG];
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            gs[j] = 0.0f;
#pragma unroll
            for (int c = 0; c < 4 / NG; ++c)
                gs[j] += sum[j * (4 / NG) + c];
            gs[j] *= sm;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int from = (2 * t + e) * 4;  // a lane whose g is this row
            u.fac[nt][e] = __shfl_sync(0xffffffffu, inv, from) * 16777216.0f * sm;
#pragma unroll
            for (int j = 0; j < NG; ++j)
                u.qsum[nt][e][j] = __shfl_sync(0xffffffffu, gs[j], from);
            const int row = r0 + nt * 8 + 2 * t + e;
            u.p[nt][e] = row < z.R ? at.k.n - a.q_len + row / z.heads : -1;
            u.m[nt][e] = __uint_as_float(0xff800000u);
            u.l[nt][e] = 0.0f;
            u.e[nt][e] = kMinExp;
#pragma unroll
            for (int j = 0; j < NG; ++j)
                u.omin[nt][e][j] = 0.0f;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int i2 = 0; i2 < 4; ++i2)
                    u.o[nt][c][jj][i2] = 0.0f;
    }
}

// MT times 16 keys of the tile, from key k0 of it on.  Masked: some row may not see some of them.
template <int NT, int NG, int MT, bool Masked>
__device__ __forceinline__ void keys_step(Unit<NT, NG> &u, const Kv4AttnArgs &a, const At &at,
                                          uint32_t base, int k0, uint64_t valid, int lane)
{
    const int g = lane >> 2;
    const uint32_t kb = base, vb = base + kTile * 64, ksb = vb + kTile * 64,
                   vsb = ksb + kTile * 4 * NG;
    const float ninf = __uint_as_float(0xff800000u);
    float s[NT][MT][4];
    // ---- scores ----------------------------------------------------------------------------------
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        uint32_t lo[4], hi[4];  // words of chunk c (32 columns) of keys g and g + 8
        {
            const int key = k0 + mt * 16 + (lane & 7), c = lane >> 3;
            ldmatrix_x4(lo, kb + key * 64 + ((c ^ ((key >> 1) & 3)) << 4));
            ldmatrix_x4(hi, kb + (key + 8) * 64 + ((c ^ ((key >> 1) & 3)) << 4));
        }
        float acc[NT][NG][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < NG; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[nt][j][i] = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t wl = lo[c] >> (8 * h), wh = hi[c] >> (8 * h);
                const uint32_t f[4] = {wl & 0x000f000fu, wh & 0x000f000fu, wl & 0x00f000f0u,
                                       wh & 0x00f000f0u};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16816<true>(acc[nt][c * NG / 4], f, u.q[nt][c][2 * h], u.q[nt][c][2 * h + 1]);
            }
        uint32_t sc[2][NG];
        lds_scales<NG>(sc[0], ksb + (k0 + mt * 16 + g) * 4 * NG);
        lds_scales<NG>(sc[1], ksb + (k0 + mt * 16 + g + 8) * 4 * NG);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x = 0.0f;
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    const uint32_t w = sc[i >> 1][j];
                    x = __fmaf_rn(bf_lo(w) * u.fac[nt][i & 1], acc[nt][j][i],
                                  __fmaf_rn(bf_hi(w), u.qsum[nt][i & 1][j], x));
                }
                if constexpr (Masked) {
                    const int key = k0 + mt * 16 + g + 8 * (i >> 1);
                    const int v = at.tile * kTile + key;
                    const int pos = v < at.k.ns ? v : v + at.k.skip;
                    const int p = u.p[nt][i & 1];
                    const bool seen = ((valid >> key) & 1) && pos <= p &&
                                      (a.window == 0 || p - pos < a.window || pos < a.n_sink);
                    x = seen ? x : ninf;
                }
                s[nt][mt][i] = x;
            }
    }
    // ---- maxima: of the scores, and of the values' scales ----------------------------------------
    int top = 0;  // largest scale's bits (not of NaN and infinite ones, which show in the output)
    if constexpr (!Masked) {
#pragma unroll
        for (int i = 0; i < MT / 2; ++i) {
            uint32_t w[NG];
            lds_scales<NG>(w, vsb + (k0 + i * 32 + lane) * 4 * NG);
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const int x = (int)(w[j] & 0x7fffu);
                top = max(top, x >= 0x7f80 ? 0 : x);
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
    }
    bool moved = false;
    float up[NT][2], mref[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float mx = ninf;
            int tp = top;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                mx = fmaxf(mx, fmaxf(s[nt][mt][e], s[nt][mt][e + 2]));
            if constexpr (Masked) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t w[NG];
                        lds_scales<NG>(w, vsb + (k0 + mt * 16 + g + 8 * h) * 4 * NG);
#pragma unroll
                        for (int j = 0; j < NG; ++j) {
                            const int x = (int)(w[j] & 0x7fffu);
                            tp = max(tp, x >= 0x7f80 || s[nt][mt][e + 2 * h] == ninf ? 0 : x);
                        }
                    }
            }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                if constexpr (Masked)
                    tp = max(tp, __shfl_xor_sync(0xffffffffu, tp, off));
            }
            const float mn = fmaxf(u.m[nt][e], mx);
            const int en = max(u.e[nt][e], (tp >> 7) - 126);
            const float alpha = mn == u.m[nt][e] ? 1.0f : exp2_fast(u.m[nt][e] - mn);
            moved = moved || mn != u.m[nt][e] || en != u.e[nt][e];
            up[nt][e] = alpha * (en - u.e[nt][e] > 120 ? 0.0f : pow2i(u.e[nt][e] - en));
            u.l[nt][e] *= alpha;
#pragma unroll
            for (int j = 0; j < NG; ++j)
                u.omin[nt][e][j] *= alpha;
            u.m[nt][e] = mn;
            u.e[nt][e] = en;
            mref[nt][e] = mn == ninf ? 0.0f : mn;
        }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        u.o[nt][c][jj][i] *= up[nt][i & 1];
    }
    // ---- weights and the values' product -----------------------------------------------------------
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        uint32_t sc[2][NG];
        lds_scales<NG>(sc[0], vsb + (k0 + mt * 16 + g) * 4 * NG);
        lds_scales<NG>(sc[1], vsb + (k0 + mt * 16 + g + 8) * 4 * NG);
        uint32_t b[NT][NG][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = exp2_fast(s[nt][mt][i] - mref[nt][i & 1]);
                u.l[nt][i & 1] += p[i];
            }
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x = sc[i >> 1][j];
                    const bool none = Masked && p[i] == 0.0f;
                    // two factors, each in range: the scale up to FP16's, then the weight
                    w[i] = none ? 0.0f : p[i] * (bf_lo(x) * pow2i(15 - u.e[nt][i & 1]));
                    u.omin[nt][i & 1][j] =
                        none ? u.omin[nt][i & 1][j] : __fmaf_rn(p[i], bf_hi(x), u.omin[nt][i & 1][j]);
                }
                b[nt][j][0] = movmatrix_trans(pack_f16x2(w[0], w[1]));
                b[nt][j][1] = movmatrix_trans(pack_f16x2(w[2], w[3]));
            }
        }
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
            uint32_t v[4];  // chunk 2 c2: keys 0-7, 8-15; chunk 2 c2 + 1: the same
            {
                const int key = k0 + mt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
                const int c = 2 * c2 + (lane >> 4);
                ldmatrix_x4_trans(v, vb + key * 64 + ((c ^ ((key >> 1) & 3)) << 4));
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = 2 * c2 + h;
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const uint32_t wl = v[2 * h] >> (8 * jj), wh = v[2 * h + 1] >> (8 * jj);
                    const uint32_t f[4] = {wl & 0x000f000fu, wl & 0x00f000f0u, wh & 0x000f000fu,
                                           wh & 0x00f000f0u};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816<true>(u.o[nt][c][jj], f, b[nt][c * NG / 4][0], b[nt][c * NG / 4][1]);
                }
            }
        }
    }
}

// Results of a whole unit, or the part of a cut one.
template <int NT, int NG>
__device__ __forceinline__ void end_unit(Unit<NT, NG> &u, const Kv4AttnArgs &a, const Sizes &z,
                                         const At &at, bool whole, int64_t part, int lane)
{
    const int g = lane >> 2, t = lane & 3;
    const int kv = at.hr / z.rtiles, r0 = (at.hr - kv * z.rtiles) * NT * 8;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
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
            if (r >= z.R)
                continue;
            const float back = pow2i(u.e[nt][e]);  // and 2^(24 - 15): codes' unit over weights' scaling
            const float m = u.m[nt][e];
            if (whole) {
                const int i = r / z.heads, head = kv * z.heads + r - i * z.heads;
                const int64_t row = at.b * a.q_len + i;
                const float inv = __fdiv_rn(1.0f, l);
                uint16_t *out = (uint16_t *)a.out + row * a.out_stride + head * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float d[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = u.o[nt][c][j >> 1][e + 2 * (j & 1)] * (j & 1 ? 32.0f : 512.0f);
                        d[j] = l == 0.0f ? 0.0f : __fmaf_rn(x, back, om[c * NG / 4]) * inv;
                    }
                    st_global_v2(out + c * 32 + 4 * g, pack_bf16x2(d[0], d[1]),
                                 pack_bf16x2(d[2], d[3]));
                }
                if (a.lse && g == 0)
                    a.lse[row * a.n_q + head] =
                        l == 0.0f ? __uint_as_float(0xff800000u) : (m + log2f(l)) * kLn2;
            } else {
                float *out = z.part_o + (part * NT * 8 + in_tile) * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float d[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = u.o[nt][c][j >> 1][e + 2 * (j & 1)] * (j & 1 ? 32.0f : 512.0f);
                        d[j] = __fmaf_rn(x, back, om[c * NG / 4]);
                    }
                    *reinterpret_cast<float4 *>(out + c * 32 + 4 * g) =
                        make_float4(d[0], d[1], d[2], d[3]);
                }
                if (g == 0)
                    *reinterpret_cast<float2 *>(z.part_ml + (part * NT * 8 + in_tile) * 2) =
                        make_float2(m, l);
            }
        }
}

// Slots of keys `lane` and `lane + 32` of a tile; -1: not to be seen.
__device__ __forceinline__ void load_slots(int (&slot)[2], const Kv4AttnArgs &a, const At &p, int lane)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int v = p.tile * kTile + i * 32 + lane;
        slot[i] = -1;
        if (v < p.k.count) {
            const int64_t s = a.table[p.b * a.table_stride + (v < p.k.ns ? v : v + p.k.skip)];
            slot[i] = s >= 0 && s < a.num_slots ? (int)s : -1;
        }
    }
}

template <int NG>
__device__ __forceinline__ void copy_tile(uint32_t base, const int (&slot)[2], const Kv4AttnArgs &a, int kv,
                                          int lane)
{
    const uint64_t valid = (uint64_t)__ballot_sync(0xffffffffu, slot[0] >= 0) |
                           (uint64_t)__ballot_sync(0xffffffffu, slot[1] >= 0) << 32;
#pragma unroll
    for (int i = 0; i < kTile / 8; ++i) {
        const int key = i * 8 + (lane >> 2), c = lane & 3;
        const int s = __shfl_sync(0xffffffffu, slot[i / 4], key & 31);
        const int64_t off = s >= 0 ? ((int64_t)s * a.n_kv + kv) * 64 + c * 16 : 0;
        const uint32_t at = base + key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
        cp_async16(at, a.cache[0] + off, s >= 0 ? 16u : 0u);
        cp_async16(at + kTile * 64, a.cache[1] + off, s >= 0 ? 16u : 0u);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t off = slot[i] >= 0 ? ((int64_t)slot[i] * a.n_kv + kv) * 4 * NG : 0;
        const uint32_t n = slot[i] >= 0 ? 4u * NG : 0u;
        const uint32_t at = base + kTile * 128 + (i * 32 + lane) * 4 * NG;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const char *src = (const char *)a.scales[x] + off;
            if constexpr (NG == 1)
                cp_async4(at + x * kTile * 4 * NG, src, n);
            else if constexpr (NG == 2)
                cp_async8(at + x * kTile * 4 * NG, src, n);
            else
                cp_async16(at + x * kTile * 4 * NG, src, n);
        }
    }
    if (lane == 0)
        asm volatile("st.shared.u64 [%0], %1;" ::"r"(base + kTile * 128 + 2 * kTile * 4 * NG), "l"(valid)
                     : "memory");
}

template <int NT, int NG>
__global__ void __launch_bounds__(kThreads, 1)
    kv4_attn_kernel(const Kv4AttnArgs a, const Sizes z, int64_t per)
{
    extern __shared__ __align__(128) char smem[];
    __shared__ int64_t s_before[kThreads];
    __shared__ int64_t s_warp[kWarps];
    constexpr int kStages = stages_of(NG);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t total = scan_tiles(a, z, s_before, s_warp, per);
    // neighbouring shares go to different blocks, so that few shares are spread over all SMs
    const int64_t me = (int64_t)warp * gridDim.x + blockIdx.x;
    const int64_t share = (total + z.warps - 1) / z.warps;
    const int64_t start = me * share, end = start + share < total ? start + share : total;
    if (start >= end)
        return;
    const int hrs = a.n_kv * z.rtiles;
    At ld;
    {
        int lo = 0, hi = kThreads - 1;  // the last thread's run that starts at or before `start`
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (s_before[mid] <= start)
                lo = mid;
            else
                hi = mid - 1;
        }
        int64_t cum = s_before[lo];
        for (ld.b = lo * per;; ++ld.b) {
            ld.k = keys_of(a, ld.b);
            const int64_t n = tiles_of(ld.k) * hrs;
            if (start < cum + n) {
                ld.tiles = (int)tiles_of(ld.k);
                ld.hr = (int)((start - cum) / ld.tiles);
                ld.tile = (int)((start - cum) - (int64_t)ld.hr * ld.tiles);
                break;
            }
            cum += n;
        }
    }
    At cp = ld;
    const uint32_t base =
        (uint32_t)__cvta_generic_to_shared(smem) + warp * kStages * stage_bytes(NG);
    int64_t to_load = end - start;
    int slot[2];
    load_slots(slot, a, ld, lane);
    auto load_next = [&](int stage) {
        if (to_load > 0) {
            copy_tile<NG>(base + stage * stage_bytes(NG), slot, a, ld.hr / z.rtiles, lane);
            if (--to_load > 0) {
                advance(ld, a, hrs);
                load_slots(slot, a, ld, lane);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s)
        load_next(s);

    Unit<NT, NG> u;
    bool fresh = true, from_start = false;
    int stage = 0;
    for (int64_t j = start; j < end; ++j) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        load_next(stage == 0 ? kStages - 1 : stage - 1);
        if (fresh) {
            begin_unit(u, a, z, cp, lane);
            from_start = cp.tile == 0;
            fresh = false;
        }
        const uint32_t at = base + stage * stage_bytes(NG);
        uint64_t valid;
        asm volatile("ld.shared.u64 %0, [%1];"
                     : "=l"(valid)
                     : "r"(at + kTile * 128 + 2 * kTile * 4 * NG)
                     : "memory");
        // every row sees every key of the tile: the last key for the first row, the first for the last
        const int v0 = cp.tile * kTile, v1 = v0 + kTile - 1;
        const int64_t p0 = v0 < cp.k.ns ? v0 : v0 + cp.k.skip, p1 = v1 < cp.k.ns ? v1 : v1 + cp.k.skip;
        const bool all = valid == ~0ull && p1 <= cp.k.n - a.q_len &&
                         (a.window == 0 || p1 < a.n_sink ||
                          cp.k.n - 1 - (p0 < a.n_sink ? a.n_sink : p0) < a.window);
        constexpr int MT = NT == 1 ? 4 : 2;
#pragma unroll 1
        for (int k0 = 0; k0 < kTile; k0 += MT * 16) {
            if (all)
                keys_step<NT, NG, MT, false>(u, a, cp, at, k0, valid, lane);
            else
                keys_step<NT, NG, MT, true>(u, a, cp, at, k0, valid, lane);
        }
        const bool last = cp.tile + 1 == cp.tiles;
        if (last || j + 1 == end) {
            // the share's first unit leaves its part in place 0, a later one in place 1
            const bool first_unit = j - cp.tile <= start;
            end_unit(u, a, z, cp, from_start && last, me * 2 + (first_unit ? 0 : 1), lane);
            fresh = true;
        }
        if (j + 1 < end)
            advance(cp, a, hrs);
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
}

// Rows of units that were cut, from their parts in order; rows of sequences without keys.  A warp takes a row.
template <int NT>
__global__ void __launch_bounds__(kThreads)
    kv4_join_kernel(const Kv4AttnArgs a, const Sizes z, int64_t per)
{
    __shared__ int64_t s_before[kThreads];
    __shared__ int64_t s_warp[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t total = scan_tiles(a, z, s_before, s_warp, per);
    const int64_t share = (total + z.warps - 1) / z.warps;
    const int64_t rows = (int64_t)a.B * a.q_len * a.n_q;
    for (int64_t w = (int64_t)blockIdx.x * kWarps + warp; w < rows; w += (int64_t)gridDim.x * kWarps) {
        const int64_t row = w / a.n_q;
        const int head = (int)(w - row * a.n_q);
        const int64_t b = row / a.q_len;
        const int kv = head / z.heads;
        const int r = (int)(row - b * a.q_len) * z.heads + head - kv * z.heads;
        const int rt = r / (NT * 8), in_tile = r - rt * NT * 8;
        const int64_t tiles = tiles_of(keys_of(a, b));
        uint16_t *out = (uint16_t *)a.out + row * a.out_stride + head * 128 + lane * 4;
        if (tiles == 0) {
            st_global_v2(out, 0u, 0u);
            if (a.lse && lane == 0)
                a.lse[w] = __uint_as_float(0xff800000u);
            continue;
        }
        int64_t t0 = s_before[b / per];
        for (int64_t i = b / per * per; i < b; ++i)
            t0 += tiles_of(keys_of(a, i)) * a.n_kv * z.rtiles;
        t0 += ((int64_t)kv * z.rtiles + rt) * tiles;
        const int64_t w0 = t0 / share, w1 = (t0 + tiles - 1) / share;
        if (w0 == w1)
            continue;  // written whole
        // part of share i: its place 0 if the unit is the share's first
        auto part = [&](int64_t i) { return (i * 2 + (i * share >= t0 ? 0 : 1)) * NT * 8 + in_tile; };
        // a share that starts inside the unit holds it as its first; only share w0 may start before it
        float m = __uint_as_float(0xff800000u);
        for (int64_t i = w0 + lane; i <= w1; i += 32)
            m = fmaxf(m, z.part_ml[part(i) * 2]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float mref = m == __uint_as_float(0xff800000u) ? 0.0f : m;
        float l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int64_t i0 = w0; i0 <= w1; i0 += 32) {
            float f = 0.0f, lf = 0.0f;
            if (i0 + lane <= w1) {
                const float2 ml = *reinterpret_cast<const float2 *>(z.part_ml + part(i0 + lane) * 2);
                f = exp2_fast(ml.x - mref);
                lf = ml.y * f;
            }
            const int n = w1 - i0 + 1 < 32 ? (int)(w1 - i0 + 1) : 32;
#pragma unroll 8
            for (int i = 0; i < n; ++i) {
                const float4 x =
                    *reinterpret_cast<const float4 *>(z.part_o + part(i0 + i) * 128 + lane * 4);
                const float fi = __shfl_sync(0xffffffffu, f, i);
                l += __shfl_sync(0xffffffffu, lf, i);
                o.x = __fmaf_rn(x.x, fi, o.x);
                o.y = __fmaf_rn(x.y, fi, o.y);
                o.z = __fmaf_rn(x.z, fi, o.z);
                o.w = __fmaf_rn(x.w, fi, o.w);
            }
        }
        const float inv = __fdiv_rn(1.0f, l);
        const bool none = l == 0.0f;
        st_global_v2(out, none ? 0u : pack_bf16x2(o.x * inv, o.y * inv),
                     none ? 0u : pack_bf16x2(o.z * inv, o.w * inv));
        if (a.lse && lane == 0)
            a.lse[w] = none ? __uint_as_float(0xff800000u) : (m + log2f(l)) * kLn2;
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
    z.warps = p.ctas * kWarps;
    z.part_o = (float *)a.workspace;
    z.part_ml = z.part_o + (int64_t)z.warps * 2 * NT * 8 * 128;
    const int64_t per = ((int64_t)a.B + kThreads - 1) / kThreads;
    const int smem = kWarps * stages_of(NG) * stage_bytes(NG);
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
        e = launch_pdl(kv4_attn_kernel<NT, NG>, dim3(p.ctas), dim3(kThreads), smem, stream, a, z, per);
    if (e == cudaSuccess) {
        const int64_t rows = (int64_t)a.B * a.q_len * a.n_q;
        const int64_t blocks = (rows + kWarps - 1) / kWarps;
        e = launch_pdl(kv4_join_kernel<NT>, dim3((unsigned)(blocks < kSms * 8 ? blocks : kSms * 8)),
                       dim3(kThreads), 0, stream, a, z, per);
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

Kv4AttnPlan kv4_attn_plan(int32_t B, int32_t q_len, int32_t n_q, int32_t n_kv, int64_t width,
                          int64_t window, int64_t n_sink)
{
    Kv4AttnPlan p{};
    p.heads = n_q / n_kv;
    p.R = q_len * p.heads;
    const int32_t t8 = (p.R + 7) / 8;
    p.nt = t8 < 3 ? t8 : 3;
    p.rtiles = (t8 + p.nt - 1) / p.nt;
    // no more warps than tiles there can be
    int64_t most = width;
    if (window > 0 && window + q_len + n_sink < width)
        most = window + q_len + n_sink;
    const double tiles = (double)((most + kTile - 1) / kTile) * B * n_kv * p.rtiles;
    p.ctas = tiles < kSms ? (int32_t)(tiles < 1 ? 1 : tiles) : kSms;
    p.bytes = (int64_t)p.ctas * kWarps * 2 * p.nt * 8 * (128 + 2) * 4;
    return p;
}

cudaError_t launch_kv4_attn(const Kv4AttnArgs &a, const Kv4AttnPlan &p, cudaStream_t stream)
{
    return p.nt == 1   ? launch_groups<1>(a, p, stream)
           : p.nt == 2 ? launch_groups<2>(a, p, stream)
                       : launch_groups<3>(a, p, stream);
}

}  // namespace beam
