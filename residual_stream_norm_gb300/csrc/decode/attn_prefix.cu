// attn_prefix.cu -- attention of a decode batch over the slot cache, with a shared prefix (sm_103a).
//
// softmax(q K^T) V over a list of keys is computed in one pass: with the running maximum m, the
// running sum l of exp(s - m) and the running O = sum exp(s - m) v, a larger maximum m' scales l and O
// by exp(m - m').  Parts of a list join by the same rule.  Exponents are taken to base 2, scores
// carry the factor log2(e).
//
// Rows kernel: a warp works on 16 keys at a time for 8 or 16 query rows of one KV head.  It computes
// the transposed products S^T = K Q^T and O^T = V^T P^T, so that the keys fill the 16 rows of the
// matrix instruction and the few query rows its 8 columns.  Each warp copies its own keys (cp.async,
// a gather by slot) into its own stages, so warps meet only when their parts are joined.

#include "decode_kernels.h"
#include "decode_mma.cuh"

namespace beam {
namespace {

constexpr int kD = 128;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kWarpKeys = 16;
constexpr int kTileKeys = kWarps * kWarpKeys;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <bool FP8>
struct RowsConfig {
    static constexpr int kRow = FP8 ? 128 : 256;          // bytes of a cache row of one head
    static constexpr int kChunks = kRow / 16;
    static constexpr int kStages = FP8 ? 4 : 3;
    static constexpr int kTileBytes = kWarpKeys * kRow;   // keys or values of a stage
    static constexpr int kWarpBytes = kStages * 2 * kTileBytes;
    static constexpr int kCtasPerSm = FP8 ? 3 : 2;
    static constexpr int kSmem = kWarps * kWarpBytes;
};

// Where the 16-byte chunk of a key lies in its row of shared memory: eight keys' same chunk fall into
// eight different bank groups (ldmatrix); for FP8 an even and an odd key's chunks 0..3 do as well
// (the 16-byte loads of the keys).
template <bool FP8>
__device__ __forceinline__ int swizzle(int key, int chunk)
{
    return FP8 ? chunk ^ (((key & 1) << 2) | ((key >> 1) & 3)) : chunk ^ (key & 7);
}

// The block whose share [c tot / C, (c + 1) tot / C) contains tile x (C <= tot).
__device__ __forceinline__ int64_t owner(int64_t x, int64_t tot, int64_t ctas)
{
    return ((x + 1) * ctas - 1) / tot;
}

// The keys that any row of a sequence of n entries sees: [first, n).
__device__ __forceinline__ int64_t first_key(int64_t n, int q_len, int64_t window)
{
    const int64_t lo = n - q_len + 1 - window;
    return window > 0 && lo > 0 ? lo : 0;
}

__device__ __forceinline__ int64_t seq_len(const AttnArgs &a, int64_t b)
{
    const int64_t n = a.len[b];
    return n < 0 ? 0 : (n > a.width ? a.width : n);
}

__device__ __forceinline__ int64_t seq_tiles(const AttnArgs &a, int64_t b)
{
    const int64_t n = seq_len(a, b);
    return (n - first_key(n, a.q_len, a.window) + kTileKeys - 1) / kTileKeys;
}

// Factor 2^k that brings a row of largest magnitude bits `mx` (FP32) to [2^14, 2^15), and its
// inverse; 1 for zero, infinite and NaN rows.
__device__ __forceinline__ void f16_row_factor(uint32_t mx, float &f, float &inv)
{
    const int e = (int)(mx >> 23);
    int k = e == 255 || mx == 0u ? 0 : 141 - e;
    k = min(k, 120);
    f = __uint_as_float((uint32_t)(127 + k) << 23);
    inv = __uint_as_float((uint32_t)(127 - k) << 23);
}

// The A fragment of V^T for 16 elements d (tile mt) and the 16 keys of a stage.  FP8: 16-bit units of
// the transposed load are pairs (d, d + 1); after the split, matrix row g is element 2g of the 16
// and row g + 8 element 2g + 1.
template <bool FP8>
__device__ __forceinline__ void load_values(uint32_t (&af)[4], uint32_t vt, int mt, int lane)
{
    using C = RowsConfig<FP8>;
    if constexpr (!FP8) {
        const int key = (lane >> 4) * 8 + (lane & 7), ch = 2 * mt + ((lane >> 3) & 1);
        ldmatrix_x4_trans(af, vt + key * C::kRow + 16 * swizzle<FP8>(key, ch));
    } else {
        uint32_t r[4];
        const int key = lane & 15, ch = (mt & ~1) + (lane >> 4);
        ldmatrix_x4_trans(r, vt + key * C::kRow + 16 * swizzle<FP8>(key, ch));
        const uint32_t r0 = mt & 1 ? r[2] : r[0], r1 = mt & 1 ? r[3] : r[1];
        const uint32_t x0 = e4m3x2_to_f16x2(r0), x1 = e4m3x2_to_f16x2(r0 >> 16);
        const uint32_t y0 = e4m3x2_to_f16x2(r1), y1 = e4m3x2_to_f16x2(r1 >> 16);
        af[0] = __byte_perm(x0, x1, 0x5410), af[1] = __byte_perm(x0, x1, 0x7632);
        af[2] = __byte_perm(y0, y1, 0x5410), af[3] = __byte_perm(y0, y1, 0x7632);
    }
}

// Whether a stage's values hold an infinity or NaN (E4M3 has NaN only: all bits but the sign set).
template <bool FP8>
__device__ __forceinline__ bool tile_has_nonfinite(uint32_t vt, int lane)
{
    bool bad = false;
#pragma unroll 1
    for (int i = lane; i < RowsConfig<FP8>::kTileBytes / 16; i += 32) {
        const uint4 v = lds128(vt + 16 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = word(v, j);
            if constexpr (FP8)
                bad = bad || __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0u;
            else
                bad = bad || __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u) != 0u;
        }
    }
    return __any_sync(0xffffffffu, bad);
}

// Row rr (of `rows`, per KV head): token and head of it.
__device__ __forceinline__ int64_t row_token(const AttnArgs &a, const AttnPlan &p, int64_t rr,
                                             int &i, int &hg)
{
    const uint32_t b = (uint32_t)rr / (uint32_t)p.R;  // B * q_len * n_q < 2^31
    const uint32_t r = (uint32_t)rr - b * p.R;
    i = (int)(r / (uint32_t)p.group);
    hg = (int)r - i * p.group;
    return (int64_t)b * a.q_len + i;
}

template <int NT, bool FP8>
__global__ void __launch_bounds__(kThreads, RowsConfig<FP8>::kCtasPerSm)
    attn_rows_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnPlan p)
{
    using C = RowsConfig<FP8>;
    constexpr int M = 8 * NT;
    extern __shared__ __align__(128) char smem[];
    __shared__ int64_t s_start[3];  // sequence of the first tile, its first tile, all tiles
    __shared__ float2 s_ml[kWarps][M];
    __shared__ int64_t s_scan[kWarps + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t wbuf = smem_addr(smem) + warp * C::kWarpBytes;
    pdl_launch_dependents();
    pdl_wait();

    // ---- the share of this block ---------------------------------------------------------------
    const int64_t p_units = a.n_kv * p.p_rtiles;
    const int64_t p_total = p_units * p.p_tiles;
    const int64_t per_seq = (int64_t)a.n_kv * p.s_rtiles;
    int64_t *cum = reinterpret_cast<int64_t *>(a.workspace + p.cum_off);
    int64_t total = p_total;
    for (int64_t b0 = 0; b0 < a.B; b0 += kThreads) {  // the sum over the sequences
        const int64_t b = b0 + tid;
        int64_t v = b < a.B ? per_seq * seq_tiles(a, b) : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, v, off);
            if (lane >= off)
                v += o;
        }
        if (lane == 31)
            s_scan[warp] = v;
        __syncthreads();
        int64_t before = 0, sum = 0;
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? s_scan[w] : 0;
            sum += s_scan[w];
        }
        if (blockIdx.x == 0 && b < a.B)
            cum[b + 1] = total + before + v;
        total += sum;
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0)
        cum[0] = p_total;
    const int64_t shares = min((int64_t)p.ctas, total);  // none of them empty
    if (blockIdx.x >= shares)
        return;
    int64_t tile = total * blockIdx.x / shares;
    const int64_t tile_end = total * (blockIdx.x + 1) / shares;
    int64_t b = 0, b_start = p_total;  // sequence of `tile` (once past the prefix), its first tile
    if (tile >= p_total) {
        int64_t run = p_total;
        for (int64_t b0 = 0; b0 < a.B; b0 += kThreads) {
            const int64_t bb = b0 + tid;
            const int64_t own = bb < a.B ? per_seq * seq_tiles(a, bb) : 0;
            int64_t v = own;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, v, off);
                if (lane >= off)
                    v += o;
            }
            if (lane == 31)
                s_scan[warp] = v;
            __syncthreads();
            int64_t before = 0, sum = 0;
            for (int w = 0; w < kWarps; ++w) {
                before += w < warp ? s_scan[w] : 0;
                sum += s_scan[w];
            }
            const int64_t end = run + before + v;
            if (tile >= end - own && tile < end) {
                s_start[0] = bb;
                s_start[1] = end - own;
            }
            run += sum;
            __syncthreads();
            if (tile < run)
                break;
        }
        b = s_start[0];
        b_start = s_start[1];
    }

    // ---- the units of the share ----------------------------------------------------------------
    while (tile < tile_end) {
        int64_t unit, unit_start, unit_tiles, key_first, key_end, row0, row_end;
        int kvh;
        const int64_t *list;
        const bool prefix = tile < p_total;
        if (prefix) {
            unit = tile / p.p_tiles;
            unit_tiles = p.p_tiles;
            unit_start = unit * unit_tiles;
            kvh = (int)(unit / p.p_rtiles);
            row0 = (unit - kvh * p.p_rtiles) * M;
            row_end = p.rows;
            list = a.prefix;
            key_first = p.p_first;
            key_end = a.n_prefix;
        } else {
            int64_t tb = seq_tiles(a, b);
            while (tile >= b_start + per_seq * tb) {
                b_start += per_seq * tb;
                tb = seq_tiles(a, ++b);
            }
            const int64_t u = (tile - b_start) / tb;
            unit = p_units + b * per_seq + u;
            unit_tiles = tb;
            unit_start = b_start + u * tb;
            kvh = (int)(u / p.s_rtiles);
            row0 = b * p.R + (u - (int64_t)kvh * p.s_rtiles) * M;
            row_end = (b + 1) * p.R;
            list = a.table + b * a.table_stride;
            key_end = seq_len(a, b);
            key_first = first_key(key_end, a.q_len, a.window);
        }
        const int64_t seg_end = min(tile_end, unit_start + unit_tiles);
        const bool whole = tile == unit_start && seg_end == unit_start + unit_tiles;
        const int64_t k0 = key_first + (tile - unit_start) * kTileKeys;
        const int64_t k1 = min(key_end, key_first + (seg_end - unit_start) * kTileKeys);

        // ---- query fragments (columns g), and the rows' scale and keys (columns 2t, 2t + 1) --------
        uint32_t qf[NT][8][2];
        float row_inv[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int64_t rr = row0 + 8 * n + g;
            const bool act = rr < row_end;
            int i = 0, hg = 0;
            const int64_t tok = act ? row_token(a, p, rr, i, hg) : 0;
            const char *qp = (const char *)a.q +
                             2 * (tok * a.q_stride + (int64_t)(kvh * p.group + hg) * kD);
            row_inv[n] = 1.0f;
            if constexpr (!FP8) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t *w = reinterpret_cast<const uint32_t *>(qp + 32 * ks + 4 * t);
                    qf[n][ks][0] = act ? w[0] : 0u;
                    qf[n][ks][1] = act ? w[4] : 0u;
                }
            } else {
                uint32_t mx = 0u;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 v = act ? ld_cached(qp + 128 * s + 32 * t + 16 * h)
                                            : make_uint4(0u, 0u, 0u, 0u);
                        qf[n][4 * s + 2 * h][0] = v.x, qf[n][4 * s + 2 * h][1] = v.y;
                        qf[n][4 * s + 2 * h + 1][0] = v.z, qf[n][4 * s + 2 * h + 1][1] = v.w;
                    }
                }
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        mx = max(mx, (qf[n][ks][j] << 16) & 0x7fffffffu);
                        mx = max(mx, qf[n][ks][j] & 0x7fff0000u);
                    }
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                float f;
                f16_row_factor(mx, f, row_inv[n]);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        qf[n][ks][j] = pack_f16x2(__fmul_rn(bf_lo(qf[n][ks][j]), f),
                                                  __fmul_rn(bf_hi(qf[n][ks][j]), f));
            }
        }
        float scale[NT][2];
        int64_t lo[NT][2], hi[NT][2];  // keys of the list that the row sees
        int64_t lo_all = 0, hi_all = key_end;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t rr = row0 + 8 * n + 2 * t + e;
                scale[n][e] = __fmul_rn(__fmul_rn(a.sm_scale * a.k_scale, kLog2e),
                                        __shfl_sync(0xffffffffu, row_inv[n], 4 * (2 * t + e)));
                lo[n][e] = 0;
                hi[n][e] = key_end;
                if (rr < row_end) {
                    int i, hg;
                    row_token(a, p, rr, i, hg);
                    const int64_t rb = rr / p.R;
                    const int64_t pos = seq_len(a, rb) - a.q_len + i;  // index in the suffix
                    const int64_t at = prefix ? a.n_prefix + pos : pos;  // index in the list
                    lo[n][e] = a.window > 0 && at + 1 - a.window > 0 ? at + 1 - a.window : 0;
                    hi[n][e] = pos < 0 ? 0 : (prefix ? a.n_prefix : pos + 1);
                }
                lo_all = max(lo_all, lo[n][e]);
                hi_all = min(hi_all, hi[n][e]);
            }
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            lo_all = max(lo_all, (int64_t)__shfl_xor_sync(0xffffffffu, lo_all, off));
            hi_all = min(hi_all, (int64_t)__shfl_xor_sync(0xffffffffu, hi_all, off));
        }

        float o[8][NT][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
                o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.0f;
        }

        // ---- the keys: 16 a step and warp ----------------------------------------------------------
        const int steps = (int)((k1 - k0 - warp * kWarpKeys + kTileKeys - 1) / kTileKeys);
        const int64_t pitch = (int64_t)a.n_kv * C::kRow;
        const char *kbase = (const char *)a.k_cache + kvh * C::kRow;
        const char *vbase = (const char *)a.v_cache + kvh * C::kRow;
        auto load_slot = [&](int s) -> int {  // lane i < 16: slot of key i, or -1
            const int64_t key = k0 + (int64_t)s * kTileKeys + warp * kWarpKeys + lane;
            if (lane >= kWarpKeys || s >= steps || key >= k1)
                return -1;
            const int64_t slot = list[key];
            return slot >= 0 && slot < a.num_slots ? (int)slot : -1;
        };
        uint64_t masks = 0;  // which keys of the stages in flight exist, 16 bits each
        auto issue = [&](int s, int slot) {
            masks = (masks << 16) | (__ballot_sync(0xffffffffu, slot >= 0) & 0xffffu);
            if (s < steps) {
                const uint32_t kdst = wbuf + (s % C::kStages) * 2 * C::kTileBytes;
                constexpr int kRowsPer = 32 / C::kChunks;
                const int ch = lane % C::kChunks, r0 = lane / C::kChunks;
#pragma unroll
                for (int j = 0; j < kWarpKeys / kRowsPer; ++j) {
                    const int r = j * kRowsPer + r0;
                    const int sl = __shfl_sync(0xffffffffu, slot, r);
                    const int64_t off = (sl < 0 ? 0 : sl) * pitch + 16 * ch;
                    const uint32_t dst = r * C::kRow + 16 * swizzle<FP8>(r, ch);
                    const uint32_t bytes = sl < 0 ? 0u : 16u;
                    cp_async16(kdst + dst, kbase + off, bytes);
                    cp_async16(kdst + C::kTileBytes + dst, vbase + off, bytes);
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int s = 0; s < C::kStages - 1; ++s)
            issue(s, load_slot(s));
        int next_slot = load_slot(C::kStages - 1);
        for (int s = 0; s < steps; ++s) {
            cp_async_wait<C::kStages - 2>();
            __syncwarp();
            issue(s + C::kStages - 1, next_slot);
            next_slot = load_slot(s + C::kStages);
            const uint32_t kt = wbuf + (s % C::kStages) * 2 * C::kTileBytes;
            const uint32_t vt = kt + C::kTileBytes;
            const uint32_t mask = (uint32_t)(masks >> (16 * (C::kStages - 1))) & 0xffffu;
            const int64_t key0 = k0 + (int64_t)s * kTileKeys + warp * kWarpKeys;

            float sc[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
            if constexpr (!FP8) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    uint32_t af[4];
                    const int key = lane & 15, ch = 2 * ks + (lane >> 4);
                    ldmatrix_x4(af, kt + key * C::kRow + 16 * swizzle<FP8>(key, ch));
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816<FP8>(sc[n], af, qf[n][ks][0], qf[n][ks][1]);
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 x = lds128(kt + g * C::kRow + 16 * swizzle<FP8>(g, 4 * h + t));
                    const uint4 y =
                        lds128(kt + (g + 8) * C::kRow + 16 * swizzle<FP8>(g + 8, 4 * h + t));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t xw = word(x, j), yw = word(y, j);
                        const uint32_t af[4] = {e4m3x2_to_f16x2(xw), e4m3x2_to_f16x2(yw),
                                                e4m3x2_to_f16x2(xw >> 16),
                                                e4m3x2_to_f16x2(yw >> 16)};
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816<FP8>(sc[n], af, qf[n][4 * h + j][0], qf[n][4 * h + j][1]);
                    }
                }
            }
            // scores to base 2; keys that a row does not see get -inf
            const bool all_seen = mask == 0xffffu && key0 >= lo_all && key0 + kWarpKeys <= hi_all;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = g + 8 * (e >> 1), col = e & 1;
                    const float v = __fmul_rn(sc[n][e], scale[n][col]);
                    const int64_t key = key0 + row;
                    const bool seen = all_seen || (((mask >> row) & 1u) && key >= lo[n][col] &&
                                                   key < hi[n][col]);
                    sc[n][e] = seen ? v : -INFINITY;
                }
            if (a.weight_out && !prefix) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int64_t rr = row0 + 8 * n + 2 * t + (e & 1);
                        const int64_t key = key0 + g + 8 * (e >> 1);
                        if (rr < row_end && key < k1) {
                            const int64_t sb = rr / p.R;
                            float *dst = reinterpret_cast<float *>(a.workspace + p.score_off);
                            dst[((sb * a.n_kv + kvh) * p.R + (rr - sb * p.R)) * p.score_width +
                                key] = sc[n][e];
                        }
                    }
            }
            uint32_t pf[NT][2];
            bool grew = false;
            float alpha[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float ps[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(sc[n][e], sc[n][e + 2]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float mn = fmaxf(m[n][e], mx);
                    const float ms = mn == -INFINITY ? 0.0f : mn;
                    alpha[n][e] = exp2_fast(__fsub_rn(m[n][e], ms));
                    grew = grew || mn != m[n][e];
                    m[n][e] = mn;
                    ps[e] = exp2_fast(__fsub_rn(sc[n][e], ms));
                    ps[e + 2] = exp2_fast(__fsub_rn(sc[n][e + 2], ms));
                    l[n][e] = __fmaf_rn(l[n][e], alpha[n][e], __fadd_rn(ps[e], ps[e + 2]));
                }
                pf[n][0] = movmatrix_trans(FP8 ? pack_f16x2(ps[0], ps[1]) : pack_bf16x2(ps[0], ps[1]));
                pf[n][1] = movmatrix_trans(FP8 ? pack_f16x2(ps[2], ps[3]) : pack_bf16x2(ps[2], ps[3]));
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[mt][n][e] = __fmul_rn(o[mt][n][e], alpha[n][e & 1]);
            }
            // A weight of zero does not hide an infinite or NaN value of a key that only other rows
            // see, so such a tile (rare) goes column by column with those values left out.
            if (!all_seen && tile_has_nonfinite<FP8>(vt, lane)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        const uint32_t b0 = g == c ? pf[n][0] : 0u, b1 = g == c ? pf[n][1] : 0u;
                        const float lo_s = c & 1 ? sc[n][1] : sc[n][0];
                        const float hi_s = c & 1 ? sc[n][3] : sc[n][2];
                        // bit k: the column sees key k (lanes 4 k + c / 2 hold keys k and k + 8)
                        const uint32_t lb = __ballot_sync(0xffffffffu, lo_s != -INFINITY);
                        const uint32_t hb = __ballot_sync(0xffffffffu, hi_s != -INFINITY);
                        uint32_t keep[2] = {0u, 0u};
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int bit = 4 * (2 * t + j) + c / 2;
                            keep[0] |= ((lb >> bit) & 1u) ? 0xffffu << (16 * j) : 0u;
                            keep[1] |= ((hb >> bit) & 1u) ? 0xffffu << (16 * j) : 0u;
                        }
#pragma unroll
                        for (int mt = 0; mt < 8; ++mt) {
                            uint32_t af[4];
                            load_values<FP8>(af, vt, mt, lane);
                            af[0] &= keep[0], af[1] &= keep[0];
                            af[2] &= keep[1], af[3] &= keep[1];
                            float add[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma16816<FP8>(add, af, b0, b1);
#pragma unroll
                            for (int e = 0; e < 4; ++e)  // the other columns' zeros met them too
                                if (2 * t + (e & 1) == c)
                                    o[mt][n][e] = __fadd_rn(o[mt][n][e], add[e]);
                        }
                    }
                continue;
            }
            if constexpr (!FP8) {
#pragma unroll
                for (int mt = 0; mt < 8; ++mt) {
                    uint32_t af[4];
                    load_values<FP8>(af, vt, mt, lane);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816<FP8>(o[mt][n], af, pf[n][0], pf[n][1]);
                }
            } else {
                // 16-bit units of the transposed load are pairs (d, d + 1): after the split, matrix
                // row g is element 2g of the 16, row g + 8 element 2g + 1
#pragma unroll
                for (int c2 = 0; c2 < 4; ++c2) {
                    uint32_t r[4];
                    const int key = lane & 15, ch = 2 * c2 + (lane >> 4);
                    ldmatrix_x4_trans(r, vt + key * C::kRow + 16 * swizzle<FP8>(key, ch));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t x0 = e4m3x2_to_f16x2(r[2 * h]);
                        const uint32_t x1 = e4m3x2_to_f16x2(r[2 * h] >> 16);
                        const uint32_t y0 = e4m3x2_to_f16x2(r[2 * h + 1]);
                        const uint32_t y1 = e4m3x2_to_f16x2(r[2 * h + 1] >> 16);
                        const uint32_t af[4] = {__byte_perm(x0, x1, 0x5410),
                                                __byte_perm(x0, x1, 0x7632),
                                                __byte_perm(y0, y1, 0x5410),
                                                __byte_perm(y0, y1, 0x7632)};
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816<FP8>(o[2 * c2 + h][n], af, pf[n][0], pf[n][1]);
                    }
                }
            }
        }

        // ---- join the warps ------------------------------------------------------------------------
        cp_async_wait<0>();
        __syncthreads();
        constexpr int kPitch = kD + 4;
        float *so = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[n][e];
                v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 4));
                v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 8));
                v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 16));
                if (g == 0)
                    s_ml[warp][8 * n + 2 * t + e] = make_float2(m[n][e], v);
            }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 8 * n + 2 * t + (e & 1);
                    const int d = FP8 ? 16 * mt + 2 * g + (e >> 1) : 16 * mt + g + 8 * (e >> 1);
                    so[(warp * M + r) * kPitch + d] = o[mt][n][e];
                }
        __syncthreads();
        const bool direct = whole && !prefix && p_units == 0;
        const int64_t part = unit + blockIdx.x;
        for (int x = tid; x < M * (kD / 2); x += kThreads) {
            const int r = x / (kD / 2), d = 2 * (x % (kD / 2));
            const int64_t rr = row0 + r;
            if (rr >= row_end)
                continue;
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                mm = fmaxf(mm, s_ml[w][r].x);
            const float ms = mm == -INFINITY ? 0.0f : mm;
            float ll = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2_fast(__fsub_rn(s_ml[w][r].x, ms));
                const float2 v = *reinterpret_cast<const float2 *>(&so[(w * M + r) * kPitch + d]);
                ll = __fmaf_rn(f, s_ml[w][r].y, ll);
                o0 = __fmaf_rn(f, v.x, o0);
                o1 = __fmaf_rn(f, v.y, o1);
            }
            if (direct) {
                int i, hg;
                const int64_t tok = row_token(a, p, rr, i, hg);
                const int h = kvh * p.group + hg;
                const float f = ll == 0.0f ? 0.0f : __fdiv_rn(a.v_scale, ll);
                *reinterpret_cast<uint32_t *>((char *)a.out +
                                              2 * (tok * a.out_stride + (int64_t)h * kD + d)) =
                    ll == 0.0f ? 0u : pack_bf16x2(__fmul_rn(o0, f), __fmul_rn(o1, f));
                if (d == 0) {
                    const float lse2 = ll == 0.0f ? -INFINITY : __fadd_rn(mm, log2f(ll));
                    if (a.lse)
                        a.lse[tok * a.n_q + h] =
                            ll == 0.0f ? -INFINITY : __fmaf_rn(mm, kLn2, logf(ll));
                    if (a.weight_out)
                        reinterpret_cast<float *>(a.workspace + p.lse_off)[kvh * p.rows + rr] = lse2;
                }
            } else {
                float *po = reinterpret_cast<float *>(a.workspace + p.o_off);
                *reinterpret_cast<float2 *>(po + (part * M + r) * kD + d) = make_float2(o0, o1);
                if (d == 0)
                    reinterpret_cast<float2 *>(a.workspace + p.ml_off)[part * M + r] =
                        make_float2(mm, ll);
            }
        }
        __syncthreads();
        tile = seg_end;
    }
}

// Joins a row's parts: one warp per row and KV head, four elements a lane.
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnArgs a,
                                                        const __grid_constant__ AttnPlan p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t x = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (x >= p.rows * a.n_kv)  // B * q_len * n_q < 2^31
        return;
    const int M = 8 * p.nt;
    const int kvh = (int)(x / p.rows);
    const int64_t rr = x - kvh * p.rows, b = rr / p.R;
    const int64_t *cum = reinterpret_cast<const int64_t *>(a.workspace + p.cum_off);
    const int64_t total = cum[a.B], shares = min((int64_t)p.ctas, total);
    const int64_t per_seq = (int64_t)a.n_kv * p.s_rtiles;
    const int64_t rt = (rr - b * p.R) / M;
    const int64_t tb = (cum[b + 1] - cum[b]) / per_seq;
    // the parts of the prefix unit, then those of the suffix unit
    int64_t first[2] = {0, 0}, at[2] = {0, 0};
    int count[2] = {0, 0};
    if (p.p_rtiles > 0) {
        const int64_t unit = kvh * p.p_rtiles + rr / M, s = unit * p.p_tiles;
        const int64_t c0 = owner(s, total, shares);
        first[0] = unit + c0;
        count[0] = (int)(owner(s + p.p_tiles - 1, total, shares) - c0) + 1;
        at[0] = rr % M;
    }
    if (tb > 0) {
        const int64_t u = (int64_t)kvh * p.s_rtiles + rt, s = cum[b] + u * tb;
        const int64_t c0 = owner(s, total, shares);
        first[1] = a.n_kv * p.p_rtiles + b * per_seq + u + c0;
        count[1] = (int)(owner(s + tb - 1, total, shares) - c0) + 1;
        at[1] = rr - b * p.R - rt * M;
        if (p.p_rtiles == 0 && count[1] == 1)
            return;  // the rows kernel wrote it
    }
    const float2 *ml = reinterpret_cast<const float2 *>(a.workspace + p.ml_off);
    const float *po = reinterpret_cast<const float *>(a.workspace + p.o_off);
    float m = -INFINITY;
    for (int k = 0; k < 2; ++k)
        for (int c = lane; c < count[k]; c += 32)
            m = fmaxf(m, ml[(first[k] + c) * M + at[k]].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float ms = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k = 0; k < 2; ++k)
        for (int c = 0; c < count[k]; ++c) {
            const int64_t r = (first[k] + c) * M + at[k];
            const float2 w = ml[r];
            if (w.y == 0.0f)
                continue;
            const float f = exp2_fast(__fsub_rn(w.x, ms));
            const float4 v = *reinterpret_cast<const float4 *>(po + r * kD + 4 * lane);
            l = __fmaf_rn(f, w.y, l);
            o.x = __fmaf_rn(f, v.x, o.x);
            o.y = __fmaf_rn(f, v.y, o.y);
            o.z = __fmaf_rn(f, v.z, o.z);
            o.w = __fmaf_rn(f, v.w, o.w);
        }
    int i, hg;
    const int64_t tok = row_token(a, p, rr, i, hg);
    const int h = kvh * p.group + hg;
    const float f = l == 0.0f ? 0.0f : __fdiv_rn(a.v_scale, l);
    st_global_v2((char *)a.out + 2 * (tok * a.out_stride + (int64_t)h * kD + 4 * lane),
                 pack_bf16x2(__fmul_rn(o.x, f), __fmul_rn(o.y, f)),
                 pack_bf16x2(__fmul_rn(o.z, f), __fmul_rn(o.w, f)));
    if (lane == 0) {
        if (a.lse)
            a.lse[tok * a.n_q + h] = l == 0.0f ? -INFINITY : __fmaf_rn(m, kLn2, logf(l));
        if (a.weight_out)
            reinterpret_cast<float *>(a.workspace + p.lse_off)[kvh * p.rows + rr] =
                l == 0.0f ? -INFINITY : __fadd_rn(m, log2f(l));
    }
}

// The weight each suffix key received: one thread per key, over the scores that the rows kernel kept.
__global__ void __launch_bounds__(256) attn_weight_kernel(const __grid_constant__ AttnArgs a,
                                                          const __grid_constant__ AttnPlan p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (j >= a.width)
        return;
    for (int64_t b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int64_t n = seq_len(a, b);
    float w = a.weight_in ? a.weight_in[b * a.weight_stride + j] : 0.0f;
    if (j < n && j >= first_key(n, a.q_len, a.window)) {
        const float *lse = reinterpret_cast<const float *>(a.workspace + p.lse_off);
        const float *sc = reinterpret_cast<const float *>(a.workspace + p.score_off);
        float sum = 0.0f;
        for (int h = 0; h < a.n_kv; ++h)
            for (int r = 0; r < p.R; ++r) {
                const float x = lse[h * p.rows + b * p.R + r];
                const float s = sc[((b * a.n_kv + h) * p.R + r) * p.score_width + j];
                if (x != -INFINITY)
                    sum = __fadd_rn(sum, exp2_fast(__fsub_rn(s, x)));
            }
        w = __fadd_rn(w, sum);
    }
    a.weight_out[b * a.weight_stride + j] = w;
    }
}

template <int NT, bool FP8>
cudaError_t launch_rows(const AttnArgs &a, const AttnPlan &p, cudaStream_t stream)
{
    static_assert(RowsConfig<FP8>::kSmem >= kWarps * 8 * NT * (kD + 4) * 4, "join buffer");
    const cudaError_t e =
        cudaFuncSetAttribute(attn_rows_kernel<NT, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             RowsConfig<FP8>::kSmem);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(attn_rows_kernel<NT, FP8>, dim3(p.ctas), dim3(kThreads),
                      RowsConfig<FP8>::kSmem, stream, a, p);
}

inline int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

}  // namespace

AttnPlan attn_plan(int32_t B, int32_t q_len, int32_t n_q, int32_t n_kv, int64_t n_prefix,
                   int64_t width, int64_t window, bool weights)
{
    AttnPlan p{};
    p.group = n_q / n_kv;
    p.R = q_len * p.group;
    p.rows = (int64_t)B * p.R;
    p.p_first = window > 0 && n_prefix + 1 > window ? n_prefix + 1 - window : 0;
    if (p.p_first > n_prefix)
        p.p_first = n_prefix;
    const int64_t p_keys = n_prefix - p.p_first;
    p.nt = (p.R > 8 || (p_keys > 0 && p.rows > 8)) ? 2 : 1;
    const int M = 8 * p.nt;
    p.s_rtiles = (p.R + M - 1) / M;
    p.p_rtiles = p_keys > 0 ? (p.rows + M - 1) / M : 0;
    p.p_tiles = (p_keys + kTileKeys - 1) / kTileKeys;
    p.units = n_kv * (p.p_rtiles + (int64_t)B * p.s_rtiles);
    int64_t keys = width;
    if (window > 0 && window + q_len - 1 < keys)
        keys = window + q_len - 1;
    const int64_t tiles =
        n_kv * (p.p_rtiles * p.p_tiles +
                (int64_t)B * p.s_rtiles * ((keys + kTileKeys - 1) / kTileKeys));
    const int64_t most = kPlanSms * 3;
    p.ctas = (int32_t)(tiles < 1 ? 1 : (tiles < most ? tiles : most));
    p.score_width = align_up(width, 8);
    int64_t at = 0;
    auto take = [&at](int64_t bytes) {
        const int64_t here = at;
        at = align_up(at + bytes, 256);
        return here;
    };
    p.cum_off = take(8 * ((int64_t)B + 1));
    p.o_off = take((p.units + p.ctas) * M * kD * 4);
    p.ml_off = take((p.units + p.ctas) * M * 8);
    p.lse_off = take(weights ? n_kv * p.rows * 4 : 0);
    p.score_off = take(weights ? n_kv * p.rows * p.score_width * 4 : 0);
    p.bytes = at;
    return p;
}

cudaError_t launch_attn_prefix(const AttnArgs &a, const AttnPlan &p, cudaStream_t stream)
{
    cudaError_t e;
    if (a.fp8)
        e = p.nt == 1 ? launch_rows<1, true>(a, p, stream) : launch_rows<2, true>(a, p, stream);
    else
        e = p.nt == 1 ? launch_rows<1, false>(a, p, stream) : launch_rows<2, false>(a, p, stream);
    if (e != cudaSuccess)
        return e;
    const int64_t rows = p.rows * a.n_kv;
    e = launch_pdl(attn_join_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream, a, p);
    if (e != cudaSuccess || !a.weight_out || a.width == 0)
        return e != cudaSuccess ? e : cudaGetLastError();
    e = launch_pdl(attn_weight_kernel, dim3((unsigned)((a.width + 255) / 256), (unsigned)(a.B < 65535 ? a.B : 65535)),
                   dim3(256), 0, stream, a, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace beam
