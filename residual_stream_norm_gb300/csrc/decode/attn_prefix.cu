// attn_prefix.cu -- attention of a decode batch over the slot cache, with a shared prefix (sm_103a).
//
// softmax(q K^T) V over a list of keys is computed in one pass: with the running maximum m, the
// running sum l of exp(s - m) and the running O = sum exp(s - m) v, a larger maximum m' scales l and O
// by exp(m - m').  Parts of a list join by the same rule.  Exponents are taken to base 2, scores
// carry the factor log2(e).
//
// The weights exp(s - m) meet the values in 16 bits, since a matrix instruction has both operands in one
// type: BF16, at most 2^-8 of each weight off, for a BF16 cache; FP16, 2^-11, for an FP8 cache, whose values
// it holds exactly.  The sum l takes them in FP32.  (Two BF16 parts of each weight would take the second
// product twice.)  FP16 has only 2^-14 to 2^16 at full precision, so for an FP8 cache m stands kTop below the
// maximum and the weights reach 2^kTop: 2^-11 of each then holds down to 2^-29 of the largest, and what lies
// below errs by 2^-40 of it at most.
//
// Rows kernel (every sequence's own keys; the prefix where that is little work): a warp works on 16 keys
// (FP8: 32) at a time for 8 or 16 query rows of one KV head.  It computes the transposed products
// S^T = K Q^T and O^T = V^T P^T, so that the keys fill the 16 rows of the matrix instruction and the few
// query rows its 8 columns; the 128-row tiles of tcgen05 would stay nearly empty, and the matrix pipe
// is 8 to 14% busy as it is.  Each warp copies its own keys into its own three stages (TMA, by slot),
// two steps ahead and on across the units, so warps meet only when their parts are joined; one warp
// copying for four took twice the time (104 -> 196 us for the sequences below).
//
// What bounds it: the keys' and values' bytes.  8 sequences of 16-20K keys take 104 us for 586 MB
// (5.6 TB/s, 0.83 of the copy rate), FP8 with twice the keys 110 us; where lists are short, what each
// unit costs besides its keys.  Any order of lists is shared out evenly by the device itself: the
// lengths are not known to the host, and one long list among short ones must not hold the call up.

#include "attn_common.cuh"
#include "decode_mma.cuh"
#include "decode_tma.cuh"

namespace beam {
namespace {

constexpr float kTop = 15.0f;
constexpr float kTopInv = 1.0f / 32768.0f;  // 2^-kTop
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

// A stage holds the keys and values of one step of a warp: rows of 128 bytes with their 16-byte chunks
// exchanged by the copy (chunk c of row r at c ^ (r % 8)), so that ldmatrix finds eight rows' same
// chunk in eight different bank groups.  BF16: 16 keys, the two halves of a head one after the other;
// FP8: 32 keys.
template <bool FP8>
struct RowsConfig {
    static constexpr int kMt = FP8 ? 2 : 1;       // 16-key tiles of a step
    static constexpr int kKeys = 16 * kMt;
    static constexpr int kTileKeys = kWarps * kKeys;
    static constexpr int kHalf = 16 * 128;        // BF16: bytes of 16 keys' half heads
    static constexpr int kValues = 4096;          // where the stage's values start
    static constexpr int kStageBytes = 8192;
    static constexpr int kStages = 3;
    static constexpr int kWarpBytes = kStages * kStageBytes;
};

// Shared memory of the rows kernel: the stages, the join's buffer, then the small arrays.
struct RowsSmem {
    static constexpr int kStagesEnd = kWarps * RowsConfig<false>::kWarpBytes;
    static constexpr int kMl = kStagesEnd + kWarps * 8 * kD * 4;     // float2 [kWarps][8]
    static constexpr int kBars = kMl + kWarps * 8 * 8;               // uint64_t [kWarps][kStages]
    static constexpr int kScan = kBars + kWarps * RowsConfig<false>::kStages * 8;  // int64_t [kWarps + 2]
    static constexpr int kFail = kScan + (kWarps + 2) * 8;           // int
    static constexpr int kBytes = kFail + 8;
};

__device__ unsigned int g_decode_fault_word = 0u;

// What a unit costs a block besides its key tiles (queries, joining the warps, results), in tiles:
// shares are dealt out over the tiles and this, so that a block of many short units has fewer tiles.
// The first kUnitCost places of a unit's stretch stand for it; a share that ends among them has no
// tile of the unit.
constexpr int kUnitCost = 3;

// A row's log-sum-exp, natural and to base 2, from its reference and sum.  FP8: with kTop moved back from the
// sum to the reference first, since the sum of two numbers of opposite sign near kTop would cost bits.
__device__ __forceinline__ float log_sum(bool fp8, float m, float l)
{
    return fp8 ? __fmaf_rn(__fadd_rn(m, kTop), kLn2, logf(__fmul_rn(l, kTopInv)))
               : __fmaf_rn(m, kLn2, logf(l));
}

__device__ __forceinline__ float log2_sum(bool fp8, float m, float l)
{
    return fp8 ? __fadd_rn(__fadd_rn(m, kTop), log2f(__fmul_rn(l, kTopInv)))
               : __fadd_rn(m, log2f(l));
}

// The block whose share [c tot / C, (c + 1) tot / C) contains tile x (C <= tot).
__device__ __forceinline__ int64_t owner(int64_t x, int64_t tot, int64_t ctas)
{
    const int64_t y = (x + 1) * ctas - 1;
    return (uint64_t)(y | tot) >> 32 ? y / tot : (uint32_t)y / (uint32_t)tot;
}

// x / y, x >= 0, y > 0: most often both fit 32 bits, and the division is much shorter.
__device__ __forceinline__ int64_t div32(int64_t x, int64_t y)
{
    return (uint64_t)(x | y) >> 32 ? x / y : (uint32_t)x / (uint32_t)y;
}

// Keys of a sequence's units: its own, behind the prefix's where that is in line with them.  A sequence
// without a key of its own has no row that sees any.
__device__ __forceinline__ int64_t line_len(const AttnArgs &a, const AttnPlan &p, int64_t b)
{
    const int64_t n = seq_len(a, b);
    return n > 0 ? p.in_line + n : 0;
}

__device__ __forceinline__ int64_t seq_tiles(const AttnArgs &a, const AttnPlan &p, int64_t b)
{
    const int64_t n = line_len(a, p, b);
    // tile_keys is a power of two
    return (n - first_tile_key(n, a.q_len, a.window) + p.tile_keys - 1) >> (31 - __clz(p.tile_keys));
}

// The A fragments of V^T for 16 elements d and 16 keys.  BF16 (`mt`: which 16 elements): matrix row is
// d.  FP8: one load gives two fragments (mt, mt + 1; mt even), whose 16-bit units are pairs (d, d + 1);
// after the split, matrix row g is element 2g of the 16 and row g + 8 element 2g + 1.
__device__ __forceinline__ void load_values_bf16(uint32_t (&af)[4], uint32_t vt, int mt, int lane)
{
    const int key = (lane >> 4) * 8 + (lane & 7), ch = 2 * mt + ((lane >> 3) & 1);
    ldmatrix_x4_trans(af, vt + (ch >> 3) * RowsConfig<false>::kHalf + key * 128 +
                              16 * ((ch & 7) ^ (key & 7)));
}

__device__ __forceinline__ void load_values_fp8(uint32_t (&a0)[4], uint32_t (&a1)[4], uint32_t vt,
                                                int mt, int lane)
{
    uint32_t r[4];
    const int key = lane & 15, ch = mt + (lane >> 4);
    ldmatrix_x4_trans(r, vt + key * 128 + 16 * (ch ^ (key & 7)));
    uint32_t x0 = e4m3x2_to_f16x2(r[0]), x1 = e4m3x2_to_f16x2(r[0] >> 16);
    uint32_t y0 = e4m3x2_to_f16x2(r[1]), y1 = e4m3x2_to_f16x2(r[1] >> 16);
    a0[0] = __byte_perm(x0, x1, 0x5410), a0[1] = __byte_perm(x0, x1, 0x7632);
    a0[2] = __byte_perm(y0, y1, 0x5410), a0[3] = __byte_perm(y0, y1, 0x7632);
    x0 = e4m3x2_to_f16x2(r[2]), x1 = e4m3x2_to_f16x2(r[2] >> 16);
    y0 = e4m3x2_to_f16x2(r[3]), y1 = e4m3x2_to_f16x2(r[3] >> 16);
    a1[0] = __byte_perm(x0, x1, 0x5410), a1[1] = __byte_perm(x0, x1, 0x7632);
    a1[2] = __byte_perm(y0, y1, 0x5410), a1[3] = __byte_perm(y0, y1, 0x7632);
}

// Whether a stage's values hold an infinity or NaN (E4M3 has NaN only: all bits but the sign set).
template <bool FP8>
__device__ __forceinline__ bool stage_has_nonfinite(uint32_t vt, int lane)
{
    bool bad = false;
#pragma unroll 1
    for (int i = lane; i < 256; i += 32) {
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

// Places of each of a sequence's units: its tiles and what it costs besides; none without a key (but
// with whole units these write their rows' zeros).
__device__ __forceinline__ int64_t seq_places(const AttnArgs &a, const AttnPlan &p, int64_t b)
{
    const int64_t t = seq_tiles(a, p, b);
    return t > 0 || p.whole ? t + kUnitCost : 0;
}

// A place in the units' sequence, and the unit that holds it: from unit to unit it only counts on.
struct Cursor {
    int64_t tile, end;    // the next place of the share, and the share's end
    int64_t start;        // the unit's first place
    int64_t unit, rt;     // the unit, and its tile of rows
    int32_t places;       // of the unit
    int32_t b, kvh;       // sequence (b < 0: the prefix) and KV head
    int32_t key_first, key_end;
};

// A unit's part that lies in the share.
struct Unit {
    const int64_t *list;  // of the keys from `split` on; those before are the prefix's
    int32_t split;
    int64_t unit;
    int32_t b, kvh;       // sequence (prefix: -1) and KV head
    int32_t row0, row_end;
    int32_t row_base;     // the sequence's first row (suffix)
    int32_t k0, k1;       // keys of the part; k1 <= k0: none
    int32_t key_end;      // of the list
    bool prefix, whole;
};

// Row rr of a unit: its token, query and head within the group.
__device__ __forceinline__ int64_t unit_row(const AttnArgs &a, const AttnPlan &p, const Unit &u,
                                            int rr, int &i, int &hg)
{
    if (u.prefix)
        return row_token(a, p, rr, i, hg);
    const uint32_t r = (uint32_t)(rr - u.row_base);
    i = p.group_magic ? (int)__umulhi(r, p.group_magic) : (int)(r / (uint32_t)p.group);
    hg = (int)r - i * p.group;
    return (int64_t)u.b * a.q_len + i;
}

__device__ __forceinline__ void cursor_keys(const AttnArgs &a, const AttnPlan &p, Cursor &c)
{
    if (c.b < 0) {
        c.key_first = (int32_t)p.p_first;
        c.key_end = (int32_t)a.n_prefix;
        c.places = (int32_t)p.p_tiles + kUnitCost;
    } else {
        c.key_end = (int32_t)line_len(a, p, c.b);
        c.key_first = (int32_t)first_tile_key(c.key_end, a.q_len, a.window);
        c.places = (int32_t)seq_places(a, p, c.b);
    }
}

// The cursor of a share that starts at place `tile`: sequence b (its first place b_start) holds it, or
// the prefix (b < 0, b_start 0).
__device__ __forceinline__ Cursor first_cursor(const AttnArgs &a, const AttnPlan &p, int64_t tile,
                                               int64_t end, int64_t b, int64_t b_start)
{
    Cursor c;
    c.tile = tile;
    c.end = end;
    c.b = (int32_t)b;
    cursor_keys(a, p, c);
    const int64_t rtiles = b < 0 ? p.p_rtiles : p.s_rtiles;
    const int64_t x = div32(tile - b_start, c.places);
    c.start = b_start + x * c.places;
    c.kvh = (int32_t)div32(x, rtiles);
    c.rt = x - c.kvh * rtiles;
    c.unit = x + (b < 0 ? 0 : a.n_kv * (p.p_rtiles + b * p.s_rtiles));
    if (p.whole && tile > c.start)  // the unit belongs to the share that has its first place
        c.tile = c.start + c.places;
    return c;
}

__device__ __forceinline__ Unit next_unit(const AttnArgs &a, const AttnPlan &p, int M, Cursor &c)
{
    if (c.tile >= c.start + c.places) {  // on to the unit that follows
        c.start += c.places;
        ++c.unit;
        if (++c.rt == (c.b < 0 ? p.p_rtiles : p.s_rtiles)) {
            c.rt = 0;
            if (++c.kvh == a.n_kv) {
                c.kvh = 0;
                c.b = c.b < 0 ? 0 : c.b + 1;
                cursor_keys(a, p, c);
                while (c.places == 0) {  // sequences without a key have no places
                    c.unit += (int64_t)a.n_kv * p.s_rtiles;
                    ++c.b;
                    cursor_keys(a, p, c);
                }
            }
        }
    }
    Unit u;
    u.prefix = c.b < 0;
    u.unit = c.unit;
    u.b = c.b;
    u.kvh = c.kvh;
    u.key_end = c.key_end;
    u.row_base = u.prefix ? 0 : c.b * p.R;
    u.row0 = u.row_base + (int32_t)c.rt * M;
    u.row_end = u.prefix ? (int32_t)p.rows : u.row_base + p.R;
    u.split = u.prefix ? 0 : (int32_t)p.in_line;
    u.list = u.prefix ? a.prefix : a.table + c.b * a.table_stride - u.split;
    const int64_t start = c.start + kUnitCost, stop = c.start + c.places;
    const int64_t seg_end = p.whole ? stop : min(c.end, stop), first = max(c.tile, start);
    u.whole = first == start && seg_end == stop;
    u.k0 = c.key_first + (int32_t)(first - start) * p.tile_keys;
    u.k1 = (int32_t)min((int64_t)u.key_end, c.key_first + (seg_end - start) * p.tile_keys);
    c.tile = seg_end;
    return u;
}

// The sum over the sequences of their units' places after `base`; every thread of the block takes
// part.  find >= base: also finds the sequence that holds tile `find`.  cum (or nullptr) receives the
// running sums; last_own, last_end: this thread's last sequence's places and their running sum.
__device__ __forceinline__ int64_t scan_sequences(const AttnArgs &a, const AttnPlan &p, int64_t base,
                                                  int64_t find, int64_t *cum, int64_t *s_scan,
                                                  int64_t &last_own, int64_t &last_end)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t per_seq = (int64_t)a.n_kv * p.s_rtiles;
    int64_t total = base;
    if (cum && tid == 0)
        cum[0] = base;
    for (int64_t b0 = 0; b0 < a.B; b0 += kThreads) {
        const int64_t b = b0 + tid;
        const int64_t own = b < a.B ? per_seq * seq_places(a, p, b) : 0;
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
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? s_scan[w] : 0;
            sum += s_scan[w];
        }
        const int64_t end = total + before + v;
        if (cum && b < a.B)
            cum[b + 1] = end;
        if (find >= end - own && find < end) {
            s_scan[kWarps] = b;
            s_scan[kWarps + 1] = end - own;
        }
        total += sum;
        __syncthreads();
        last_own = own, last_end = end;
        if (find >= base && find < total)
            break;
    }
    return total;
}

template <int NT, bool FP8, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads, 2)
    attn_rows_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnPlan p,
                     const __grid_constant__ CacheMaps maps)
{
    using C = RowsConfig<FP8>;
    using S = RowsSmem;
    constexpr int M = 8 * NT, MT = C::kMt;
    extern __shared__ __align__(1024) char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t wbuf = smem_addr(smem) + warp * C::kWarpBytes;
    float2 *s_ml = reinterpret_cast<float2 *>(smem + S::kMl);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kBars) + warp * C::kStages;
    int64_t *s_scan = reinterpret_cast<int64_t *>(smem + S::kScan);
    volatile int *s_fail = reinterpret_cast<int *>(smem + S::kFail);
    if (tid == 0) {
        *s_fail = smem_addr(smem) % 1024 != 0;  // the copies' exchange of chunks goes by address
        if (*s_fail)
            atomicOr(&g_decode_fault_word, kFaultCopyTimeout);
    }
    if (lane == 0) {
        for (int i = 0; i < C::kStages; ++i)
            mbar_init(&bars[i], 1);
        fence_mbar_init();
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
        prefetch_map(&maps.k_run);
        prefetch_map(&maps.v_run);
    }
    __syncwarp();
    pdl_launch_dependents();
    // Behind the tensor-core kernel too, whose results it does not read: what earlier kernels wrote
    // (lengths, table, queries, cache) is visible to the grid that waits, not to one that is merely
    // started by a grid that has waited.
    pdl_wait();

    // ---- the share of this block ---------------------------------------------------------------
    const int64_t p_units = a.n_kv * p.p_rtiles;
    const int64_t p_total = p_units * (p.p_tiles + kUnitCost);
    int64_t *cum = reinterpret_cast<int64_t *>(a.workspace + p.cum_off);
    int64_t own = 0, own_end = 0;
    const int64_t total = scan_sequences(a, p, p_total, -1, blockIdx.x == 0 ? cum : nullptr, s_scan,
                                         own, own_end);
    const int64_t shares = min((int64_t)p.ctas, total);  // none of them empty
    __syncthreads();
    if (blockIdx.x >= shares || *s_fail)
        return;
    const int64_t tile0 = div32(total * blockIdx.x, shares);
    int64_t b0 = -1, b0_start = 0;
    if (tile0 >= p_total) {
        if (a.B > kThreads) {
            scan_sequences(a, p, p_total, tile0, nullptr, s_scan, own, own_end);
        } else {  // the sums are at hand
            if (tile0 >= own_end - own && tile0 < own_end) {
                s_scan[kWarps] = tid;
                s_scan[kWarps + 1] = own_end - own;
            }
            __syncthreads();
        }
        b0 = s_scan[kWarps];
        b0_start = s_scan[kWarps + 1];
    }
    Cursor at = first_cursor(a, p, tile0, div32(total * (blockIdx.x + 1), shares), b0, b0_start);

    // ---- the copies: this warp's steps of every unit of the share, ahead of the arithmetic -----------
    Cursor ahead = at;
    Unit lu;
    int ls = 0, lsteps = 0;
    auto steps_of = [&](const Unit &u) {
        return (max(u.k1 - u.k0, 0) - warp * C::kKeys + C::kTileKeys - 1) / C::kTileKeys;
    };
    // The slots of a step are loaded two steps before its copies are issued, and only looked at
    // then: a load that is waited for at once held every step up by its latency.
    struct Fetched {
        int64_t slot;  // lane i: of key i, or -1
        int32_t kvh;
        bool have;
    };
    auto fetch = [&]() {
        while (ls >= lsteps && ahead.tile < ahead.end) {
            lu = next_unit(a, p, M, ahead);
            ls = 0;
            lsteps = steps_of(lu);
        }
        const int key = lu.k0 + ls * C::kTileKeys + warp * C::kKeys + lane;
        Fetched f{-1, lu.kvh, ls < lsteps};
        if (f.have && lane < C::kKeys && key < lu.k1)
            f.slot = key < lu.split ? a.prefix[key] : lu.list[key];
        ++ls;
        return f;
    };
    Fetched next = fetch(), second = fetch();
    uint32_t masks[C::kStages];  // which keys of the stages in flight exist; the newest first
#pragma unroll
    for (int i = 0; i < C::kStages; ++i)
        masks[i] = 0;
    int in_stage = 0;
    bool failed = false;  // a wait of this warp ran out: it copies nothing more
    auto issue = [&]() {
        const bool have = next.have && !failed;
        const int slot = next.slot >= 0 && next.slot < a.num_slots ? (int)next.slot : -1;
#pragma unroll
        for (int i = C::kStages - 1; i > 0; --i)
            masks[i] = masks[i - 1];
        masks[0] = __ballot_sync(0xffffffffu, slot >= 0);
        if (have) {
            const uint32_t dst = wbuf + in_stage * C::kStageBytes;
            if (lane == 0)
                mbar_arrive_expect_tx(&bars[in_stage], C::kStageBytes);
            // runs of 16 slots go as one copy, other slots four by four (one of -1 is out of the map
            // and gives zeros)
            const int s0 = __shfl_sync(0xffffffffu, slot, FP8 ? lane & 16 : 0);
            const uint32_t in_run = __ballot_sync(
                0xffffffffu, s0 >= 0 && slot == s0 + (FP8 ? lane & 15 : lane));
            const uint32_t in_map = __ballot_sync(0xffffffffu, s0 >= 0 && s0 + 15 < a.num_slots);
            const int x = next.kvh * kD;
            if (FP8 ? in_run == 0xffffffffu && in_map == 0xffffffffu
                    : (in_run & 0xffffu) == 0xffffu && (in_map & 1u)) {
                // lanes 0..3: K and V of the two halves of the head (BF16) or of the two runs (FP8)
                const int sub = lane & 1, isv = lane >> 1;
                const int y = __shfl_sync(0xffffffffu, slot, FP8 ? 16 * sub : 0);
                if (lane < 4)
                    copy_run(dst + isv * C::kValues + sub * C::kHalf,
                             isv ? &maps.v_run : &maps.k_run, FP8 ? x : x + 64 * sub, y,
                             &bars[in_stage]);
            } else {
                // lanes 0..15: four keys each of K or V
                const int grp = FP8 ? lane & 7 : lane & 3, half = FP8 ? 0 : (lane >> 2) & 1;
                const int isv = (lane >> 3) & 1;
                const int y0 = __shfl_sync(0xffffffffu, slot, 4 * grp);
                const int y1 = __shfl_sync(0xffffffffu, slot, 4 * grp + 1);
                const int y2 = __shfl_sync(0xffffffffu, slot, 4 * grp + 2);
                const int y3 = __shfl_sync(0xffffffffu, slot, 4 * grp + 3);
                if (lane < 16)
                    gather4(dst + isv * C::kValues + half * C::kHalf + grp * 512,
                            isv ? &maps.v : &maps.k, x + half * 64, y0, y1, y2, y3,
                            &bars[in_stage]);
            }
        }
        in_stage = in_stage + 1 == C::kStages ? 0 : in_stage + 1;
        next = second;
        second = fetch();
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i)
        issue();
    int out_stage = 0, phase = 0;

    // ---- the units of the share ----------------------------------------------------------------
    while (at.tile < at.end) {
        const Unit u = next_unit(a, p, M, at);
        if (u.k1 <= u.k0 && !p.whole)
            continue;
        // query fragments (columns g), and the rows' scale and keys (columns 2t, 2t + 1)
        uint32_t qf[NT][8][2];
        float row_inv[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int rr = u.row0 + 8 * n + g;
            const bool act = rr < u.row_end;
            int i = 0, hg = 0;
            const int64_t tok = act ? unit_row(a, p, u, rr, i, hg) : 0;
            const char *qp = (const char *)a.q +
                             2 * (tok * a.q_stride + (int64_t)(u.kvh * p.group + hg) * kD);
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
                for (int ks = 0; ks < 8; ++ks) {
                    const uint2 w = act ? *reinterpret_cast<const uint2 *>(qp + 32 * ks + 8 * t)
                                        : make_uint2(0u, 0u);
                    qf[n][ks][0] = w.x;
                    qf[n][ks][1] = w.y;
                    mx = max(mx, max((w.x << 16) & 0x7fffffffu, w.x & 0x7fff0000u));
                    mx = max(mx, max((w.y << 16) & 0x7fffffffu, w.y & 0x7fff0000u));
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
        int lo[NT][2], hi[NT][2];  // keys of the list that the row sees
        int lo_all = 0, hi_all = u.key_end;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = u.row0 + 8 * n + 2 * t + e;
                scale[n][e] = __fmul_rn(__fmul_rn(a.sm_scale * a.k_scale, kLog2e),
                                        __shfl_sync(0xffffffffu, row_inv[n], 4 * (2 * t + e)));
                lo[n][e] = 0;
                hi[n][e] = u.key_end;
                if (rr < u.row_end) {
                    int64_t pos;  // in the suffix (a suffix unit: in the line, split + that)
                    if (!u.prefix) {
                        pos = (int64_t)u.key_end - 1;  // in the line
                        if (a.q_len > 1) {
                            int i, hg;
                            unit_row(a, p, u, rr, i, hg);
                            pos += i - (a.q_len - 1);
                        }
                    } else {
                        int i, hg;
                        row_token(a, p, rr, i, hg);
                        pos = seq_len(a, (uint32_t)rr / (uint32_t)p.R) - a.q_len + i;
                    }
                    const int64_t where = u.prefix ? a.n_prefix + pos : pos;  // in the list
                    lo[n][e] = a.window > 0 && where + 1 - a.window > 0
                                   ? (int)min((int64_t)u.key_end, where + 1 - a.window)
                                   : 0;
                    hi[n][e] = pos < u.split ? 0 : (u.prefix ? u.key_end : (int)pos + 1);
                }
                lo_all = max(lo_all, lo[n][e]);
                hi_all = min(hi_all, hi[n][e]);
            }
        lo_all = __reduce_max_sync(0xffffffffu, lo_all);
        hi_all = __reduce_min_sync(0xffffffffu, hi_all);
        float *score[NT][2];  // where the rows' scores are kept
        if constexpr (WEIGHTS) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int rr = u.row0 + 8 * n + 2 * t + e;
                    score[n][e] = u.prefix || rr >= u.row_end
                                      ? nullptr
                                      : reinterpret_cast<float *>(a.workspace + p.score_off) +
                                            (((int64_t)u.b * a.n_kv + u.kvh) * p.R +
                                             (rr - u.row_base)) * p.score_width -
                                            u.split;
                }
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

        const int steps = steps_of(u);
        for (int s = 0; s < steps; ++s) {
            __syncwarp();  // every lane has read the stage that the next copy overwrites
            issue();
            if (!failed &&
                __any_sync(0xffffffffu, !mbar_wait(&bars[out_stage], phase))) {
                failed = true;
                *s_fail = 1;
                atomicOr(&g_decode_fault_word, kFaultCopyTimeout);
            }
            const uint32_t kt = wbuf + out_stage * C::kStageBytes, vt = kt + C::kValues;
            const uint32_t mask = masks[C::kStages - 1];
            if (++out_stage == C::kStages)
                out_stage = 0, phase ^= 1;
            const int key0 = u.k0 + s * C::kTileKeys + warp * C::kKeys;

            float sc[MT][NT][4];
#pragma unroll
            for (int mk = 0; mk < MT; ++mk) {
                // two chains of products, joined at the end: half the latency
                float odd[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[mk][n][e] = odd[n][e] = 0.0f;
                const int key = 16 * mk + (lane & 15);
#pragma unroll
                for (int ks = 0; ks < 8; ks += FP8 ? 2 : 1) {
                    uint32_t r[4];
                    if constexpr (!FP8) {
                        const int ch = 2 * ks + (lane >> 4);
                        ldmatrix_x4(r, kt + (ch >> 3) * C::kHalf + key * 128 +
                                           16 * ((ch & 7) ^ (key & 7)));
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816<FP8>(ks & 1 ? odd[n] : sc[mk][n], r, qf[n][ks][0],
                                          qf[n][ks][1]);
                    } else {
                        const int ch = ks + (lane >> 4);
                        ldmatrix_x4(r, kt + key * 128 + 16 * (ch ^ (key & 7)));
                        const uint32_t a0[4] = {e4m3x2_to_f16x2(r[0]), e4m3x2_to_f16x2(r[1]),
                                                e4m3x2_to_f16x2(r[0] >> 16),
                                                e4m3x2_to_f16x2(r[1] >> 16)};
                        const uint32_t a1[4] = {e4m3x2_to_f16x2(r[2]), e4m3x2_to_f16x2(r[3]),
                                                e4m3x2_to_f16x2(r[2] >> 16),
                                                e4m3x2_to_f16x2(r[3] >> 16)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma16816<FP8>(sc[mk][n], a0, qf[n][ks][0], qf[n][ks][1]);
                            mma16816<FP8>(odd[n], a1, qf[n][ks + 1][0], qf[n][ks + 1][1]);
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[mk][n][e] =
                            __fmul_rn(__fadd_rn(sc[mk][n][e], odd[n][e]), scale[n][e & 1]);
            }
            // keys that a row does not see get -inf
            const bool all_seen = mask == (FP8 ? 0xffffffffu : 0xffffu) && key0 >= lo_all &&
                                  key0 + C::kKeys <= hi_all;
            if (!all_seen) {
#pragma unroll
                for (int mk = 0; mk < MT; ++mk)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int row = 16 * mk + g + 8 * (e >> 1), key = key0 + row;
                            const bool seen = ((mask >> row) & 1u) && key >= lo[n][e & 1] &&
                                              key < hi[n][e & 1];
                            sc[mk][n][e] = seen ? sc[mk][n][e] : -INFINITY;
                        }
            }
            if constexpr (WEIGHTS) {
#pragma unroll
                for (int mk = 0; mk < MT; ++mk)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = key0 + 16 * mk + g + 8 * (e >> 1);
                            if (score[n][e & 1] && key < u.k1 && key >= u.split)
                                score[n][e & 1][key] = sc[mk][n][e];
                        }
            }
            uint32_t pf[MT][NT][2];
            bool grew = false;
            float alpha[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float ms[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(sc[0][n][e], sc[0][n][e + 2]);
#pragma unroll
                    for (int mk = 1; mk < MT; ++mk)
                        mx = fmaxf(mx, fmaxf(sc[mk][n][e], sc[mk][n][e + 2]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    if constexpr (FP8)
                        mx = __fsub_ru(mx, kTop);  // upwards: no weight above 2^kTop
                    const float mn = fmaxf(m[n][e], mx);
                    ms[e] = mn == -INFINITY ? 0.0f : mn;
                    alpha[n][e] = exp2_fast(__fsub_rn(m[n][e], ms[e]));
                    grew = grew || mn != m[n][e];
                    m[n][e] = mn;
                    l[n][e] = __fmul_rn(l[n][e], alpha[n][e]);
                }
#pragma unroll
                for (int mk = 0; mk < MT; ++mk) {
                    float ps[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        ps[e] = exp2_fast(__fsub_rn(sc[mk][n][e], ms[e & 1]));
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        l[n][e] = __fadd_rn(l[n][e], __fadd_rn(ps[e], ps[e + 2]));
                    pf[mk][n][0] = movmatrix_trans(FP8 ? pack_f16x2(ps[0], ps[1])
                                                       : pack_bf16x2(ps[0], ps[1]));
                    pf[mk][n][1] = movmatrix_trans(FP8 ? pack_f16x2(ps[2], ps[3])
                                                       : pack_bf16x2(ps[2], ps[3]));
                }
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
            // see, so such a stage (rare) goes column by column with those values left out.
            const bool hidden = key0 < lo_all || hi_all < min(key0 + C::kKeys, u.key_end);
            if (hidden && stage_has_nonfinite<FP8>(vt, lane)) {
#pragma unroll
                for (int mk = 0; mk < MT; ++mk)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            const uint32_t b0 = g == c ? pf[mk][n][0] : 0u;
                            const uint32_t b1 = g == c ? pf[mk][n][1] : 0u;
                            const float s_lo = c & 1 ? sc[mk][n][1] : sc[mk][n][0];
                            const float s_hi = c & 1 ? sc[mk][n][3] : sc[mk][n][2];
                            // the column's scores of keys k and k + 8 lie in lane 4 k + c / 2
                            const uint32_t lb = __ballot_sync(0xffffffffu, s_lo != -INFINITY);
                            const uint32_t hb = __ballot_sync(0xffffffffu, s_hi != -INFINITY);
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
                                if constexpr (FP8) {
                                    uint32_t other[4];
                                    if (mt & 1)
                                        load_values_fp8(other, af, vt + mk * 2048, mt - 1, lane);
                                    else
                                        load_values_fp8(af, other, vt + mk * 2048, mt, lane);
                                } else {
                                    load_values_bf16(af, vt, mt, lane);
                                }
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
#pragma unroll
            for (int mk = 0; mk < MT; ++mk) {
                if constexpr (!FP8) {
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt) {
                        uint32_t af[4];
                        load_values_bf16(af, vt, mt, lane);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816<FP8>(o[mt][n], af, pf[mk][n][0], pf[mk][n][1]);
                    }
                } else {
#pragma unroll
                    for (int mt = 0; mt < 8; mt += 2) {
                        uint32_t a0[4], a1[4];
                        load_values_fp8(a0, a1, vt + mk * 2048, mt, lane);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma16816<FP8>(o[mt][n], a0, pf[mk][n][0], pf[mk][n][1]);
                            mma16816<FP8>(o[mt + 1][n], a1, pf[mk][n][0], pf[mk][n][1]);
                        }
                    }
                }
            }
        }

        // ---- join the warps: each adds up a quarter of the head's elements for all four ------------------
        const bool direct = u.whole && !u.prefix && p_units == 0 && p.tc_parts == 0;
        const int64_t part = u.unit + blockIdx.x;
        float4 *buf = reinterpret_cast<float4 *>(smem + S::kStagesEnd);  // [warp][mt][lane]
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            __syncthreads();  // the last join has been read
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[n][e];
                v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 4));
                v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 8));
                v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 16));
                if (g == 0)
                    s_ml[warp * 8 + 2 * t + e] = make_float2(m[n][e], v);
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
                buf[(warp * 8 + mt) * 32 + lane] =
                    make_float4(o[mt][n][0], o[mt][n][1], o[mt][n][2], o[mt][n][3]);
            __syncthreads();
            if (*s_fail)  // after a wait that ran out nothing more is written
                continue;
            float mm[2], ll[2], f[kWarps][2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float2 x[kWarps];
                mm[e] = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    x[w] = s_ml[w * 8 + 2 * t + e];
                    mm[e] = fmaxf(mm[e], x[w].x);
                }
                const float ms = mm[e] == -INFINITY ? 0.0f : mm[e];
                ll[e] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    f[w][e] = exp2_fast(__fsub_rn(x[w].x, ms));
                    ll[e] = __fmaf_rn(f[w][e], x[w].y, ll[e]);
                }
            }
            float v[2][4];  // this warp's two tiles of 16 elements
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[h][e] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 x = buf[(w * 8 + 2 * warp + h) * 32 + lane];
                    v[h][0] = __fmaf_rn(f[w][0], x.x, v[h][0]);
                    v[h][1] = __fmaf_rn(f[w][1], x.y, v[h][1]);
                    v[h][2] = __fmaf_rn(f[w][0], x.z, v[h][2]);
                    v[h][3] = __fmaf_rn(f[w][1], x.w, v[h][3]);
                }
            }
            const int r0 = 8 * n + 2 * t;  // this lane's rows: r0, r0 + 1
            if (direct) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int rr = u.row0 + r0 + e;
                    const float c = ll[e] == 0.0f ? 0.0f : __fdiv_rn(a.v_scale, ll[e]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        v[h][e] = ll[e] == 0.0f ? 0.0f : __fmul_rn(v[h][e], c);
                        v[h][e + 2] = ll[e] == 0.0f ? 0.0f : __fmul_rn(v[h][e + 2], c);
                    }
                    if (warp == 0 && g == 0 && rr < u.row_end) {
                        int i, hg;
                        const int64_t tok = unit_row(a, p, u, rr, i, hg);
                        if (a.lse)
                            a.lse[tok * a.n_q + u.kvh * p.group + hg] =
                                ll[e] == 0.0f ? -INFINITY : log_sum(FP8, mm[e], ll[e]);
                        if (WEIGHTS)
                            reinterpret_cast<float *>(
                                a.workspace + p.lse_off)[((int64_t)u.b * a.n_kv + u.kvh) * p.R +
                                                         (rr - u.row_base)] =
                                ll[e] == 0.0f ? -INFINITY : log2_sum(FP8, mm[e], ll[e]);
                    }
                }
                // FP8: a lane holds d = 16 mt + 2g, + 1 of both rows; BF16: d = 16 mt + g and + 8, so the
                // lanes of an even and an odd g exchange a row each
                const int own = FP8 ? 0 : g & 1;
                const int rr = u.row0 + r0 + own;
                const bool in0 = rr < u.row_end, in1 = FP8 && rr + 1 < u.row_end;
                int i = 0, hg = 0, hg1 = 0;
                const int64_t tok = in0 ? unit_row(a, p, u, rr, i, hg) : 0;
                const int64_t tok1 = in1 ? unit_row(a, p, u, rr + 1, i, hg1) : 0;
                char *dst = (char *)a.out + 64 * warp +
                            2 * (tok * a.out_stride + (int64_t)(u.kvh * p.group + hg) * kD);
                char *dst1 = (char *)a.out + 64 * warp +
                             2 * (tok1 * a.out_stride + (int64_t)(u.kvh * p.group + hg1) * kD);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (FP8) {
                        if (in0)
                            *reinterpret_cast<uint32_t *>(dst + 32 * h + 4 * g) =
                                pack_bf16x2(v[h][0], v[h][2]);
                        if (in1)
                            *reinterpret_cast<uint32_t *>(dst1 + 32 * h + 4 * g) =
                                pack_bf16x2(v[h][1], v[h][3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float give = own ? v[h][2 * k] : v[h][2 * k + 1];
                            const float got = __shfl_xor_sync(0xffffffffu, give, 4);
                            const uint32_t w = own ? pack_bf16x2(got, v[h][2 * k + 1])
                                                   : pack_bf16x2(v[h][2 * k], got);
                            if (in0)
                                *reinterpret_cast<uint32_t *>(dst + 32 * h + 16 * k +
                                                              2 * (g & ~1)) = w;
                        }
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = r0 + e;
                    if (u.row0 + r >= u.row_end)
                        continue;
                    if (warp == 0 && g == 0)
                        reinterpret_cast<float2 *>(a.workspace + p.ml_off)[part * M + r] =
                            make_float2(mm[e], ll[e]);
                    float *dst = reinterpret_cast<float *>(a.workspace + p.o_off) +
                                 (part * M + r) * kD + 32 * warp;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (FP8) {
                            *reinterpret_cast<float2 *>(dst + 16 * h + 2 * g) =
                                make_float2(v[h][e], v[h][e + 2]);
                        } else {
                            dst[16 * h + g] = v[h][e];
                            dst[16 * h + g + 8] = v[h][e + 2];
                        }
                    }
                }
            }
        }
    }
    // a wait that ran out: the copies still in flight end before the block does (a bounded wait)
    if (failed) {
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < kWaitLimitNs / 4) {
        }
    }
}

// Joins a row's parts: WARPS warps a row and KV head, which share out the parts; a lane has four
// elements.  Few rows have many parts: four warps then (a sequence of 2047 keys, the whole call:
// 15.5 -> 11.9 us with these loads and four warps).  A warp looks at 32 parts' maxima and sums at a time, a
// lane each, and its loads of the parts do not wait for one another.
template <int WARPS>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnArgs a,
                                                        const __grid_constant__ AttnPlan p)
{
    __shared__ float4 s_o[4][32];
    __shared__ float2 s_ml[4];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = WARPS == 1 ? 0 : warp;
    const int64_t x = WARPS == 1 ? (int64_t)blockIdx.x * 4 + warp : blockIdx.x;
    if (x >= p.rows * a.n_kv)  // B * q_len * n_q < 2^31
        return;
    const int M = 8 * p.nt;
    const int kvh = (int)((uint32_t)x / (uint32_t)p.rows);
    const int64_t rr = x - kvh * p.rows, b = (uint32_t)rr / (uint32_t)p.R;
    const int64_t *cum = reinterpret_cast<const int64_t *>(a.workspace + p.cum_off);
    const int64_t total = cum[a.B], shares = min((int64_t)p.ctas, total);
    const int64_t c0b = cum[b], c1b = cum[b + 1];
    const int64_t per_seq = (int64_t)a.n_kv * p.s_rtiles;
    const int64_t rt = (rr - b * p.R) / M;
    const int64_t places = div32(c1b - c0b, per_seq), tb = places - kUnitCost;
    // the parts of the prefix unit, then those of the suffix unit, then the tensor-core kernel's
    int64_t first[3] = {0, 0, 0};
    int at[2] = {0, 0}, count[3] = {0, 0, 0};
    if (p.p_rtiles > 0) {
        const int64_t unit = kvh * p.p_rtiles + rr / M;
        const int64_t s = unit * (p.p_tiles + kUnitCost) + kUnitCost;
        const int64_t c0 = owner(s, total, shares);
        first[0] = unit + c0;
        count[0] = (int)(owner(s + p.p_tiles - 1, total, shares) - c0) + 1;
        at[0] = (int)(rr % M);
    }
    if (tb > 0) {
        const int64_t u = (int64_t)kvh * p.s_rtiles + rt, s = c0b + u * places + kUnitCost;
        const int64_t c0 = owner(s, total, shares);
        first[1] = a.n_kv * p.p_rtiles + b * per_seq + u + c0;
        count[1] = (int)(owner(s + tb - 1, total, shares) - c0) + 1;
        at[1] = (int)(rr - b * p.R - rt * M);
        if (p.p_rtiles == 0 && p.tc_parts == 0 && count[1] == 1)
            return;  // the rows kernel wrote it
    }
    const float2 *ml = reinterpret_cast<const float2 *>(a.workspace + p.ml_off);
    const float *po = reinterpret_cast<const float *>(a.workspace + p.o_off);
    const float2 *tml = reinterpret_cast<const float2 *>(a.workspace + p.tc_ml_off);
    const float *tpo = reinterpret_cast<const float *>(a.workspace + p.tc_o_off);
    first[2] = x * p.tc_parts;
    count[2] = p.tc_parts;
    const int c01 = count[0] + count[1], parts = c01 + count[2];
    // where part c's row lies among its kernel's parts
    auto row_of = [&](int c) {
        return c < count[0] ? (first[0] + c) * M + at[0]
               : c < c01    ? (first[1] + c - count[0]) * M + at[1]
                            : first[2] + c - c01;
    };
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int kLoads = WARPS == 1 ? 4 : 8;  // at a time
    const int begin = parts * sub / WARPS, end = parts * (sub + 1) / WARPS;  // this warp's parts
    for (int c0 = begin; c0 < end; c0 += 32) {
        const int n = min(32, end - c0);
        float2 w = make_float2(-INFINITY, 0.0f);
        if (lane < n)
            w = (c0 + lane < c01 ? ml : tml)[row_of(c0 + lane)];
        // a part that saw nothing adds nothing, whatever its sums hold
        float mx = w.y == 0.0f ? -INFINITY : w.x;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.0f : mn;
        const float f0 = exp2_fast(__fsub_rn(m, ms));
        const float f = w.y == 0.0f ? 0.0f : exp2_fast(__fsub_rn(w.x, ms));
        m = mn;
        float ls = __fmul_rn(f, w.y);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            ls = __fadd_rn(ls, __shfl_xor_sync(0xffffffffu, ls, off));
        l = __fmaf_rn(l, f0, ls);
        o.x = __fmul_rn(o.x, f0), o.y = __fmul_rn(o.y, f0);
        o.z = __fmul_rn(o.z, f0), o.w = __fmul_rn(o.w, f0);
        const uint32_t live = __ballot_sync(0xffffffffu, lane < n && w.y != 0.0f);
        for (int c = 0; c < n; c += kLoads) {
            float4 v[kLoads];
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                v[j] = (live >> (c + j)) & 1u
                           ? *reinterpret_cast<const float4 *>(
                                 (c0 + c + j < c01 ? po : tpo) + row_of(c0 + c + j) * kD + 4 * lane)
                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const float fj = __shfl_sync(0xffffffffu, f, (c + j) & 31);
                o.x = __fmaf_rn(fj, v[j].x, o.x);
                o.y = __fmaf_rn(fj, v[j].y, o.y);
                o.z = __fmaf_rn(fj, v[j].z, o.z);
                o.w = __fmaf_rn(fj, v[j].w, o.w);
            }
        }
    }
    if constexpr (WARPS > 1) {
        s_o[warp][lane] = o;
        if (lane == 0)
            s_ml[warp] = make_float2(m, l);
        __syncthreads();
        if (warp > 0)
            return;
#pragma unroll
        for (int k = 1; k < WARPS; ++k)
            m = fmaxf(m, s_ml[k].x);
        const float ms = m == -INFINITY ? 0.0f : m;
        l = 0.0f;
        o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < WARPS; ++k) {
            const float f = exp2_fast(__fsub_rn(s_ml[k].x, ms));
            const float4 v = s_o[k][lane];
            l = __fmaf_rn(f, s_ml[k].y, l);
            o.x = __fmaf_rn(f, v.x, o.x), o.y = __fmaf_rn(f, v.y, o.y);
            o.z = __fmaf_rn(f, v.z, o.z), o.w = __fmaf_rn(f, v.w, o.w);
        }
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
            a.lse[tok * a.n_q + h] = l == 0.0f ? -INFINITY : log_sum(a.fp8, m, l);
        if (a.weight_out)
            reinterpret_cast<float *>(
                a.workspace + p.lse_off)[(b * a.n_kv + kvh) * p.R + (rr - b * p.R)] =
                l == 0.0f ? -INFINITY : log2_sum(a.fp8, m, l);
    }
}

// The weight each suffix key received, out of the scores that the rows kernel kept: a thread a key, eight
// loads at a time.  SHARES 4: a block takes 64 keys only, and its four groups of threads a quarter of
// the rows each, added in order: less time where few keys can have a weight (20 sequences of 156 keys
// and 192 rows: 14 us less; a window of 512 in 15 tables of 31,918: 90 -> 70 us for the call), more where
// many can (8 of 100K keys: 34 us more).  SHARES 8, 32 keys a block, where the tables have few blocks: 10
// of 3,407 keys 42.2 -> 38.6 us for the call, 15 of 1,410 keys 47.9 -> 43.9; for 32 of 4,096 keys 140.5 ->
// 142.5, for 15 of 31,918 69.8 -> 71.7, so not there.
template <int SHARES>
__global__ void __launch_bounds__(256) attn_weight_kernel(const __grid_constant__ AttnArgs a,
                                                          const __grid_constant__ AttnPlan p)
{
    constexpr int kWeightKeys = 256 / SHARES;
    __shared__ float s_part[SHARES][kWeightKeys];
    pdl_launch_dependents();
    pdl_wait();
    const int t = threadIdx.x % kWeightKeys, q = threadIdx.x / kWeightKeys;
    const int64_t j0 = (int64_t)blockIdx.x * kWeightKeys, j = j0 + t;
    const int rows = a.n_kv * p.R;  // rows of a sequence, KV head by KV head
    const int r_begin = (int)((int64_t)rows * q / SHARES);
    const int r_end = (int)((int64_t)rows * (q + 1) / SHARES);
    for (int64_t b = blockIdx.y; b < a.B; b += gridDim.y) {
        const int64_t n = seq_len(a, b), first = first_key(n, a.q_len, a.window);
        const bool any = j0 < n && j0 + kWeightKeys > first;  // the same for the whole block
        float sum = 0.0f;
        if (any) {
            const float *lse = reinterpret_cast<const float *>(a.workspace + p.lse_off) + b * rows;
            const float *sc = reinterpret_cast<const float *>(a.workspace + p.score_off) +
                              b * rows * p.score_width + j;
            const bool in = j < n && j >= first;
            for (int x0 = r_begin; x0 < r_end; x0 += 8) {
                float s[8], z[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const bool have = in && x0 + k < r_end;
                    s[k] = have ? sc[(int64_t)(x0 + k) * p.score_width] : 0.0f;
                    z[k] = have ? lse[x0 + k] : -INFINITY;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (z[k] != -INFINITY)
                        sum = __fadd_rn(sum, exp2_fast(__fsub_rn(s[k], z[k])));
            }
            if (SHARES > 1) {
                s_part[q][t] = sum;
                __syncthreads();
            }
        }
        if (q == 0 && j < a.width) {
            float w = a.weight_in ? a.weight_in[b * a.weight_stride + j] : 0.0f;
            if (SHARES > 1 && any)
#pragma unroll
                for (int k = 1; k < SHARES; ++k)
                    sum = __fadd_rn(sum, s_part[k][t]);
            w = __fadd_rn(w, sum);
            a.weight_out[b * a.weight_stride + j] = w;
        }
        if (SHARES > 1 && any)
            __syncthreads();
    }
}

template <int NT, bool FP8, bool WEIGHTS>
cudaError_t launch_rows(const AttnArgs &a, const AttnPlan &p, const CacheMaps &maps,
                        cudaStream_t stream)
{
    constexpr int bytes = RowsSmem::kBytes;
    const cudaError_t e = allow_smem<attn_rows_kernel<NT, FP8, WEIGHTS>>(bytes);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(attn_rows_kernel<NT, FP8, WEIGHTS>, dim3(p.ctas), dim3(kThreads), bytes,
                      stream, a, p, maps);
}

template <int NT>
cudaError_t launch_rows_type(const AttnArgs &a, const AttnPlan &p, const CacheMaps &maps,
                             cudaStream_t stream)
{
    if (a.fp8)
        return a.weight_out ? launch_rows<NT, true, true>(a, p, maps, stream)
                            : launch_rows<NT, true, false>(a, p, maps, stream);
    return a.weight_out ? launch_rows<NT, false, true>(a, p, maps, stream)
                        : launch_rows<NT, false, false>(a, p, maps, stream);
}

inline int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Up to so many prefix keys stand in line with each sequence's own and are read again for each, out of
// the cache; more are units of their own, joined later (the tensor-core kernel, where it is preferred, comes
// first).  In units and in line, us, behind 16, 128 and 256 keys: 1 sequence 8.4, 8.6, 8.8 and 8.0, 8.2, 8.2; 32 of
// 50-100 keys 15.8, 16.8, 17.5 and 11.5, 13.6, 15.4; 96 of 4 tokens and 30-60 keys 66, 71, 81 and 39, 50, 62; 128 of
// 250-500 keys 62, 63, 66 and 48, 52, 58.  Behind 512 keys in line is ahead by up to a seventh but 3% behind for
// 64 sequences, behind 768 it is slower for 32 to 128 (21.8 against 20.5, 80.7 against 77.8).
constexpr int64_t kInLine = 256;

// The prefix goes to the tensor-core kernel where that is expected to take less time, in tenths of a
// microsecond: it costs 11 us to set up and write out and 1.8 us a step (bench of 1 to 43 steps); the
// rows kernel 1.3 us a tile of 64 keys for 16 rows, or a unit's cost of kUnitCost of them, on each
// of its blocks.  (128 rows behind 512 keys: 7 against 13 us; 384 rows behind 5001: 69 against 22 us.  Whole
// calls, 6 rows of a KV head a sequence: 16 sequences behind 3000 keys 22.8 against 23.6 us, 8192 keys 35.9 against
// 26.4; 128 sequences behind 300 keys 48.6 against 45.7, 1000 keys 65 against 49.  Over 80 such sizes the
// choice was at most a sixth from the better side, most often within 3%.)
bool prefer_tc(const AttnPlan &p, int32_t n_kv, int64_t keys)
{
    const int64_t places = n_kv * ((p.rows + 15) / 16) * ((keys + 63) / 64 + kUnitCost);
    const int64_t rows = 13 * ((places + 2 * kPlanSms - 1) / (2 * kPlanSms));
    const int64_t blocks = (int64_t)p.tc_rtiles * n_kv * p.tc_blocks;
    const int64_t tc = 110 + 18 * p.tc_steps * ((blocks + kPlanSms - 1) / kPlanSms);
    return tc < rows;
}

// Divides the prefix among the tensor-core kernel's blocks: tiles of 256 rows, or, up to 128 rows, of
// 128 rows with every other key tile to each half of the block.  The number of parts is the one
// that fills the SMs best; a part costs about three key tiles besides its own.
void plan_tc(AttnPlan &p, int32_t n_kv, int64_t keys)
{
    p.tc_split = p.rows <= 128;
    p.tc_rtiles = (int32_t)((p.rows + 255) / 256);
    const int64_t tiles = (keys + 127) / 128;               // key tiles
    const int64_t most = p.tc_split ? (tiles + 1) / 2 : tiles;  // steps of a block
    const int64_t units = (int64_t)p.tc_rtiles * n_kv;
    int64_t best = INT64_MAX;
    for (int64_t parts = 1; parts <= most && parts <= 4 * kPlanSms; ++parts) {
        const int64_t steps = (most + parts - 1) / parts;
        const int64_t cost = (units * parts + kPlanSms - 1) / kPlanSms * (steps + 3);
        if (cost < best) {
            best = cost;
            p.tc_steps = (int32_t)steps;
        }
    }
    p.tc_blocks = (int32_t)((most + p.tc_steps - 1) / p.tc_steps);
    if (prefer_tc(p, n_kv, keys))
        p.tc_parts = p.tc_split ? 2 * p.tc_blocks : p.tc_blocks;
}

}  // namespace

AttnPlan attn_plan(int32_t B, int32_t q_len, int32_t n_q, int32_t n_kv, int64_t n_prefix,
                   int64_t width, int64_t window, bool weights, bool fp8, bool tc)
{
    AttnPlan p{};
    if (window > n_prefix + width)
        window = 0;  // longer than any list
    p.tile_keys = fp8 ? RowsConfig<true>::kTileKeys : RowsConfig<false>::kTileKeys;
    p.group = n_q / n_kv;
    p.R = q_len * p.group;
    // r / group = high word of r * magic while r * group < 2^32
    p.group_magic = p.group > 1 && (int64_t)p.R * p.group < (int64_t)1 << 32
                        ? (uint32_t)((((int64_t)1 << 32) + p.group - 1) / p.group)
                        : 0;
    p.rows = (int64_t)B * p.R;
    p.p_first = window > 0 && n_prefix + 1 > window ? n_prefix + 1 - window : 0;
    p.p_first = (p.p_first < n_prefix ? p.p_first : n_prefix) & ~(int64_t)15;
    const int64_t p_keys = n_prefix - p.p_first;
    if (tc && p_keys > 0)
        plan_tc(p, n_kv, p_keys);
    // A short prefix goes in front of each sequence's own keys: it is read again for each of them (out
    // of the cache), but needs no units of its own and no join.
    const bool in_line = p.tc_parts == 0 && n_prefix <= kInLine && width < (int64_t)1 << 30;
    p.in_line = in_line ? n_prefix : 0;
    const bool with_prefix = p_keys > 0 && p.tc_parts == 0 && !in_line;
    // (24 rows a unit were measured too: the kernel then spills, and calls of few units, which wait
    // rather than work, take longer: 8 queries of 7 sequences 13 -> 19 us.)
    p.nt = (p.R > 8 || (with_prefix && p.rows > 8)) ? 2 : 1;
    const int M = 8 * p.nt;
    p.s_rtiles = (p.R + M - 1) / M;
    p.p_rtiles = with_prefix ? (p.rows + M - 1) / M : 0;
    p.p_tiles = (p_keys + p.tile_keys - 1) / p.tile_keys;
    p.units = n_kv * (p.p_rtiles + (int64_t)B * p.s_rtiles);
    int64_t keys = p.in_line + width;
    if (window > 0 && window + q_len - 1 < keys)
        keys = window + q_len - 1 + 15;
    // Units that are not split need no join: where none has more than one tile, or where the longest that
    // there can be takes no more places than an even share of the units' costs alone, so that whatever
    // the lengths no block has more than twice an even share.  Against split units: 14 sequences of
    // 3 tokens 13.2 -> 10.1 us, 21 of at most 53 keys with weights 12.7 -> 10.9; 8 KV heads, 512 sequences
    // of 1-300 keys 104 -> 94, 256 of 1-300 56.6 -> 53.6, 256 behind a window of 512 94.5 -> 87.5, 256 of
    // 1-1024 113 -> 121.  Without the bound, one list of 100K keys among 256 short ones held the
    // call up (1859 us; split 141).
    const int64_t most = kPlanSms * 2;
    p.whole = p.p_rtiles == 0 && p.tc_parts == 0 &&
              (keys + 15 <= p.tile_keys ||
               ((keys + 15 + p.tile_keys - 1) / p.tile_keys + kUnitCost) * most <=
                   p.units * kUnitCost);
    // the most places there can be: no block is worth less than one
    const int64_t tiles =
        n_kv * (p.p_rtiles * (p.p_tiles + kUnitCost) +
                (int64_t)B * p.s_rtiles * ((keys + p.tile_keys - 1) / p.tile_keys + kUnitCost));
    p.ctas = (int32_t)(tiles < 1 ? 1 : (tiles < most ? tiles : most));
    p.score_width = align_up(width, 8);
    int64_t at = 0;
    auto take = [&at](int64_t bytes) {
        const int64_t here = at;
        at = align_up(at + bytes, 256);
        return here;
    };
    p.cum_off = take(8 * ((int64_t)B + 1));
    p.o_off = take((p.units + most) * M * kD * 4);
    p.ml_off = take((p.units + most) * M * 8);
    p.lse_off = take(weights ? n_kv * p.rows * 4 : 0);
    p.tc_o_off = take(n_kv * p.rows * p.tc_parts * kD * 4);
    p.tc_ml_off = take(n_kv * p.rows * p.tc_parts * 8);
    p.score_off = take(weights ? n_kv * p.rows * p.score_width * 4 : 0);
    p.bytes = at;
    return p;
}

cudaError_t launch_attn_prefix(const AttnArgs &a, const AttnPlan &p, cudaStream_t stream)
{
    CacheMaps maps;
    cudaError_t e = make_cache_maps(maps, a);
    if (e != cudaSuccess)
        return e;
    if (p.tc_parts > 0) {
        e = launch_attn_tc(a, p, maps, stream);
        if (e != cudaSuccess)
            return e;
    }
    e = p.nt == 1 ? launch_rows_type<1>(a, p, maps, stream) : launch_rows_type<2>(a, p, maps, stream);
    if (e != cudaSuccess)
        return e;
    const int64_t rows = p.rows * a.n_kv;
    if (p.whole)
        e = cudaSuccess;
    else
        e = rows < kPlanSms * 8
            ? launch_pdl(attn_join_kernel<4>, dim3((unsigned)rows), dim3(128), 0, stream, a, p)
            : launch_pdl(attn_join_kernel<1>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream,
                         a, p);
    if (e != cudaSuccess || !a.weight_out || a.width == 0)
        return e != cudaSuccess ? e : cudaGetLastError();
    const unsigned by = (unsigned)(a.B < 65535 ? a.B : 65535);
    int64_t keys = a.width;  // that can have a weight
    if (a.window > 0 && (int64_t)a.window + a.q_len - 1 < keys)
        keys = (int64_t)a.window + a.q_len - 1;
    if (a.B * ((a.width + 255) / 256) < 2 * kPlanSms)
        e = launch_pdl(attn_weight_kernel<8>, dim3((unsigned)((a.width + 31) / 32), by), dim3(256),
                       0, stream, a, p);
    else if (a.B * ((keys + 255) / 256) < 8 * kPlanSms)
        e = launch_pdl(attn_weight_kernel<4>, dim3((unsigned)((a.width + 63) / 64), by), dim3(256),
                       0, stream, a, p);
    else
        e = launch_pdl(attn_weight_kernel<1>, dim3((unsigned)((a.width + 255) / 256), by), dim3(256),
                       0, stream, a, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t read_decode_fault_word(unsigned int *value, bool clear)
{
    unsigned int tc = 0u;
    cudaError_t e = read_attn_tc_fault_word(&tc, clear);
    if (e == cudaSuccess)
        e = cudaMemcpyFromSymbol(value, g_decode_fault_word, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0u;
        e = cudaMemcpyToSymbol(g_decode_fault_word, &zero, sizeof(unsigned int));
    }
    *value |= tc;
    return e;
}

}  // namespace beam
