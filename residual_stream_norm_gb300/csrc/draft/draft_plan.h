// draft_plan.h -- how calls of the operators of a draft-checking decode step are divided, as functions of their sizes
// alone.  Host code without CUDA, so that it is tested by itself.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define BEAM_PLAN_FN __host__ __device__
#else
#define BEAM_PLAN_FN
#endif

namespace beam {

// ---------------------------------------------------------------------------------------------
// attention on the 4-bit cache
// ---------------------------------------------------------------------------------------------

namespace kv4 {

constexpr int kSms = 152;
constexpr int kScan = 256;  // threads that count tiles
constexpr int kTile = 32;   // keys
constexpr double kGangExtra = 40;  // tiles of 8 rows

// Warps of a block, as the registers of NT 8-row tiles allow without spilling more than a few (128 or 168 a thread).
// Between tiles a unit's output is kept in tensor memory, 32 columns of a warp's own lanes for each row tile: with the
// outputs in registers 8 contexts of 100K keys (NT = 1, groups of 32) took 197 us with 12 warps, 184 so with 16; 32
// sequences of up to 20K keys in groups of 64 with NT = 2 145 us with 12 warps, 119 so with 12 (and with 16), with NT = 3
// 180 with 8, 160 so with 12.  (NT = 1 with 20 warps, which spill: groups of 128 152 us, with 16 137.)
BEAM_PLAN_FN constexpr int warps_of(int NT, int NG)
{
    return NT == 1 || (NT == 2 && NG == 1) ? 16 : 12;
}

}  // namespace kv4

// How one call is divided; a function of its sizes alone, for B * q_len * n_q < 2^31 and B > 0.
struct Kv4AttnPlan {
    int32_t heads;     // query heads of a KV head
    int32_t R;         // rows of a sequence and KV head: q_len * heads
    int32_t nt;        // 8-row tiles of a unit: 1, 2 or 3
    int32_t rtiles;    // units of a sequence and KV head
    int32_t teams;     // of n_kv * rtiles warps
    int32_t ctas, warps;  // of a block
    int32_t gang;      // 0: even shares of all keys; else the warps that take a unit whole
    int64_t bytes;     // workspace
};

inline Kv4AttnPlan kv4_attn_plan(int32_t B, int32_t q_len, int32_t n_q, int32_t n_kv, int64_t width,
                                 int64_t window, int64_t n_sink, int32_t group)
{
    using namespace kv4;
    Kv4AttnPlan p{};
    p.heads = n_q / n_kv;
    p.R = q_len * p.heads;
    const int64_t t8 = ((int64_t)p.R + 7) / 8;  // R: up to 2^31 - 1
    p.nt = t8 < 3 ? (int32_t)t8 : 3;
    p.rtiles = (int32_t)((t8 + p.nt - 1) / p.nt);
    // as many teams as all SMs' warps make, but no more than there can be tiles
    int64_t most = width;
    if (window > 0 && window < width && n_sink < width && window + q_len + n_sink < width)
        most = window + q_len + n_sink;
    const double tiles = (double)((most + kTile - 1) / kTile) * B;
    const int32_t team = n_kv * p.rtiles, warps = kSms * warps_of(p.nt, 128 / group);
    p.teams = team < warps ? warps / team : 1;
    p.teams = tiles < p.teams ? (int32_t)(tiles < 1 ? 1 : tiles) : p.teams;
    // few warps are spread over the SMs, but at least those that count the tiles stay together
    const int64_t all = (int64_t)p.teams * team;
    p.warps = (int32_t)((all + kSms - 1) / kSms);
    p.warps = p.warps < kScan / 32 ? kScan / 32 : p.warps;
    p.warps = p.warps < warps / kSms ? p.warps : warps / kSms;
    p.ctas = (int32_t)((all + p.warps - 1) / p.warps);
    p.ctas = p.ctas < kSms ? p.ctas : kSms;
    p.bytes = all * 2 * p.nt * 8 * (128 + 2) * 4;
    // Units whole, by gangs of up to 16 warps that join in shared memory, save the second kernel.  Two things have to hold.
    // No SM gets much more than its even share where all sequences are as long as they can be: it takes some 0.1 us a tile
    // and 8 rows.  And the longest unit is short, because a table says how long sequences may be, not how long they are:
    // one long sequence among short ones is left to its own gangs, at some 0.1 us a tile for each unit that a block has
    // in hand.  A window makes most units equally long, so more is allowed behind one.  Measured, whole and shares, us,
    // for tables that are filled; filled to a random length each; one of them filled and the others to a hundredth:
    //   19 sequences, 2000 keys   17.5 23.2; 15.9 20.3; 15.4 15.5     4000   27.4 31.8; 25.0 25.3; 22.2 21.0
    //                 8000        42.8 46.3; -; 36.2 30.8             100K   -; -; 354 59
    //   57 sequences, 1000 keys   23.3 28.1; 20.1 24.0; 19.7 15.1     2000   34.4 39.8; 32.2 30.0; 30.4 19.1
    //   128 sequences, 500 keys   26.3 33.5; 23.2 29.3; 22.6 13.2     1000   40.3 46.7; 38.9 36.4; 36.5 16.0
    //   1000 sequences, 200 keys  85.8 91.3; 60.3 76.1; 31.0 42.4
    //   19 of 4 tokens, 2000 keys 29.4 38.7; 29.8 34.3; 27.1 23.5     4000   44.7 52.9; 47.0 41.7; 40.8 32.7
    // and of one sequence of 500 keys 9.3 10.8, of 1000 11.4 10.6, of 2000 15.2 10.9; 8 of 1000 11.9 13.3, of 2000 15.9
    // 17.1, of 4000 22.6 20.7; behind a window of 512 128 sequences 29.6 35.8, of 1024 300 sequences 72 89, of 2048 50
    // sequences 34.9 39.5, 100 62 57, 128 72.8 67.0.
    const double units = (double)B * team;
    const int64_t unit_tiles = (most + kTile - 1) / kTile;
    const double even = units * (double)unit_tiles / kSms;
    const double each = (double)(int64_t)((units + kSms - 1) / kSms);  // units that some SM has to take
    const int32_t fit = warps_of(p.nt, 128 / group);
    const int32_t in_block = each < 1 ? 1 : (each < fit ? (int32_t)each : fit);
    const bool windowed = most < width;
    const bool brief = unit_tiles <= (windowed ? 40 : 17) || unit_tiles * in_block <= (windowed ? 200 : 128);
    if (brief && units < 1.0e9 && ((double)unit_tiles * each - even) * p.nt <= kGangExtra) {
        // as many warps to a unit as there are for `each` units at a time, and no more units to a block than that (128
        // sequences behind a window of 512, 1024 units: 147 blocks of 7 units 29.4 us, 128 of 8 30.2; 100 sequences
        // 25.7 and 29.6)
        const int64_t count = (int64_t)units, blocks = (count + in_block - 1) / in_block;
        p.gang = fit / in_block;
        p.warps = in_block * p.gang;
        p.ctas = (int32_t)(blocks < kSms * 64 ? (blocks < 1 ? 1 : blocks) : kSms * 64);
    }
    return p;
}

// ---------------------------------------------------------------------------------------------
// verification of drafted tokens
// ---------------------------------------------------------------------------------------------

constexpr int kVerifyWarps = 8;  // of a block

// Blocks of a sequence: 8 while each warp's stretch has 128 tokens.  Where not all blocks have room at a time (4 an SM)
// at most 4, and fewer while a block has less than 16,000 tokens, so that none gets more than 32,000 for it (128 rows of
// 160,000: 35.8 us with 8, 34.9 with 4, 53 with 2; 400 of 160,000: 73 with 4, 105 with 1; 1000 of 32,000: 57 with 4, 46
// with 2, 49 with 1; of 8000: 44 with 4, 20 with 1).  And as many as a grid holds.
inline int verify_ranks(int64_t B, int64_t V)
{
    int ranks = 8;
    while (ranks > 1 && V < (int64_t)ranks * kVerifyWarps * 128)
        ranks /= 2;
    while (ranks > 1 && B * ranks > 152 * 4 && (ranks == 8 || V < (int64_t)ranks * 16000))
        ranks /= 2;
    while (ranks > 1 && B * ranks > 0x7fffffff)
        ranks /= 2;
    return ranks;
}

}  // namespace beam
