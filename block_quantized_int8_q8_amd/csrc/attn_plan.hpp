// attn_plan.hpp -- layout of the int8 paged cache, shape checks and launch
// planning of the operators on it and of the rotary positions (pure host C++,
// no HIP calls, so that every refusal and every choice can be exercised
// without a GPU).
//
// The cache.  A page holds `page` tokens of every key/value head.  A head's
// part of a page is a run of tiles of 16 tokens, each 32 D + 128 bytes:
//   0      K codes  [D / 16][16 tokens][16]        (16 consecutive d)
//   16 D   V codes  [D / 64][4][64 d][4 tokens]    (4 consecutive tokens)
//   32 D   K scales fp32 [16 tokens]
//   +64    V scales fp32 [16 tokens]
// so that 64 lanes that load 16 bytes each read 1 KiB in a row and hold what
// the matrix instructions want of a lane: 16 values of one key, or four
// tokens of four value columns (the sum over tokens runs along the latter).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "i8_plan.hpp"

namespace mmq {

constexpr int64_t kv_tile_bytes(int D) { return 32 * int64_t(D) + 128; }
constexpr bool kv_dim_ok(int64_t D) { return D == 64 || D == 128 || D == 256; }
constexpr bool kv_page_ok(int64_t page) { return page == 16 || page == 32 || page == 64 || page == 128 || page == 256; }

constexpr int64_t kMaxTokens = int64_t(1) << 24;      // of one call: its grid stays below 2^32 threads
constexpr int kMaxHeads = 1024;
constexpr int kRopeMaxDim = 512;
constexpr int64_t kMaxStride = int64_t(1) << 40;

inline const char *check_kv_cache(int64_t n_pages, int page, int heads, int D) {
    if (!kv_dim_ok(D)) return "the head dimension must be 64, 128 or 256";
    if (!kv_page_ok(page)) return "a page must hold 16, 32, 64, 128 or 256 tokens";
    if (heads < 1 || heads > kMaxHeads) return "the cache must have 1..1024 heads";
    if (n_pages < 1 || n_pages > INT32_MAX / page) return "the cache must hold 1..2^31-1 tokens";
    if (n_pages * (page / 16) > INT32_MAX / heads) return "the cache must hold fewer than 2^31 tiles of 16 tokens and a head";
    return nullptr;
}

// Token and head strides of a [T, H, D] operand that is only read.
inline const char *check_strides(int64_t ldt, int64_t ldh) {
    if (ldt < 0 || ldh < 0 || ldt > kMaxStride || ldh > kMaxStride) return "strides must be 0..2^40 elements";
    return nullptr;
}
// ... of one that is written: no element may have two places in it.
inline const char *check_out_strides(int64_t T, int64_t H, int64_t D, int64_t ldt, int64_t ldh) {
    if (const char *bad = check_strides(ldt, ldh)) return bad;
    if (T == 0) return nullptr;
    const bool heads_inside = (H == 1 || ldh >= D) && (T == 1 || ldt >= (H - 1) * ldh + D);
    // ldh >= (T - 1) * ldt + D, of which the product may pass 64 bits
    const bool tokens_inside = (T == 1 || ldt >= D) && (H == 1 || (ldh >= D && (T == 1 || ldt <= (ldh - D) / (T - 1))));
    if (!heads_inside && !tokens_inside) return "the output's tokens or heads overlap";
    return nullptr;
}

inline const char *check_tokens(int64_t T, int H) {
    if (T < 0 || T > kMaxTokens) return "the number of tokens must be 0..2^24";
    if (H < 1 || H > kMaxHeads) return "the number of heads must be 1..1024";
    return nullptr;
}

// Scalings of the rotary frequencies (their formulas: rope_frequencies).
enum RopeScaling : int { ROPE_PLAIN = 0, ROPE_LINEAR = 1, ROPE_BANDS = 2, ROPE_YARN = 3 };

inline const char *check_frequencies(int scaling, int rot, double base, double factor, double low, double high,
                                     int64_t original) {
    if (scaling < ROPE_PLAIN || scaling > ROPE_YARN) return "unknown scaling";
    if (rot < 2 || rot % 2 || rot > kRopeMaxDim) return "the rotated part must be an even number of values in 2..512";
    if (!(base > 1.0) || !std::isfinite(base)) return "the base must be above 1";
    if (scaling == ROPE_PLAIN) return nullptr;
    if (!(factor > 0.0) || !std::isfinite(factor)) return "the factor must be above 0";
    if (scaling == ROPE_LINEAR) return nullptr;
    if (!(low > 0.0) || !(high > low) || !std::isfinite(high)) return "low and high must be 0 < low < high (turns within the original length)";
    if (original < 1) return "the original length must be at least 1";
    return nullptr;
}

// freqs[i]: radians per position of pair i.  A frequency that makes `high`
// turns or more within the original length is kept, one that makes `low` or
// fewer is divided by the factor, with a ramp between: linear in the turns
// (bands), or in the number of the pair, between the pairs at which those
// turns fall, rounded outwards (yarn, which also scales the rotated values).
inline void rope_frequencies(int scaling, int rot, double base, double factor, double low, double high, int64_t original,
                             double *freqs, double *mscale) {
    constexpr double kTurn = 6.283185307179586477;
    *mscale = scaling == ROPE_YARN && factor > 1.0 ? 0.1 * std::log(factor) + 1.0 : 1.0;
    auto pair_of = [&](double turns) { return rot * std::log(double(original) / (turns * kTurn)) / (2.0 * std::log(base)); };
    double first = 0.0, last = 0.0;
    if (scaling == ROPE_YARN) {
        first = std::max(std::floor(pair_of(high)), 0.0);
        last = std::min(std::ceil(pair_of(low)), rot - 1.0);
    }
    for (int i = 0; i < rot / 2; i++) {
        const double f = std::pow(base, -2.0 * i / rot);
        double keep = 0.0;
        if (scaling == ROPE_PLAIN) keep = 1.0;
        if (scaling == ROPE_BANDS) keep = (double(original) * f / kTurn - low) / (high - low);
        if (scaling == ROPE_YARN) keep = 1.0 - (i - first) / std::max(last - first, 0.001);
        keep = std::min(std::max(keep, 0.0), 1.0);
        freqs[i] = scaling == ROPE_PLAIN ? f : f / factor * (1.0 - keep) + f * keep;
    }
}

inline const char *check_rope(int D, int rot, int layout) {
    if (D < 8 || D > kRopeMaxDim || D % 8) return "the head dimension must be a multiple of 8 in 8..512";
    if (rot < 2 || rot % 2 || rot > D) return "the rotated part must be an even number of values in 2..head dimension";
    if (layout != 0 && layout != 1) return "unknown layout of the rotated pairs";
    return nullptr;
}

// Attention.  Rows are (new token, query head of the group) pairs; a
// sequence of few rows runs in the rows kernel, of more in the tile kernel.
// Both kernels decide from the sequence's own row count on the device, so a
// batch may mix them.  Where the border lies: 16 sequences of 8192 keys, 32 on
// 4 heads of 128, 8, 16 and 32 rows each in the rows kernel 32, 33 and 51 us;
// 40, 64 and 128 rows in the tile kernel 71, 72 and 78.
constexpr int kAttnFewRows = 32;          // most rows of a sequence in the rows kernel
constexpr int kAttnRowsChunk = 128;       // keys: least share of a workgroup of the rows kernel
constexpr int kAttnTileChunk = 256;       // ... of the tile kernel
constexpr int kAttnAlongKeys = 8192;      // keys from which the tile kernel takes no few-row sequence along

struct AttnPlan {
    int few_tiles;            // rows kernel: 16-row blocks per workgroup (1, 2); 0: not launched
    int few_split;            // ... most shares of a sequence's keys
    int64_t few_grid;
    int tile_rows;            // tile kernel: rows per workgroup; 0: not launched
    int tile_split;
    int64_t tiles, tile_grid; // tiles: most row tiles there can be
    int few_target, tile_target;     // workgroups of each that the device runs at once
    int64_t few_bytes, tile_bytes;   // workspace of each, 256-byte multiples
};

inline const char *check_attention(int64_t T, int64_t B, int Hq, int Hkv, int D, int64_t max_pages, int page, int64_t max_q) {
    if (const char *bad = check_tokens(T, Hq)) return bad;
    if (T * Hq > (int64_t(1) << 30)) return "new tokens times query heads must be at most 2^30";
    if (!kv_dim_ok(D)) return "the head dimension must be 64, 128 or 256";
    if (!kv_page_ok(page)) return "a page must hold 16, 32, 64, 128 or 256 tokens";
    if (B < 0 || B > (int64_t(1) << 20)) return "the number of sequences must be 0..2^20";
    if (Hkv < 1 || Hq % Hkv) return "the query heads must be a multiple of the key/value heads";
    if (max_pages < 0 || max_pages > (1 << 30) / page) return "a sequence's pages must hold at most 2^30 tokens";
    if (max_q < 1) return "max_q must be at least 1";
    return nullptr;
}

inline int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

inline bool make_plan_attention(int64_t T, int64_t B, int Hq, int Hkv, int D, int64_t max_pages, int page, int64_t max_q,
                                int cu_count, AttnPlan *p, char *why, size_t len) {
    *p = AttnPlan{};
    const int64_t G = Hq / Hkv, max_keys = max_pages * page;
    if (max_q > T) max_q = T;
    const int64_t most_rows = max_q * G;
    // Three workgroups of the rows kernel a CU: four of one row block with heads
    // of 64 and 128 are resident (128 registers), and the shares' remainders
    // take the fourth's place (64 sequences of 2K to 16K keys, kernel and join
    // together: target of 2 per CU 122 us, 3 112, 4 129, 6 118; one of 256K keys
    // 59, 61, 64, 67).  Of two row blocks with heads of 64 three are resident,
    // with heads of 128 two, of heads of 256 two and one: there the same target
    // runs its shares in rounds (64 sequences of 8192 keys with heads of 256 211
    // us, 213 by the bytes).
    p->few_target = 3 * cu_count;
    p->tile_target = D == 64 ? 2 * cu_count : cu_count;
    auto ceil_div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    // Where sequences have many rows on the average, the tile kernel takes the
    // few-row ones along: they run beside its tiles, the rows kernel would
    // run before them (24 sequences, half of them decoding, half chunks of up
    // to 700 tokens: 160 -> 145 us; one prompt: a launch less).  Not where one
    // of them may hold many keys, which the tile kernel does not split once its
    // tiles fill the device, 2 us for 64 keys: along and apart, a prompt of 2048
    // tokens and one decoded token over 4096 keys 83 and 93 us, over 8192 107 and
    // 89, over 256K 2640 and 176; a prompt of 8192 and seven over 256K 5350 and
    // 920; 24 mixed ones of up to 8192 keys 403 and 419.  (What a table could hold
    // decides, as lengths are on the device: one with room for more than its
    // sequences have pays the second launch, about 10 us, for nothing.)
    // And where T says that all have max_q, none has few (16 sequences of 40
    // rows over 8192 keys 75 -> 71 us); a batch padded to B max_q rows says so
    // too, and has its short sequences in the tile kernel.
    if (most_rows <= kAttnFewRows || (G <= kAttnFewRows && T < B * max_q && (T * G < 128 * B || max_keys >= kAttnAlongKeys))) {
        p->few_tiles = (most_rows < kAttnFewRows ? most_rows : kAttnFewRows) > 16 ? 2 : 1;
        const int64_t units = B * Hkv;
        int64_t s = ceil_div(4 * int64_t(p->few_target), units);        // lengths differ: more shares than the device needs
        const int64_t most = ceil_div(max_keys + kAttnRowsChunk, kAttnRowsChunk);
        if (units >= p->few_target) s = 1;
        if (s > most) s = most;
        if (s > 512) s = 512;
        p->few_split = int(s < 1 ? 1 : s);
        p->few_grid = units * p->few_split;
        if (p->few_split > 1) p->few_bytes = up256(p->few_grid * 16 * p->few_tiles * (D + 2) * 4 + units * 4);
    }
    if (most_rows > kAttnFewRows) {
        p->tile_rows = D == 128 ? 256 : 128;
        p->tiles = T * G / p->tile_rows + (T < B ? T : B);
        if (p->tiles < 1) p->tiles = 1;
        const int64_t units = p->tiles * Hkv;
        int64_t s = 2 * int64_t(p->tile_target) / units;
        const int64_t most = ceil_div(max_keys + kAttnTileChunk, kAttnTileChunk);
        if (s > most) s = most;
        p->tile_split = int(s < 1 ? 1 : s);
        p->tile_grid = units * p->tile_split;
        if (p->tile_split > 1) p->tile_bytes = up256(p->tile_grid * p->tile_rows * (D + 2) * 4);
    }
    // a launch holds fewer than 2^32 threads
    if (p->few_grid >= (int64_t(1) << 23) || p->tile_grid >= (int64_t(1) << 22)) {
        std::snprintf(why, len, "too many workgroups for one launch");
        return false;
    }
    return true;
}

}  // namespace mmq
