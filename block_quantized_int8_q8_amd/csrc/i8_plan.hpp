// i8_plan.hpp -- shape checks and launch planning of the per-token /
// per-channel int8 operators (pure host C++, no HIP calls, so that every
// refusal and every choice can be exercised without a GPU).
#pragma once

#include <cstdint>
#include <cstdio>

namespace mmq {

enum Type : int { TYPE_F32 = 0, TYPE_BF16 = 1, TYPE_F16 = 2 };

constexpr bool type_ok(int t) { return t == TYPE_F32 || t == TYPE_BF16 || t == TYPE_F16; }
constexpr int type_bytes(int t) { return t == TYPE_F32 ? 4 : 2; }
constexpr const char *type_name(int t) { return t == TYPE_F32 ? "fp32" : t == TYPE_BF16 ? "bf16" : "fp16"; }

// Longest row: 128 * 128 * K stays below 2^31, so the int32 sum over a whole
// row is exact for any codes.
constexpr int64_t kI8MaxK = 131056;
// Row pitch bound: the offset of any byte of a tile's 256 rows fits 31 bits.
constexpr int64_t kI8MaxPitch = int64_t(1) << 22;
constexpr int kI8MaxExperts = 2048;

constexpr int64_t pad16(int64_t k) { return (k + 15) / 16 * 16; }

// Checks shared by the two row quantizers: nullptr when they are fine.
inline const char *check_quantize_i8(int64_t M, int64_t K, int64_t ldx, int64_t ldq) {
    if (M < 0 || K < 1) return "M must be >= 0 and K >= 1";
    if (M > INT32_MAX) return "M must be below 2^31";
    if (K > kI8MaxK) return "K must be at most 131056";
    if (ldx < K) return "the input's row pitch is shorter than a row";
    if (ldx > (int64_t(1) << 40)) return "the input's row pitch must be at most 2^40";
    if (ldq < pad16(K) || ldq % 16) return "the codes' row pitch must be a multiple of 16 that holds K rounded up to 16";
    if (ldq > kI8MaxPitch) return "the codes' row pitch must be at most 2^22";
    return nullptr;
}

inline const char *check_gemm_i8(int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldw, int64_t ldo) {
    if (M < 0 || N < 1 || K < 1) return "M must be >= 0, N and K >= 1";
    if (M > INT32_MAX || N > INT32_MAX) return "M and N must be below 2^31";
    if (K % 16) return "K must be a multiple of 16 (pad the codes with zeros)";
    if (K > kI8MaxK) return "K must be at most 131056 (the int32 sum of a row)";
    if (ldx < K || ldw < K || ldx % 16 || ldw % 16)
        return "the codes' row pitches must be multiples of 16 that hold K values";
    if (ldx > kI8MaxPitch || ldw > kI8MaxPitch) return "the codes' row pitches must be at most 2^22";
    if (ldo < N) return "the output's row pitch is shorter than a row";
    if (ldo > (int64_t(1) << 40)) return "the output's row pitch must be at most 2^40";
    return nullptr;
}

// Kernels of the products: the tile kernel (tiles of BM x BN outputs), and
// the rows kernel (workgroups of BM x BN outputs that split K over waves).
enum I8Kernel : int {
    I8_TILE_256x256, I8_TILE_128x256, I8_TILE_128x128, I8_TILE_64x128,
    I8_ROWS_16x16, I8_ROWS_16x32, I8_ROWS_32x32, I8_ROWS_32x64, I8_ROWS_64x64,
    I8_KERNELS
};
struct I8KernelInfo {
    const char *name;
    int tile_m, tile_n, threads;
    int per_cu;                // workgroups resident per CU (tile kernels: their LDS; they walk over the tiles)
    // microseconds of one 128-wide k-step of one tile, and of a tile's start
    // and end, with every CU at work (measured at K = 3584 and 18944).  Memory
    // traffic is not in them: at short K, where it counts, the sums fall short
    // (12008 rows of 128 experts, 2048 x 768: 54 us said, 84 taken) and only
    // rank the tiles
    double step_us, fixed_us;
};
constexpr I8KernelInfo kI8Kernels[I8_KERNELS] = {
    {"tile", 256, 256, 512, 1, 1.40, 9.0}, {"tile", 128, 256, 512, 1, 0.87, 5.5}, {"tile", 128, 128, 256, 2, 0.51, 3.0},
    {"tile", 64, 128, 256, 2, 0.30, 2.0},  {"rows", 16, 16, 256, 0, 0.0, 0.0},    {"rows", 16, 32, 256, 0, 0.0, 0.0},
    {"rows", 32, 32, 256, 0, 0.0, 0.0},    {"rows", 32, 64, 256, 0, 0.0, 0.0},    {"rows", 64, 64, 256, 0, 0.0, 0.0},
};

struct I8Plan {
    int kernel = 0, tile_m = 0, tile_n = 0, threads = 0;
    int64_t tiles_m = 0, tiles_n = 0, workgroups = 0;
};

constexpr int64_t kI8BufBytes = 0xfffff000LL;

// Tiles along the rows: `experts` groups (0: one dense matrix) of M rows in
// all have at most one partial tile each.
inline int64_t i8_row_tiles(int64_t M, int experts, int tile_m) {
    return experts ? M / tile_m + (M < experts ? M : experts) : (M + tile_m - 1) / tile_m;
}

// M rows in all (grouped: over all experts; experts = 0: one dense matrix).
// Returns false and says why when the launch cannot be made.
inline bool make_plan_i8(int64_t M, int64_t N, int64_t K, int experts, int cu_count, I8Plan *p, char *why,
                         size_t why_len) {
    if (cu_count < 1) {
        std::snprintf(why, why_len, "device reports no compute units");
        return false;
    }
    // rows that share a weight matrix, on average, and the tiles to expect: a
    // group's last row tile is half full on average
    const int64_t per = experts ? (M + experts - 1) / experts : M, groups = experts ? (M < experts ? M : experts) : 0;
    auto tiles_of = [&](int v) {
        const I8KernelInfo &k = kI8Kernels[v];
        const int64_t row_tiles = experts ? M / k.tile_m + (groups + 1) / 2 : (M + k.tile_m - 1) / k.tile_m;
        return row_tiles * ((N + k.tile_n - 1) / k.tile_n);
    };
    // The rows kernel where a weight matrix meets few rows (16 x 18944 x 3584
    // 13.0 us against 14.5 in 64 x 128 tiles, 4 rows for each of 128 experts
    // 73.4 against 74.3, 16 rows 101 against 78) and where the smallest tiles
    // would leave half the CUs without one (128 x 3584 x 18944, 56 tiles: 22.3
    // against 48.1; 256 x 3584 x 3584, 112 tiles: 11.2 against 12.9).
    if (per <= (experts ? 4 : 16) || tiles_of(I8_TILE_64x128) * 2 < cu_count) {
        // the largest workgroup that still makes about one per CU: 64 x 3584 x
        // 18944 as 16 x 32 22.9, 32 x 32 16.2, 32 x 64 (112 of them) 22.3
        p->kernel = I8_ROWS_16x16;
        for (int v = I8_ROWS_16x32; v <= I8_ROWS_64x64; v++)
            if ((kI8Kernels[v].tile_m == 16 || per > kI8Kernels[v].tile_m / 2) && tiles_of(v) * 5 >= cu_count * 4) p->kernel = v;
    } else {
        const int64_t steps = (K + 127) / 128;
        double best = 0;
        for (int v = I8_TILE_256x256; v <= I8_TILE_64x128; v++) {
            const I8KernelInfo &k = kI8Kernels[v];
            const double us = double((tiles_of(v) + cu_count - 1) / cu_count) * (double(steps) * k.step_us + k.fixed_us);
            if (v == I8_TILE_256x256 || us < best) {
                best = us;
                p->kernel = v;
            }
        }
    }
    const I8KernelInfo &k = kI8Kernels[p->kernel];
    p->tile_m = k.tile_m;
    p->tile_n = k.tile_n;
    p->threads = k.threads;
    p->tiles_m = i8_row_tiles(M, experts, p->tile_m);
    p->tiles_n = (N + p->tile_n - 1) / p->tile_n;
    p->workgroups = p->tiles_m * p->tiles_n;
    if (p->workgroups > INT32_MAX) {
        std::snprintf(why, why_len, "%lld x %lld output tiles exceed the grid's 2^31 - 1", (long long)p->tiles_m,
                      (long long)p->tiles_n);
        return false;
    }
    if (k.per_cu && p->workgroups > int64_t(cu_count) * k.per_cu) p->workgroups = int64_t(cu_count) * k.per_cu;
    if (p->workgroups * p->threads > UINT32_MAX) {
        std::snprintf(why, why_len, "%lld output tiles of %d threads exceed a launch's 2^32 - 1 threads",
                      (long long)p->workgroups, p->threads);
        return false;
    }
    if (M > INT32_MAX - 512 || N > INT32_MAX - 512) {
        std::snprintf(why, why_len, "the last output tile would pass 2^31 rows or columns");
        return false;
    }
    return true;
}

inline void describe_i8(const I8Plan &p, char *buf, size_t len) {
    std::snprintf(buf, len, "kernel=%s tile=%dx%d threads=%d tiles=%lldx%lld workgroups=%lld", kI8Kernels[p.kernel].name, p.tile_m,
                  p.tile_n, p.threads, (long long)p.tiles_m, (long long)p.tiles_n, (long long)p.workgroups);
}

}  // namespace mmq
