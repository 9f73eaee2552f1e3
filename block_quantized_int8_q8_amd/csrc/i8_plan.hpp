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

struct I8Plan {
    int tile_m = 0, tile_n = 0, threads = 0;
    int64_t tiles_m = 0, tiles_n = 0;
};

// M rows in all (grouped: over all experts; experts = 0: one dense matrix).
// Returns false and says why when the launch cannot be made.
inline bool make_plan_i8(int64_t M, int64_t N, int64_t K, int experts, int cu_count, I8Plan *p, char *why,
                         size_t why_len) {
    (void)K;
    if (cu_count < 1) {
        std::snprintf(why, why_len, "device reports no compute units");
        return false;
    }
    p->tile_m = p->tile_n = 128;
    p->threads = 256;
    // a ragged grouping has at most one partial tile per non-empty expert
    p->tiles_m = experts ? M / p->tile_m + (M < experts ? M : experts) : (M + p->tile_m - 1) / p->tile_m;
    p->tiles_n = (N + p->tile_n - 1) / p->tile_n;
    if (p->tiles_m * p->tiles_n > INT32_MAX) {
        std::snprintf(why, why_len, "%lld x %lld output tiles exceed the grid's 2^31 - 1", (long long)p->tiles_m,
                      (long long)p->tiles_n);
        return false;
    }
    return true;
}

inline void describe_i8(const I8Plan &p, char *buf, size_t len) {
    std::snprintf(buf, len, "kernel=tile tile=%dx%d threads=%d tiles=%lldx%lld", p.tile_m, p.tile_n, p.threads,
                  (long long)p.tiles_m, (long long)p.tiles_n);
}

}  // namespace mmq
