// attn_kernels.hip -- gfx950 kernels of attention over the int8 paged cache.
//
//   k_attn_rows   sequences of few rows (decoding: one token, its group of
//                 query heads): keys and values straight into registers
//   k_attn_tile   sequences of many rows (a chunk of a prompt): keys and
//                 values converted once per workgroup, through LDS
//   k_attn_join_rows, k_attn_join_tiles
//                 join the shares that they split a sequence's keys into
//
// A row is one (new token, query head) pair; the rows of a sequence that read
// the same key/value head are multiplied together.  With codes c and scales d
// of the cache,
//     s_t = scale * dk_t * (q . ck_t),   o = sum_t exp(s_t) dv_t cv_t / sum_t exp(s_t)
// over the keys t that the row may see.  Codes are at most 127 in magnitude
// and so exact in 16 bits: the two products run on the 16-bit matrix core
// with q and the codes as they are, both scales are applied in fp32, and the
// one rounding between q and the result is that of exp(s_t) dv_t, which the
// second product reads in 16 bits (the type of q).  Sums, maxima and the running
// output are fp32.
//   The weights' bits are chosen by what they cost.  Where the output is fp32,
// and in the rows kernel always, what the rounding leaves is rounded too and
// multiplied by a second product (16 bits in bf16, 22 in fp16): fp32 outputs
// would have no use for theirs otherwise, and the rows kernel waits for memory
// (64 sequences 109 -> 110.5 us; the mean error against 64 bits falls from
// 0.0022 to 0.0014 of the mean magnitude, what the output's own rounding
// leaves).  In the tile kernel it takes the 8K prompt from 535 to 707 us, so
// there a 16-bit output has weights of as many bits as itself (0.0022).
//
// Both products are formed transposed, keys (or value columns) by rows, so
// that a lane holds scores of one row only: the maximum and the sum of a
// softmax are per-lane numbers, and the scores' registers are, converted,
// the second product's operand with no movement between lanes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attn_plan.hpp"
#include "wave_scan.hpp"

namespace mmq {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

struct AttnArgs {
    const void *q;            // [T, Hq, D]
    int64_t qdt, qdh;
    const uint8_t *cache;
    const int32_t *table;     // [B, max_pages] pages
    const int32_t *lens;      // [B] keys, the new tokens' own included
    const int32_t *offsets;   // [B + 1] bounds of each sequence's new tokens
    void *out;                // [T, Hq, D]
    int64_t odt, odh;
    int64_t n_pages, max_pages;
    int page_shift, Hkv, G;
    int T, B, max_q, window;
    float scale;              // softmax scale times log2(e)
    float *part;              // shares: outputs, then (reference, sum) pairs
    int split, target;        // most shares; workgroups that fill the device
    int units;                // rows kernel: B; tile kernel: row tiles there can be
    int few_rows;             // most rows of a sequence of the rows kernel
};

// --- 16-bit types -----------------------------------------------------------
template <typename T> struct Half;
template <> struct Half<__bf16> {
    typedef bf16x8 x8;
    static __device__ __forceinline__ f32x4 mfma16(x8 a, x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ f32x16 mfma32(x8 a, x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
    // Four int8 codes as two dwords.  Integers below 256 have zeros in the low half of their fp32 form.
    static __device__ __forceinline__ void codes(uint32_t c, uint32_t (&o)[2]) {
        const uint32_t f0 = __float_as_uint(float(int8_t(c))), f1 = __float_as_uint(float(int8_t(c >> 8)));
        const uint32_t f2 = __float_as_uint(float(int8_t(c >> 16))), f3 = __float_as_uint(float(int8_t(c >> 24)));
        o[0] = __builtin_amdgcn_perm(f1, f0, 0x07060302u);
        o[1] = __builtin_amdgcn_perm(f3, f2, 0x07060302u);
    }
};
template <> struct Half<_Float16> {
    typedef f16x8 x8;
    static __device__ __forceinline__ f32x4 mfma16(x8 a, x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ f32x16 mfma32(x8 a, x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
    // code + 128 as the low bits of 1024 + code + 128, less 1152: exact.
    static __device__ __forceinline__ void codes(uint32_t c, uint32_t (&o)[2]) {
        const uint32_t u = c ^ 0x80808080u;
        const f16x2 m = {_Float16(1152.0f), _Float16(1152.0f)};
        o[0] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - m);
        o[1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - m);
    }
};

template <typename T>
__device__ __forceinline__ typename Half<T>::x8 codes8(uint32_t lo, uint32_t hi) {
    uint32_t a[2], b[2];
    Half<T>::codes(lo, a);
    Half<T>::codes(hi, b);
    const u32x4 v = {a[0], a[1], b[0], b[1]};
    return __builtin_bit_cast(typename Half<T>::x8, v);
}

template <typename T>
__device__ __forceinline__ typename Half<T>::x8 load_x8(const T *p) {
    typename Half<T>::x8 v;
    __builtin_memcpy(&v, p, 16);                 // rows may start at any multiple of the type's size
    return v;
}

template <typename O>
__device__ __forceinline__ void store4(O *p, f32x4 v) {
    O t[4] = {O(v[0]), O(v[1]), O(v[2]), O(v[3])};
    __builtin_memcpy(p, t, sizeof(t));
}

// --- sequences --------------------------------------------------------------
struct Seq {
    int start, n;             // rows of q: first new token, how many
    int len, pos0;            // keys; position of the first new token (negative: it and those up to 0 see nothing)
};

__device__ __forceinline__ int clamp_row(const AttnArgs &a, int v) { return min(max(v, 0), a.T); }
__device__ __forceinline__ int clamp_len(const AttnArgs &a, int v) {
    return int(min(int64_t(max(v, 0)), a.max_pages << a.page_shift));
}
__device__ __forceinline__ Seq sequence(const AttnArgs &a, int b) {
    const int s = clamp_row(a, a.offsets[b]), n = max(clamp_row(a, a.offsets[b + 1]) - s, 0);
    const int len = clamp_len(a, a.lens[b]);
    return Seq{s, min(n, a.max_q), len, len - n};
}
__device__ __forceinline__ bool has_few_rows(const AttnArgs &a, int n) { return int64_t(n) * a.G <= a.few_rows; }

// The keys [begin, end) that tokens first .. last of a sequence see among
// them; begin is rounded down to a tile of 16.
struct Range {
    int begin, end;
    __device__ __forceinline__ Range(const AttnArgs &a, const Seq &s, int first, int last) {
        end = max(s.pos0 + last + 1, 0);
        begin = a.window ? max(s.pos0 + first - a.window + 1, 0) & ~15 : 0;
        if (begin >= end) begin = end = 0;
    }
};

// Tile number in the cache of 16-key tile k16 of sequence b, head h; -1 for a
// page that the cache does not have.
__device__ __forceinline__ int cache_tile(const AttnArgs &a, int b, int h, int k16) {
    const int sh = a.page_shift - 4, page = a.table[int64_t(b) * a.max_pages + (k16 >> sh)];
    if (uint32_t(page) >= uint32_t(a.n_pages)) return -1;
    return ((page * a.Hkv + h) << sh) + (k16 & ((1 << sh) - 1));
}

__device__ __forceinline__ int wave_sum(int v) { return __builtin_amdgcn_readlane(scan_sum(v), 63); }
__device__ __forceinline__ int wave_max(int v) { return __builtin_amdgcn_readlane(scan_max(v), 63); }

// Keys of each share of the rows kernel: such that all few-row sequences'
// shares together fill the device, at most `split` of them for the longest.
__device__ __forceinline__ int few_chunk(const AttnArgs &a) {
    const int lane = threadIdx.x & 63;
    int most = 0;
    float total = 0.0f;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        int k = 0;
        if (b0 + lane < a.B) {
            const Seq s = sequence(a, b0 + lane);
            if (s.n > 0 && has_few_rows(a, s.n)) {
                const Range r(a, s, 0, s.n - 1);
                k = r.end - r.begin;
            }
        }
        most = max(most, wave_max(k));
        total += float(wave_sum(k >> 7)) + 1.0f;          // 128-key blocks
    }
    // a share of the keys of every head for each of the `target` workgroups
    const float blocks = total * float(a.Hkv) / float(a.target);
    const int by_device = int(fminf(blocks, 1e6f)) + 1, by_slots = ((most + a.split - 1) / a.split + 127) >> 7;
    return max(max(by_device, by_slots), 1) << 7;
}

// ---------------------------------------------------------------------------
// Softmax of the transposed scores in a lane's registers.
//
// Scores t are in units of log2.  The second product's operand is a weight
// times its value's scale dv in 16 bits, and that scale goes into the exponent:
//   p' = 2^(t + log2 dv - m) = p dv,   the sum of the weights takes p' / dv,
// one FMA on the product where two multiplications were.  m is a running
// reference of the row, which moves up only, and only when that row has a new
// maximum of t + log2 dv more than 2^8 above the last: the largest p' lies
// between 2^6 and 2^14, within fp16's exponents (-24 to 15) whatever the size
// of dv.
//   A p' below 2^-126 is lost from the sum of the weights too, so a value's
// scale counts as some least one: 2^-100, or 2^-108 of the largest so far where
// that is above 2^8 (values past 32000; in the rows kernel, of the largest that
// the row sees and that moved its reference, and in the tile kernel of all that
// its workgroup has read).  So keys, those of zeros among them, keep their
// weight beside values of any size: none above 2^-23 of the row's largest is
// lost.
//   The sum may stand far from the reference, from 2^-115 (one value, the
// largest there is) to 2^139 (2^25 values of next to nothing): it is held in
// units of 2^12, so that neither end leaves fp32 (values past 2^121 leave its
// terms 16 bits), and where the reference moves it is scaled in two halves,
// since 2^(m - m') may be below 2^-126 where the sum times it is not.
// ---------------------------------------------------------------------------
constexpr float kSlack = 8.0f;
constexpr float kTop = 6.0f;
constexpr float kLeastScale = 0x1p-100f, kLargeScale = 0x1p8f, kScaleRange = 0x1p-108f;
constexpr float kSumUnit = 0x1p12f;

// The least scale, raised by a wave's scales of which some are large.
__device__ __forceinline__ float raised_least(float least, float scale) {
    scale = scale == scale ? scale : 0.0f;
#pragma unroll
    for (int o = 32; o; o >>= 1) scale = fmaxf(scale, __shfl_xor(scale, o));
    return fmaxf(least, scale * kScaleRange);
}

// 2^x times a sum, whatever the size of 2^x alone.
__device__ __forceinline__ float scaled_sum(float l, float x) {
    const float h = __builtin_amdgcn_exp2f(0.5f * x);
    return l * h * h;
}
// Outputs over their sum of weights (in its units; 0: the row saw nothing).
// Neither end of the sum's range has a reciprocal in fp32 as it is.
__device__ __forceinline__ f32x4 over_sum(f32x4 o, float l) {
    if (l == 0.0f) return f32x4{0, 0, 0, 0};
    const bool low = l < 1.0f;
    return o * (1.0f / (low ? l * 0x1p32f : l)) * (low ? 0x1p32f / kSumUnit : 1.0f / kSumUnit);
}

// The larger of the values of lanes i and i + 32, in both.
__device__ __forceinline__ float max_of_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// --- rows kernel ------------------------------------------------------------
//
// Bound by the cache's bytes.  A workgroup is one sequence and key/value head
// (and a share of its keys); each of its four waves takes 32 keys at a time
// straight into the operands' registers: the cache's layout is that of the
// matrix instruction's fragments, 1 KiB a load, no LDS and no wait for
// another wave before the end.  Rows are the other operand, 16 or 32 of them,
// so that a group of query heads reads its keys once.
//   64 sequences of 2K to 16K keys, 28 on 4 heads of 128: 104 us for 506 MB =
//   4.9 TB/s (a copy moves 5.12), and 6.5 for the join of its shares
//   one sequence of 256K keys, 32 on 4 heads: 61 us for 277 MB, join 8
//   one of 2011 keys: 7.3 us, a chain of offsets, pages, keys; join 3.6
// Heads of 64 have half the bytes for the same softmax, about 260 vector
// instructions for 32 keys: 64 sequences of 8192 keys 61 us in bf16 and 57 in
// fp16 (53 and 54 with weights of one part, and the sum not held apart from the
// values' sizes) against 56 for the bytes; heads of 128 106 (106), of 256 211
// (216).
template <typename T, typename O, int D, int RT>
__global__ __launch_bounds__(256) void k_attn_rows(AttnArgs a) {
    typedef typename Half<T>::x8 x8;
    constexpr int C = D / 64, TILE = int(kv_tile_bytes(D)), R = 16 * RT;
    constexpr float NEG = -__builtin_inff();
    __shared__ float S_o[4][R][68];
    __shared__ float S_m[4][R], S_l[4][R];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, g = lane >> 4;
    const int h = blockIdx.x % a.Hkv, rest = blockIdx.x / a.Hkv, b = rest % a.B, share = rest / a.B;
    const Seq s = sequence(a, b);
    const int rows = s.n * a.G;
    if (s.n == 0 || !has_few_rows(a, s.n)) return;
    const Range all(a, s, 0, s.n - 1);
    int chunk = 0x7fffff80;
    if (a.split > 1) chunk = few_chunk(a);
    const int begin = all.begin + min(int64_t(share) * chunk, int64_t(all.end - all.begin)), end = min(int64_t(all.end), int64_t(begin) + chunk);
    const bool alone = all.end - all.begin <= chunk;
    if (a.split > 1 && share == 0 && threadIdx.x == 0) {                   // for the join: how many shares there are
        float *ml = a.part + int64_t(a.units) * a.Hkv * a.split * R * (D + 2);
        reinterpret_cast<int *>(ml)[b * a.Hkv + h] = (all.end - all.begin + chunk - 1) / chunk;
    }
    if (begin >= end && share > 0) return;
    const bool two = RT > 1 && rows > 16;

    // this lane's rows: one of each block of 16
    int pos[RT];
    const uint32_t span = a.window ? uint32_t(a.window) : 0x80000000u;      // keys that a row sees, up to its position
    x8 q[RT][2 * C];
#pragma unroll
    for (int rb = 0; rb < RT; rb++) {
        const int r = 16 * rb + col, i = r / a.G;
        const bool there = r < rows;
        pos[rb] = there ? s.pos0 + i : -1;
        const T *qr = static_cast<const T *>(a.q) + int64_t(s.start + (there ? i : 0)) * a.qdt + int64_t(h * a.G + (there ? r - i * a.G : 0)) * a.qdh;
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int e = 0; e < 2; e++) q[rb][2 * c + e] = load_x8(qr + 64 * c + 16 * g + 8 * e);
    }
    float m[RT], l[RT], least[RT];
    f32x4 o[RT][C][4];
#pragma unroll
    for (int rb = 0; rb < RT; rb++) {
        m[rb] = NEG;
        l[rb] = 0.0f;
        least[rb] = kLeastScale;
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int k = 0; k < 4; k++) o[rb][c][k] = f32x4{0, 0, 0, 0};
    }

    // wave w takes the 32-key units w, w + 4, ... of the share
    const int units = (end - begin + 31) / 32;
    int tiles = -1;
    for (int u = wv, it = 0; u < units; u += 4, it++) {
        if ((it & 31) == 0) {                                        // the tiles of this unit and the 31 behind it
            const int k16 = begin / 16 + 2 * (u + 4 * (lane >> 1)) + (lane & 1);
            tiles = 16 * k16 < end ? cache_tile(a, b, h, k16) : -1;
        }
        const int key0 = begin + 32 * u;
        u32x4 kc[2][C], vc[2][C];
        f32x4 ks[2], vs[2];
        bool there[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int t = __builtin_amdgcn_readlane(tiles, 2 * (it & 31) + j);
            there[j] = t >= 0;
            const uint8_t *p = a.cache + int64_t(max(t, 0)) * TILE;  // a tile that is not there: any, and masked
#pragma unroll
            for (int c = 0; c < C; c++) {
                kc[j][c] = *reinterpret_cast<const u32x4 *>(p + c * 1024 + lane * 16);
                vc[j][c] = *reinterpret_cast<const u32x4 *>(p + 16 * D + c * 1024 + lane * 16);
            }
            ks[j] = *reinterpret_cast<const f32x4 *>(p + 32 * D + 16 * g);
            vs[j] = *reinterpret_cast<const f32x4 *>(p + 32 * D + 64 + 16 * g);
        }
        f32x4 sc[RT][2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
#pragma unroll
            for (int rb = 0; rb < RT; rb++) sc[rb][j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const x8 k = codes8<T>(kc[j][c][2 * e], kc[j][c][2 * e + 1]);
#pragma unroll
                    for (int rb = 0; rb < RT; rb++)
                        if (rb == 0 || two) sc[rb][j] = Half<T>::mfma16(k, q[rb][2 * c + e], sc[rb][j]);
                }
        }
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int i = 0; i < 4; i++) ks[j][i] = __builtin_fmaf(ks[j][i], a.scale, vs[j][i] - vs[j][i]);      // a value's NaN with the key's scale
        x8 p8[RT], rest8[RT];                                        // weights, and what their rounding leaves
#pragma unroll
        for (int rb = 0; rb < RT; rb++) {
            if (rb > 0 && !two) continue;
            float t[2][4], counted[2][4];
            auto of_row = [](float x) {                              // the largest of a row's four lanes
                x = fmaxf(x, __shfl_xor(x, 16));
                return fmaxf(x, __shfl_xor(x, 32));
            };
            auto wanted = [&] {                                      // the reference that would suit these scores
                float top = NEG;
#pragma unroll
                for (int e = 0; e < 8; e++) top = fmaxf(top, t[e / 4][e % 4]);
                return of_row(top) - kTop;
            };
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int key = key0 + 16 * j + 4 * g + i;
                    const bool seen = there[j] && uint32_t(pos[rb] - key) < span;
                    counted[j][i] = fmaxf(vs[j][i], least[rb]);
                    t[j][i] = seen ? __builtin_fmaf(sc[rb][j][i], ks[j][i], __builtin_amdgcn_logf(counted[j][i])) : NEG;
                }
            float want = wanted();
            const bool up = want > m[rb] + kSlack || (m[rb] == NEG && want > NEG);
            if (__any(up)) {                                          // rows that do not need it stay where they are
                float large = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; e++) large = fmaxf(large, t[e / 4][e % 4] > NEG ? counted[e / 4][e % 4] : 0.0f);
                large = of_row(large) * kScaleRange;
                large = up ? fmaxf(large, least[rb]) : least[rb];
                if (__any(large > least[rb])) {
#pragma unroll
                    for (int j = 0; j < 2; j++)
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const float more = fmaxf(counted[j][i], large);
                            if (t[j][i] > NEG) t[j][i] += __builtin_amdgcn_logf(more) - __builtin_amdgcn_logf(counted[j][i]);
                            counted[j][i] = more;
                        }
                    least[rb] = large;
                    want = wanted();
                }
                const float f = up ? __builtin_amdgcn_exp2f(m[rb] - want) : 1.0f;
                l[rb] = up ? scaled_sum(l[rb], m[rb] - want) : l[rb];
                m[rb] = up ? want : m[rb];
#pragma unroll
                for (int c = 0; c < C; c++)
#pragma unroll
                    for (int k = 0; k < 4; k++) o[rb][c][k] *= f;
            }
            const float ref = m[rb] == NEG ? 0.0f : m[rb];
            T w[8], rest[8];
            float sum = 0.0f;                                        // of eight: below 2^117
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float p = __builtin_amdgcn_exp2f(t[j][i] - ref);
                    sum = __builtin_fmaf(p, __builtin_amdgcn_rcpf(counted[j][i]), sum);
                    w[4 * j + i] = T(p);
                    rest[4 * j + i] = T(p - float(w[4 * j + i]));
                }
            l[rb] = __builtin_fmaf(sum, 1.0f / kSumUnit, l[rb]);
            __builtin_memcpy(&p8[rb], w, 16);
            __builtin_memcpy(&rest8[rb], rest, 16);
        }
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const x8 v = codes8<T>(vc[0][c][k], vc[1][c][k]);
#pragma unroll
                for (int rb = 0; rb < RT; rb++)
                    if (rb == 0 || two) {
                        o[rb][c][k] = Half<T>::mfma16(v, p8[rb], o[rb][c][k]);
                        o[rb][c][k] = Half<T>::mfma16(v, rest8[rb], o[rb][c][k]);
                    }
            }
    }

    // the four waves' shares, then the result, 64 columns at a time
#pragma unroll
    for (int rb = 0; rb < RT; rb++) {
        l[rb] += __shfl_xor(l[rb], 16);
        l[rb] += __shfl_xor(l[rb], 32);
        if (g == 0) {
            S_m[wv][16 * rb + col] = m[rb];
            S_l[wv][16 * rb + col] = l[rb];
        }
    }
    __syncthreads();
    float f[RT];
#pragma unroll
    for (int rb = 0; rb < RT; rb++) {
        const int r = 16 * rb + col;
        const float to = fmaxf(fmaxf(S_m[0][r], S_m[1][r]), fmaxf(S_m[2][r], S_m[3][r]));
        f[rb] = m[rb] == NEG ? 0.0f : __builtin_amdgcn_exp2f(m[rb] - to);
    }
#pragma unroll
    for (int c = 0; c < C; c++) {
        if (c) __syncthreads();
#pragma unroll
        for (int rb = 0; rb < RT; rb++)
#pragma unroll
            for (int i = 0; i < 4; i++) {                            // register i of o[..][k]: column 16 g + 4 i + k
                const f32x4 v = {o[rb][c][0][i] * f[rb], o[rb][c][1][i] * f[rb], o[rb][c][2][i] * f[rb], o[rb][c][3][i] * f[rb]};
                *reinterpret_cast<f32x4 *>(&S_o[wv][16 * rb + col][16 * g + 4 * i]) = v;
            }
        __syncthreads();
#pragma unroll
        for (int x = threadIdx.x; x < R * 16; x += 256) {
            const int r = x / 16, d = 4 * (x % 16);
            if (r >= rows) continue;
            f32x4 v = {0, 0, 0, 0};
            float to = NEG, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; w++) {
                v += *reinterpret_cast<const f32x4 *>(&S_o[w][r][d]);
                to = fmaxf(to, S_m[w][r]);
            }
#pragma unroll
            for (int w = 0; w < 4; w++) sum += S_m[w][r] == NEG ? S_l[w][r] : scaled_sum(S_l[w][r], S_m[w][r] - to);
            if (alone) {
                const int i = r / a.G;
                O *out = static_cast<O *>(a.out) + int64_t(s.start + i) * a.odt + int64_t(h * a.G + r - i * a.G) * a.odh;
                store4(out + 64 * c + d, over_sum(v, sum));
            } else {
                const int64_t slot = ((int64_t(b) * a.Hkv + h) * a.split + share) * R + r;
                *reinterpret_cast<f32x4 *>(a.part + slot * D + 64 * c + d) = v;
                if (c == 0 && d == 0) {
                    float *ml = a.part + int64_t(a.units) * a.Hkv * a.split * R * D + 2 * slot;
                    ml[0] = to;
                    ml[1] = sum;
                }
            }
        }
    }
}

// --- tile kernel ------------------------------------------------------------
//
// A workgroup is 256 rows (128 for D = 64 and 256) of one sequence and head,
// 32 a wave, and walks the keys 64 at a time.  Codes come through registers,
// are converted to 16 bits once per workgroup (two fragments' worth a wave)
// and lie in LDS in the order of the matrix instruction's fragments: every
// read is 1 KiB in a row.
//
// What bounds it (8192 x 8192 causal, 28 on 4 heads of 128, bf16: 512 to 547 us
// from card to card, 880 to 939 TFLOP/s; a large library product reaches 1233):
// VALU and matrix core together.  A step of a wave is 32 products of 32 cycles
// and 221 other vector instructions, 32 of them exponentials and 48 conversions;
// a product costs the VALU two to three instructions' time.  In a run of 600 us
// at 1.9 GHz, where the power limit holds the clock, the matrix cores are busy
// 42 % of the time.
// Steps that led here, us: scores, softmax and output one after the other
// 677; next scores behind this step's exponentials, scales behind the
// output's products, values' scales in the exponent 543; three buffers,
// fragments read across the barrier 536; no wave with more to do than the
// others before the barrier 518; younger waves first in the first half 514.
// Tried and not kept: 128 rows and two workgroups a CU (594: codes are
// converted twice as often), loads two steps ahead (546), scales loaded by
// all waves (546).
// The sequence and its tile of BM rows that tile number `tile` of the launch
// is; false past the last.  Only sequences of many rows have tiles.  `load`:
// keys for each of the `target` workgroups that the device runs at once, if
// all tiles' keys were spread over them evenly.  Sequences are taken 64 at a
// time, up to 256 of them those whose tiles see the most keys first, so that
// the last workgroups to start are short ones.
template <int BM>
__device__ __forceinline__ bool find_tile(const AttnArgs &a, int tile, int &b, int &in, int &of, float &load) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    bool found = false;
    float keys = 0.0f;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        int n = 0, most = -1, at = lane;
        float mean = 0.0f;
        if (b0 + lane < a.B) {
            const Seq s = sequence(a, b0 + lane);
            if (!has_few_rows(a, s.n)) n = int((int64_t(s.n) * a.G + BM - 1) / BM);
            mean = fmaxf(float(s.pos0) + 0.5f * float(s.n), 1.0f);
            most = s.len;
            if (a.window) {
                mean = fminf(mean, float(a.window) + 0.5f * BM);
                most = min(most, a.window);
            }
        }
        keys += float(n) * mean;
        const int here = min(a.B - b0, 64);
        if (here > 1 && a.B <= 256) {                     // (more have many workgroups each, and the sort its cost)
            int rank = 0;
            for (int j = 0; j < here; j++) {
                const int other = __builtin_amdgcn_readlane(most, j);
                rank += other > most || (other == most && j < lane);
            }
            n = __builtin_amdgcn_ds_permute(4 * rank, n);            // lanes past the last: most = -1, behind all
            at = __builtin_amdgcn_ds_permute(4 * rank, lane);
        }
        const int upto = scan_sum(n);
        const unsigned long long hit = __ballot(before + upto > tile);
        if (!found && hit) {
            const int i = __builtin_ctzll(hit);
            b = b0 + __builtin_amdgcn_readlane(at, i);
            of = __builtin_amdgcn_readlane(n, i);
            in = tile - before - (__builtin_amdgcn_readlane(upto, i) - of);
            found = true;
            if (a.split == 1) break;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    if (a.split > 1) {
#pragma unroll
        for (int o = 32; o; o >>= 1) keys += __shfl_xor(keys, o);
    }
    // the same in every lane: what follows from it is kept in scalar registers
    load = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(keys * float(a.Hkv) / float(a.target))));
    return found;
}

// Keys of each share of a tile: as many shares as come nearest to the load,
// all alike.
__device__ __forceinline__ int tile_chunk(const AttnArgs &a, const Range &r, float load) {
    const int keys = r.end - r.begin, shares = min(max(int(float(keys) / fmaxf(load, float(kAttnTileChunk)) + 0.5f), 1), a.split);
    return max(((keys + shares - 1) / shares + 63) & ~63, 64);
}

template <typename T, typename O, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_attn_tile(AttnArgs a) {
    typedef typename Half<T>::x8 x8;
    constexpr int THREADS = 64 * WAVES, BM = 32 * WAVES, TILE = int(kv_tile_bytes(D));
    constexpr int KS = D / 16, DT = D / 32;              // steps of the first product, column tiles of the second
    constexpr int LOADS = 8 * D / THREADS;               // 16-byte loads of a lane for 64 keys and 64 values
    constexpr float NEG = -__builtin_inff();
    static_assert(8 * D % (2 * THREADS) == 0, "whole loads of keys and of values");
    constexpr bool REST = sizeof(O) == 4;                 // fp32 outputs: a second product of what the weights' rounding leaves
    constexpr int RING = D == 256 ? 2 : 3;                // buffers of 64 keys, and of 64 values
    __shared__ __align__(16) uint8_t S_k[RING][128 * D], S_v[RING][128 * D];
    __shared__ __align__(16) float S_ks[4][64], S_lv[4][64], S_rv[4][64];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 31, hf = lane >> 5;
    const int h = blockIdx.x % a.Hkv, rest = blockIdx.x / a.Hkv, share = rest / a.units;
    int b, in, of;
    float share_load;
    if (!find_tile<BM>(a, rest % a.units, b, in, of, share_load)) return;
    b = __builtin_amdgcn_readfirstlane(b);
    in = of - 1 - __builtin_amdgcn_readfirstlane(in);    // the rows with the most keys first
    const Seq s = sequence(a, b);
    const int rows = s.n * a.G, row0 = in * BM;
    const Range all(a, s, row0 / a.G, (min(row0 + BM, rows) - 1) / a.G);
    const int chunk = tile_chunk(a, all, share_load);
    const int begin = all.begin + min(int64_t(share) * chunk, int64_t(all.end - all.begin)), end = min(int64_t(all.end), int64_t(begin) + chunk);
    const bool alone = all.end - all.begin <= chunk;
    if (begin >= end && share > 0) return;
    const int steps = (end - begin + 63) / 64;

    // this lane's row
    const int r = row0 + 32 * wv + col, tok = r / a.G;
    const bool there = r < rows;
    const int pos = there ? s.pos0 + tok : -1;
    const uint32_t span = a.window ? uint32_t(a.window) : 0x80000000u;      // keys that a row sees, up to its position
    // A lane past the last row has zeros: any row that it could read instead is one that, with the output over the
    // queries, another workgroup may be writing.
    x8 q[KS];
    if (there) {
        const T *qr = static_cast<const T *>(a.q) + int64_t(s.start + tok) * a.qdt + int64_t(h * a.G + r - tok * a.G) * a.qdh;
#pragma unroll
        for (int k = 0; k < KS; k++) q[k] = load_x8(qr + 16 * k + 8 * hf);
    } else {
#pragma unroll
        for (int k = 0; k < KS; k++) q[k] = x8{};
    }
    // the wave's rows see all of keys (lo_all, hi_all], and something in steps [from, to]
    const int wr0 = row0 + 32 * wv, wr1 = min(wr0 + 32, rows) - 1;
    const int hi_all = s.pos0 + wr0 / a.G, hi_any = s.pos0 + wr1 / a.G;
    const int lo_all = a.window ? hi_any - a.window : -1, lo_any = a.window ? hi_all - a.window : -1;
    const bool active = wr0 < rows && hi_any >= begin && lo_any < end;
    const int from = active ? max(lo_any + 1 - begin, 0) / 64 : steps, to = active ? min((hi_any - begin) / 64, steps - 1) : -1;

    float m = there ? NEG : -NEG, l = 0.0f;               // infinity: a lane without a row never asks for another reference
    f32x16 o[DT];
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) o[d][i] = 0.0f;

    // Load i of a wave: 64 chunks of 16 bytes of the keys (of step `step`) or,
    // behind those, of the values (of the step before).
    struct Stage {
        u32x4 st[LOADS];
        float scale;                                      // wave 0: of a key; wave 1: of a value
    };
    float least = kLeastScale;
    int tk = -1, tv = -1;                                 // cache tiles of 16 steps: lane 4 i + j holds 16-key tile j of step i
    int valid = 0;                                        // four bits a step, of four steps: which of its tiles are there
    auto load = [&](int step, Stage &g) __attribute__((always_inline)) {
        tv = tk;
        if ((step & 15) == 0) {
            const int k16 = begin / 16 + 4 * step + lane;
            tk = 16 * k16 < end ? cache_tile(a, b, h, k16) : -1;
        }
        const unsigned long long ok = __ballot(tk >= 0);
        valid = (valid & ~(15 << 4 * (step & 3))) | (int(ok >> (4 * (step & 15))) & 15) << 4 * (step & 3);
#pragma unroll
        for (int i = 0; i < LOADS; i++) {
            const int c = i * THREADS + wv * 64;
            const bool is_v = i >= LOADS / 2;
            const int part = c / D & 3, at = c % D;
            const int t = max(is_v ? __builtin_amdgcn_readlane(tv, 4 * ((step - 1) & 15) + part)
                                   : __builtin_amdgcn_readlane(tk, 4 * (step & 15) + part), 0);
            g.st[i] = *reinterpret_cast<const u32x4 *>(a.cache + int64_t(t) * TILE + (is_v ? 16 * D : 0) + (at + lane) * 16);
        }
        if (wv < 2) {                                     // wave 0: key scales; wave 1: value scales
            const int j = 4 * (step & 15), t16 = lane >> 4;
            const int t0 = __builtin_amdgcn_readlane(tk, j), t1 = __builtin_amdgcn_readlane(tk, j + 1);
            const int t2 = __builtin_amdgcn_readlane(tk, j + 2), t3 = __builtin_amdgcn_readlane(tk, j + 3);
            const int t = t16 == 0 ? t0 : t16 == 1 ? t1 : t16 == 2 ? t2 : t3;
            g.scale = t >= 0 && begin + 64 * step + lane < end
                           ? reinterpret_cast<const float *>(a.cache + int64_t(t) * TILE + 32 * D)[16 * wv + (lane & 15)]
                           : 0.0f;
        }
    };
    // The lane's places within what a wave stores, kept in registers (the
    // compiler would work them out anew in every step).
    //   K: lane = (chunk of 16 d, token); fragment (32 keys, 16 d): [half of d][key][8 d]
    //   V: lane = (four tokens g, four d); fragment (16 keys, 32 d): [g & 1][d][g >> 1][4 tokens]
    int in_k = (lane >> 4) * 1024 + (lane & 15) * 16, in_v = (lane >> 4 & 1) * 512 + (lane & 15) * 16 + (lane >> 5) * 8;
    asm volatile("" : "+v"(in_k), "+v"(in_v));
    // Unit u of the conversion to 16 bits: dword u % 4 of load u / 4.
    uint32_t cw[2][2];
    auto store = [&](const Stage &g, int kslot, int vslot, int u) __attribute__((always_inline)) {
        const int i = u / 4, k = u % 4, c = i * THREADS + wv * 64, part = c / D & 3, at = c % D;
        Half<T>::codes(g.st[i][k], cw[k & 1]);
        if (i < LOADS / 2) {
            uint8_t *p = S_k[kslot] + ((part >> 1) * KS + at / 16) * 1024 + 256 * (part & 1) + in_k;
            if (k & 1) *reinterpret_cast<u32x4 *>(p + (k >> 1) * 512) = u32x4{cw[0][0], cw[0][1], cw[1][0], cw[1][1]};
        } else {
            uint8_t *p = S_v[vslot] + (part * DT + at / 32) * 1024 + in_v;
            *reinterpret_cast<uint2 *>(p + (k >> 1) * 1024 + (k & 1) * 256) = make_uint2(cw[k & 1][0], cw[k & 1][1]);
        }
    };
    auto store_scales = [&](const Stage &g, int step) __attribute__((always_inline)) {
        if (wv == 0) S_ks[step & 3][lane] = g.scale * a.scale;
        if (wv == 1) {
            if (__any(g.scale > kLargeScale)) least = raised_least(least, g.scale);
            const float sc = fmaxf(g.scale, least);
            S_lv[step & 3][lane] = g.scale == g.scale ? __builtin_amdgcn_logf(sc) : g.scale;      // NaN reaches its rows by this, if it is seen
            S_rv[step & 3][lane] = __builtin_amdgcn_rcpf(sc) * (1.0f / kSumUnit);
        }
    };
    auto store_all = [&](const Stage &g, int step, int kslot, int vslot) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 4 * LOADS; u++) store(g, kslot, vslot, u);
        store_scales(g, step);
    };
    Stage st;
    // Element e of a lane's 32 scores of a step: key 8 (e / 4) + 4 hf + e % 4.
    auto four = [&](const float (*S)[64], int step, int chunk) __attribute__((always_inline)) {
        return *reinterpret_cast<const f32x4 *>(S[step & 3] + 4 * hf + 8 * chunk);
    };
    // The scores of one step, alone: where a wave's rows begin to see keys.
    auto first_scores = [&](int step, int kslot, f32x16 (&sc)[2], float &top) __attribute__((always_inline)) {
        const uint8_t *K = S_k[kslot] + lane * 16;
#pragma unroll
        for (int j = 0; j < 2; j++) {
#pragma unroll
            for (int i = 0; i < 16; i++) sc[j][i] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; k++) sc[j] = Half<T>::mfma32(*reinterpret_cast<const x8 *>(K + (j * KS + k) * 1024), q[k], sc[j]);
        }
        top = NEG;
#pragma unroll
        for (int ch = 0; ch < 8; ch++) {
            const f32x4 k4 = four(S_ks, step, ch), v4 = four(S_lv, step, ch);
#pragma unroll
            for (int y = 0; y < 4; y++) {
                sc[ch / 4][4 * (ch % 4) + y] = __builtin_fmaf(sc[ch / 4][4 * (ch % 4) + y], k4[y], v4[y]);
                top = fmaxf(top, sc[ch / 4][4 * (ch % 4) + y]);
            }
        }
        top = max_of_halves(top);
    };
    // One step.  `sc` holds its scaled scores and `top` their largest, and
    // takes the next step's.  Two runs of D / 8 products each, with the VALU
    // work of a step spread between them:
    //   the next step's scores     this step's exponentials
    //   this step's output         the next scores' scales and maximum, and
    //                              the conversion of the step after that
    // The order is written out and pinned, with fragments four products ahead
    // (with three buffers, across the barrier too).
    constexpr int AHEAD = 4;
    float top = NEG;
    x8 fr[AHEAD];
    f32x4 r4[2];                                          // reciprocals of the values' scales (and the sum's unit), two fours ahead
    int ring = 0;                                         // of this step's keys and values; the next step's is behind it
    auto next = [](int x) { return x + 1 == RING ? 0 : x + 1; };
    auto prefetch_r = [&](int step) __attribute__((always_inline)) {
        r4[0] = four(S_rv, step, 0);
        r4[1] = four(S_rv, step, 1);
    };
    auto prefetch = [&](int kslot) __attribute__((always_inline)) {
#pragma unroll
        for (int g = 0; g < AHEAD; g++) fr[g] = *reinterpret_cast<const x8 *>(S_k[kslot] + lane * 16 + g * 1024);
    };
    auto body = [&](int step, f32x16 (&sc)[2]) __attribute__((always_inline)) {
        constexpr int N = D / 8, E = 32 / N;
        const int key0 = begin + 64 * step, kslot = next(ring), before = RING == 2 ? kslot : next(kslot);
        __syncthreads();
        // of a SIMD's two waves the older runs first and then waits, ~1000 of a step's 4400 cycles: the younger first for half
        if (WAVES == 8 && wv >= 4) __builtin_amdgcn_s_setprio(1);
        {
            const uint8_t *K = S_k[kslot] + lane * 16, *V = S_v[ring] + lane * 16;
            if (RING == 2) prefetch(kslot);
            const int there4 = valid >> 4 * (step & 3) & 15;
            if (!(there4 == 15 && key0 + 63 <= hi_all && key0 > lo_all)) {
                top = NEG;
#pragma unroll
                for (int e = 0; e < 32; e++) {
                    const int key = key0 + 8 * (e / 4) + 4 * hf + e % 4;
                    if (!((there4 >> (e / 8) & 1) && uint32_t(pos - key) < span)) sc[e / 16][e % 16] = NEG;
                    top = fmaxf(top, sc[e / 16][e % 16]);
                }
                top = max_of_halves(top);
            }
            const float want = top - kTop;
            const bool up = want > m + kSlack || (m == NEG && want > NEG);
            if (__any(up)) {                              // rows that do not need it stay where they are
                const float f = up ? __builtin_amdgcn_exp2f(m - want) : 1.0f;
                l = up ? scaled_sum(l, m - want) : l;
                m = up ? want : m;
#pragma unroll
                for (int d = 0; d < DT; d++)
#pragma unroll
                    for (int i = 0; i < 16; i++) o[d][i] *= f;
            }
            const float ref = m == NEG ? 0.0f : m;
            union { T w[32]; x8 p[4]; } u, rest;
            float pair = 0.0f;
            f32x16 nx[2];
            f32x4 k4[2], v4[2];
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int i = 0; i < 16; i++) nx[j][i] = 0.0f;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int g = 0; g < N; g++) {
                nx[g / KS] = Half<T>::mfma32(fr[g % AHEAD], q[g % KS], nx[g / KS]);
                fr[g % AHEAD] = *reinterpret_cast<const x8 *>(g + AHEAD < N ? K + (g + AHEAD) * 1024 : V + (g + AHEAD - N) * 1024);
#pragma unroll
                for (int e = g * E; e < g * E + E; e++) {
                    const float p = __builtin_amdgcn_exp2f(sc[e / 16][e % 16] - ref);
                    l = __builtin_fmaf(p, r4[e / 4 & 1][e % 4], l);
                    if (e % 4 == 3 && e < 24) r4[e / 4 & 1] = four(S_rv, step, e / 4 + 2);
                    if (e & 1) {
                        u.w[e - 1] = T(pair);
                        u.w[e] = T(p);
                        if constexpr (REST) {
                            rest.w[e - 1] = T(pair - float(u.w[e - 1]));
                            rest.w[e] = T(p - float(u.w[e]));
                        }
                    }
                    pair = p;
                }
                if (g == N - 3) {
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        k4[c] = four(S_ks, step + 1, c);
                        v4[c] = four(S_lv, step + 1, c);
                    }
                }
                asm volatile("" : "+v"(l));               // summed here: put off, the sums would keep every p in a register
                __builtin_amdgcn_sched_barrier(0);
            }
            top = NEG;
#pragma unroll
            for (int g = 0; g < N; g++) {
                if (WAVES == 8 && g == 0) __builtin_amdgcn_s_setprio(0);
                o[g % DT] = Half<T>::mfma32(fr[g % AHEAD], u.p[g / DT], o[g % DT]);
                if constexpr (REST) o[g % DT] = Half<T>::mfma32(fr[g % AHEAD], rest.p[g / DT], o[g % DT]);
                if (g + AHEAD < N)
                    fr[g % AHEAD] = *reinterpret_cast<const x8 *>(V + (g + AHEAD) * 1024);
                else if (RING > 2)
                    fr[g % AHEAD] = *reinterpret_cast<const x8 *>(S_k[before] + lane * 16 + (g + AHEAD - N) * 1024);
#pragma unroll
                for (int e = g * E; e < g * E + E; e++) {
                    sc[e / 16][e % 16] = __builtin_fmaf(nx[e / 16][e % 16], k4[e / 4 & 1][e % 4], v4[e / 4 & 1][e % 4]);
                    top = fmaxf(top, sc[e / 16][e % 16]);
                    if (e % 4 == 3 && e < 24) {
                        k4[e / 4 & 1] = four(S_ks, step + 1, e / 4 + 2);
                        v4[e / 4 & 1] = four(S_lv, step + 1, e / 4 + 2);
                    }
                }
                if (g == N - 1) prefetch_r(step + 1);
                asm volatile("" : "+v"(top));
                if ((g + 1) * 4 * LOADS % N == 0) store(st, ring, before, (g + 1) * 4 * LOADS / N - 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            top = max_of_halves(top);
            store_scales(st, step + RING);
        }
        load(step + RING + 1, st);
        ring = kslot;
    };
    // A step whose keys the wave's rows do not see.
    auto bring = [&](int step) __attribute__((always_inline)) {
        const int kslot = next(ring);
        __syncthreads();
        store_all(st, step + RING, ring, RING == 2 ? kslot : next(kslot));
        load(step + RING + 1, st);
        ring = kslot;
    };
    // Buffers: load(s) and store(s) bring the keys of step s and the values of
    // step s - 1 (past the last step: of tile 0, not used).  Step s reads the
    // keys of s + 1 and the values of s, and stores the keys of s + RING and
    // the values of s + RING - 1 over those of s and s - 1, which all waves
    // have read before the barrier that begins it.
    if (steps > 0) {
        f32x16 sc[2];
        Stage fill[RING];
#pragma unroll
        for (int i = 0; i < RING; i++) load(i, fill[i]);
#pragma unroll
        for (int i = 0; i < RING; i++) store_all(fill[i], i, i, (i + RING - 1) % RING);
        load(RING, st);
        __syncthreads();
        int step = 0;
        for (; step < min(from, steps); step++) bring(step);
        if (from <= to) {
            first_scores(from, ring, sc, top);
            if (RING > 2) prefetch(next(ring));
            prefetch_r(from);
            for (; step <= to; step++) body(step, sc);
        }
        for (; step < steps; step++) bring(step);
    }
    l += __shfl_xor(l, 32);
    if (!there) return;
    // register i of o[2 v + p]: column 64 v + 32 (i / 4 % 2) + 16 hf + 4 (i % 4) + 2 p + i / 8
    const int64_t slot = ((int64_t(rest % a.units) * a.Hkv + h) * a.split + share) * BM + 32 * wv + col;
    O *out = static_cast<O *>(a.out) + int64_t(s.start + tok) * a.odt + int64_t(h * a.G + r - tok * a.G) * a.odh;
#pragma unroll
    for (int v = 0; v < D / 64; v++)
#pragma unroll
        for (int x = 0; x < 2; x++)
#pragma unroll
            for (int y = 0; y < 4; y++) {
                const int i = 4 * x + y, d = 64 * v + 32 * x + 16 * hf + 4 * y;
                const f32x4 w = {o[2 * v][i], o[2 * v][i + 8], o[2 * v + 1][i], o[2 * v + 1][i + 8]};
                if (alone)
                    store4(out + d, over_sum(w, l));
                else
                    *reinterpret_cast<f32x4 *>(a.part + slot * D + d) = w;
            }
    if (!alone && hf == 0) {
        float *ml = a.part + int64_t(a.units) * a.Hkv * a.split * BM * D + 2 * slot;
        ml[0] = m;
        ml[1] = l;
    }
}

// ---------------------------------------------------------------------------
// Joining shares.  Rows whose keys were not split have been written.
// ---------------------------------------------------------------------------
struct Joined {
    f32x4 v;
    float sum;
    // One share, for the largest reference `to` of all, finite: one that saw
    // no finite maximum adds nothing, unless it holds a NaN.
    __device__ __forceinline__ void add(float m, float l, f32x4 o, float to) {
        const float h = __builtin_amdgcn_exp2f(0.5f * (m - to));
        sum += l * h * h;                                 // in two halves, as in scaled_sum
        v += o * (h * h);
    }
    template <typename O>
    __device__ __forceinline__ void write(const AttnArgs &a, const Seq &s, int h, int r, int d) const {
        const int i = r / a.G;
        O *out = static_cast<O *>(a.out) + int64_t(s.start + i) * a.odt + int64_t(h * a.G + r - i * a.G) * a.odh;
        store4(out + d, over_sum(v, sum));
    }
};

// Rows kernel: up to hundreds of shares of a few rows.  A workgroup a row,
// D / 4 lanes a share.  The rows kernel left the number of shares, so that
// nothing here waits for anything but its own loads: the first shares' are
// under way before their number is known (all lie within the workspace).
template <typename O, int D, int R>
__global__ __launch_bounds__(256) void k_attn_join_rows(AttnArgs a, int most_rows) {
    constexpr int LANES = D / 4, GROUPS = 256 / LANES, EARLY = 4;
    __shared__ float S_v[GROUPS][D], S_l[GROUPS];
    const int r = blockIdx.x % most_rows, unit = blockIdx.x / most_rows, h = unit % a.Hkv, b = unit / a.Hkv;
    const int group = threadIdx.x / LANES, d = 4 * (threadIdx.x % LANES);
    const int64_t slot0 = int64_t(unit) * a.split * R + r, slots = int64_t(a.units) * a.Hkv * a.split * R;
    const float *ml = a.part + slots * D;
    f32x4 early[EARLY];
    float early_m[EARLY], early_l[EARLY];
#pragma unroll
    for (int j = 0; j < EARLY; j++) {
        const int64_t slot = slot0 + int64_t(min(group + j * GROUPS, a.split - 1)) * R;
        early[j] = *reinterpret_cast<const f32x4 *>(a.part + slot * D + d);
        early_m[j] = ml[2 * slot];
        early_l[j] = ml[2 * slot + 1];
    }
    const Seq s = sequence(a, b);
    if (s.n == 0 || !has_few_rows(a, s.n) || r >= s.n * a.G) return;          // no share was written
    const int shares = reinterpret_cast<const int *>(ml + 2 * slots)[unit];
    if (shares <= 1) return;
    float to = -__FLT_MAX__;
    for (int k = threadIdx.x & 63; k < shares; k += 64) to = fmaxf(to, ml[2 * (slot0 + int64_t(k) * R)]);
#pragma unroll
    for (int o = 32; o; o >>= 1) to = fmaxf(to, __shfl_xor(to, o));
    Joined j{{0, 0, 0, 0}, 0.0f};
#pragma unroll
    for (int e = 0; e < EARLY; e++)
        if (group + e * GROUPS < shares) j.add(early_m[e], early_l[e], early[e], to);
#pragma unroll 4
    for (int k = group + EARLY * GROUPS; k < shares; k += GROUPS) {
        const int64_t slot = slot0 + int64_t(k) * R;
        j.add(ml[2 * slot], ml[2 * slot + 1], *reinterpret_cast<const f32x4 *>(a.part + slot * D + d), to);
    }
    *reinterpret_cast<f32x4 *>(&S_v[group][d]) = j.v;
    if (d == 0) S_l[group] = j.sum;
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < GROUPS; g++) {
        j.v += *reinterpret_cast<const f32x4 *>(&S_v[g][d]);
        j.sum += S_l[g];
    }
    j.write<O>(a, s, h, r, d);
}

// Tile kernel: a few shares of many rows.  D / 4 lanes a row.
template <typename O, int D, int BM>
__global__ __launch_bounds__(256) void k_attn_join_tiles(AttnArgs a) {
    constexpr int LANES = D / 4, ROWS = 256 / LANES, BLOCKS = BM / ROWS;
    const int block = blockIdx.x % BLOCKS, unit = blockIdx.x / BLOCKS, h = unit % a.Hkv;
    int b, in, of;
    float load;
    if (!find_tile<BM>(a, unit / a.Hkv, b, in, of, load)) return;
    b = __builtin_amdgcn_readfirstlane(b);
    in = of - 1 - __builtin_amdgcn_readfirstlane(in);
    const Seq s = sequence(a, b);
    const int rows = s.n * a.G, row0 = in * BM, slot_r = block * ROWS + threadIdx.x / LANES, r = row0 + slot_r, d = 4 * (threadIdx.x % LANES);
    const Range all(a, s, row0 / a.G, (min(row0 + BM, rows) - 1) / a.G);
    const int chunk = tile_chunk(a, all, load), shares = (all.end - all.begin + chunk - 1) / chunk;
    if (shares <= 1 || r >= rows) return;
    const int64_t slot0 = int64_t(unit) * a.split * BM + slot_r;
    const float *ml = a.part + int64_t(a.units) * a.Hkv * a.split * BM * D;
    float to = -__FLT_MAX__;
#pragma unroll 8
    for (int k = 0; k < shares; k++) to = fmaxf(to, ml[2 * (slot0 + int64_t(k) * BM)]);
    Joined j{{0, 0, 0, 0}, 0.0f};
#pragma unroll 8
    for (int k = 0; k < shares; k++) {
        const int64_t slot = slot0 + int64_t(k) * BM;
        j.add(ml[2 * slot], ml[2 * slot + 1], *reinterpret_cast<const f32x4 *>(a.part + slot * D + d), to);
    }
    j.write<O>(a, s, h, r, d);
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
template <typename T, typename O, int D>
static hipError_t launch_dim(const AttnPlan &p, AttnArgs a, void *workspace, hipStream_t stream) {
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (p.few_tiles) {
        a.split = p.few_split;
        a.target = p.few_target;
        a.units = a.B;
        a.part = reinterpret_cast<float *>(ws);
        const dim3 grid{unsigned(p.few_grid)};
        const int most_rows = int(std::min(int64_t(a.max_q) * a.G, int64_t(kAttnFewRows)));
        const dim3 rows{unsigned(a.B) * unsigned(a.Hkv) * unsigned(most_rows)};
        if (p.few_tiles == 1) {
            k_attn_rows<T, O, D, 1><<<grid, 256, 0, stream>>>(a);
            if (a.split > 1) k_attn_join_rows<O, D, 16><<<rows, 256, 0, stream>>>(a, most_rows);
        } else {
            k_attn_rows<T, O, D, 2><<<grid, 256, 0, stream>>>(a);
            if (a.split > 1) k_attn_join_rows<O, D, 32><<<rows, 256, 0, stream>>>(a, most_rows);
        }
    }
    if (p.tile_rows) {
        constexpr int WAVES = D == 128 ? 8 : 4, BM = 32 * WAVES;
        a.split = p.tile_split;
        a.target = p.tile_target;
        a.units = int(p.tiles);
        a.part = reinterpret_cast<float *>(ws + p.few_bytes);
        k_attn_tile<T, O, D, WAVES><<<dim3(unsigned(p.tile_grid)), 64 * WAVES, 0, stream>>>(a);
        if (a.split > 1)
            k_attn_join_tiles<O, D, BM><<<dim3(unsigned(p.tiles) * unsigned(a.Hkv) * (BM * D / 1024)), 256, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <typename T, typename O>
static hipError_t launch_out(const AttnPlan &p, const AttnArgs &a, int D, void *workspace, hipStream_t stream) {
    if (D == 64) return launch_dim<T, O, 64>(p, a, workspace, stream);
    if (D == 128) return launch_dim<T, O, 128>(p, a, workspace, stream);
    return launch_dim<T, O, 256>(p, a, workspace, stream);
}

hipError_t launch_attention(const AttnPlan &p, int type, const void *q, int64_t qdt, int64_t qdh, const void *cache,
                            int64_t n_pages, int page, const int32_t *table, int64_t max_pages, const int32_t *lens,
                            const int32_t *offsets, int64_t B, int64_t T, int64_t max_q, int Hq, int Hkv, int D, float scale,
                            int window, int out_type, void *out, int64_t odt, int64_t odh, void *workspace,
                            hipStream_t stream) {
    AttnArgs a{};
    a.q = q; a.qdt = qdt; a.qdh = qdh;
    a.cache = static_cast<const uint8_t *>(cache);
    a.table = table; a.lens = lens; a.offsets = offsets;
    a.out = out; a.odt = odt; a.odh = odh;
    a.n_pages = n_pages; a.max_pages = max_pages;
    a.page_shift = __builtin_ctz(unsigned(page));
    a.Hkv = Hkv; a.G = Hq / Hkv;
    a.T = int(T); a.B = int(B); a.max_q = int(max_q < T ? max_q : T); a.window = window;
    a.scale = float(double(scale) * 1.4426950408889634074);
    a.few_rows = p.few_tiles ? kAttnFewRows : 0;
    if (type == TYPE_BF16)
        return out_type == TYPE_F32 ? launch_out<__bf16, float>(p, a, D, workspace, stream)
                                    : launch_out<__bf16, __bf16>(p, a, D, workspace, stream);
    return out_type == TYPE_F32 ? launch_out<_Float16, float>(p, a, D, workspace, stream)
                                : launch_out<_Float16, _Float16>(p, a, D, workspace, stream);
}

}  // namespace mmq
