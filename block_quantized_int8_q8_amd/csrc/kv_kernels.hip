// kv_kernels.hip -- gfx950 kernels of the rotary positions and of the int8
// paged cache.
//
//   k_rope       pairs of a head's values turned by position times frequency
//   k_kv_write   keys (turned first, if asked) and values -> int8 codes and a
//                scale per token and head, written to their slots
//   k_kv_read    the values that slots hold
//
// A row (one head of one token) lies across D / 8 lanes of a wave, eight
// values a lane.  All three are bound by memory where tokens are many (a copy
// moves 5.12 TB/s here) and by the chain of dependent loads where they are few:
//   rope of 8192 x 28 x 128 bf16   20.6 us for 117 MB (a copy of the same 17.7)
//   write of 8192 x 4 x 128 bf16   11.8 us turned, 8.6 not (floor 4.9); of
//                                  32768 tokens 32.6 and 24.1 (floor 19.6): the
//                                  difference is the 64-bit angles and products
//   read of 32768 x 4 x 128 bf16   19.4 us, its floor
// back to back on the same tensors.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_plan.hpp"
#include "i8_codes.hpp"

namespace mmq {

struct RopeArgs {
    const int32_t *positions;
    const double *freqs;      // radians per position of each pair
    double mscale;
    int rot;                  // values turned of each head; 0: none
    int inverse;
};

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    T t[8];
#pragma unroll
    for (int i = 0; i < 8; i++) t[i] = T(v[i]);
    __builtin_memcpy(p, t, sizeof(t));
}

// Sine and cosine of pi * y in 64 bits.  y loses its whole half-turns exactly;
// what is left is within pi/4, where the Taylor series end at x^15 and x^16
// (the next terms are below 2^-54 and 2^-58).
__device__ __forceinline__ void sincos_half_turns(double y, double &s, double &c) {
    const double n = __builtin_rint(2.0 * y), x = __builtin_fma(-0.5, n, y) * 3.14159265358979323846, z = x * x;
    double a = -1.0 / 1307674368000.0, b = 1.0 / 20922789888000.0;
    a = __builtin_fma(a, z, 1.0 / 6227020800.0);
    b = __builtin_fma(b, z, -1.0 / 87178291200.0);
    a = __builtin_fma(a, z, -1.0 / 39916800.0);
    b = __builtin_fma(b, z, 1.0 / 479001600.0);
    a = __builtin_fma(a, z, 1.0 / 362880.0);
    b = __builtin_fma(b, z, -1.0 / 3628800.0);
    a = __builtin_fma(a, z, -1.0 / 5040.0);
    b = __builtin_fma(b, z, 1.0 / 40320.0);
    a = __builtin_fma(a, z, 1.0 / 120.0);
    b = __builtin_fma(b, z, -1.0 / 720.0);
    a = __builtin_fma(a, z, -1.0 / 6.0);
    b = __builtin_fma(b, z, 1.0 / 24.0);
    b = __builtin_fma(b, z, -0.5);
    a = __builtin_fma(a * z, x, x);
    b = __builtin_fma(b, z, 1.0);
    const int q = int(int64_t(n)) & 3;                   // quarter turns; |n| < 2^53
    s = q & 1 ? b : a;
    c = q & 1 ? a : b;
    if (q & 2) s = -s;
    if ((q + 1) & 2) c = -c;
}

// Cosine and sine (times mscale) of every pair of the workgroup's tokens.
// position * frequency reaches a million radians, where fp32 has no digits of
// the angle left: 64 bits, in half turns, so that the reduction is exact.
// One angle serves all heads of its token.
// A thread keeps its pair and takes several tokens, all loads before any use.
template <int TOK>
__device__ __forceinline__ void angles(const RopeArgs &r, int64_t t0, int64_t T, double2 *tab) {
    const int pairs = r.rot / 2;
    const int wide = pairs <= 32 ? 32 : pairs <= 64 ? 64 : pairs <= 128 ? 128 : 256;
    const int p = threadIdx.x & (wide - 1), k0 = threadIdx.x / wide, step = 256 / wide;
    if (p >= pairs) return;
    const double f = r.freqs[p] * 0.318309886183790671538;
    constexpr int AT_ONCE = TOK < 4 ? 1 : 4;
    for (int k = k0; k < TOK; k += AT_ONCE * step) {
        int pos[AT_ONCE];
#pragma unroll
        for (int j = 0; j < AT_ONCE; j++) pos[j] = t0 + k + j * step < T ? r.positions[t0 + k + j * step] : 0;
#pragma unroll
        for (int j = 0; j < AT_ONCE; j++) {
            if (k + j * step >= TOK) break;
            double s, c;
            sincos_half_turns(double(pos[j]) * f, s, c);
            tab[(k + j * step) * pairs + p] = make_double2(c * r.mscale, (r.inverse ? -s : s) * r.mscale);
        }
    }
}

// A lane's eight values of a row: two fours, at a and at b.  Of ENDS pairs the
// fours are the two ends of four of them, or eight neighbours that are not
// turned; else they are eight neighbours.  For each of its four pairs the
// lane keeps cosine and sine (64 bits) over all heads of a token.
enum Pairs : int {
    ENDS,                     // (i, i + rot/2), rot/2 a multiple of four
    SIDE,                     // (2i, 2i + 1)
    ODD,                      // (i, i + rot/2), any: partners are looked up one by one
};

template <Pairs P>
struct Turn {
    int a, b, n;              // n: pairs that are turned, the first ones
    double c[4], s[4];
    __device__ __forceinline__ void place(const RopeArgs &r, int sub) {
        const int half = r.rot / 2;
        const bool ends = P == ENDS && sub < half / 4;
        a = ends ? 4 * sub : P == ENDS ? r.rot + 8 * (sub - half / 4) : 8 * sub;
        b = ends ? a + half : a + 4;
        n = P == SIDE ? min(max(half - 4 * sub, 0), 4) : ends ? 4 : 0;
    }
    __device__ __forceinline__ void set(const double2 *tab, int sub) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const double2 t = i < n ? tab[4 * sub + i] : make_double2(1.0, 0.0);
            c[i] = t.x;
            s[i] = t.y;
        }
    }
    // Two products and a sum in 64 bits, rounded to fp32 once.
    static __device__ __forceinline__ void pair(float &x, float &y, double c, double s) {
        const double u = x, w = y;
        x = float(u * c - w * s);
        y = float(w * c + u * s);
    }
    __device__ __forceinline__ void apply(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (i < n) pair(v[P == SIDE ? 2 * i : i], v[P == SIDE ? 2 * i + 1 : 4 + i], c[i], s[i]);
    }
    template <typename T>
    __device__ __forceinline__ void apply_odd(const RopeArgs &r, const T *row, const double2 *tab, float (&v)[8]) const {
        const int half = r.rot / 2;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int e = a + i;
            if (e >= r.rot) continue;
            const double2 t = tab[e < half ? e : e - half];
            const double w = row[e < half ? e + half : e - half];
            v[i] = float(double(v[i]) * t.x + (e < half ? -w : w) * t.y);
        }
    }
};

template <typename T>
struct Raw {
    T t[8];
    __device__ __forceinline__ void load(const T *row, int a, int b) {        // rows may start at any multiple of the type's size
        __builtin_memcpy(t, row + a, 4 * sizeof(T));
        __builtin_memcpy(t + 4, row + b, 4 * sizeof(T));
    }
    __device__ __forceinline__ void load8(const T *p) { __builtin_memcpy(t, p, sizeof(t)); }
    __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = float(t[i]);
    }
};

// Lanes that share a row: a power of two, so that a row lies within a wave
// (turned in place, every lane's loads are then before any lane's stores).
__device__ __forceinline__ int row_lanes(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : 64; }

// ---------------------------------------------------------------------------
// Rotary positions.
// ---------------------------------------------------------------------------
template <typename TI, typename TO, Pairs P, int TOK>
__global__ __launch_bounds__(256) void k_rope(const TI *x, int64_t ldt, int64_t ldh, TO *out, int64_t odt, int64_t odh,
                                              RopeArgs r, int64_t T, int H, int D) {
    __shared__ double2 tab[TOK * kRopeMaxDim / 2];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int64_t t0 = int64_t(blockIdx.x) * TOK, t = t0 + (TOK > 1 ? wv : 0);
    angles<TOK>(r, t0, T, tab);
    __syncthreads();
    const int lanes = row_lanes(D), rows = 64 / lanes, sub = lane & (lanes - 1);
    if (t >= T || 8 * sub >= D) return;
    const double2 *mine = tab + (TOK > 1 ? wv * (r.rot / 2) : 0);
    Turn<P> turn;
    turn.place(r, sub);
    turn.set(mine, sub);
    const TI *xt = x + t * ldt;
    TO *ot = out + t * odt;
    const int step = TOK > 1 ? rows : 4 * rows;
    int h = lane / lanes + (TOK > 1 ? 0 : rows * wv);
    if (h >= H) return;
    Raw<TI> cur, nxt;
    cur.load(xt + h * ldh, turn.a, turn.b);
    nxt = cur;
    for (; h < H; h += step) {
        if (h + step < H) nxt.load(xt + (h + step) * ldh, turn.a, turn.b);
        float v[8];
        cur.values(v);
        if constexpr (P == ODD)
            turn.apply_odd(r, xt + h * ldh, mine, v);
        else
            turn.apply(v);
        TO o[8];
#pragma unroll
        for (int i = 0; i < 8; i++) o[i] = TO(v[i]);
        __builtin_memcpy(ot + h * odh + turn.a, o, 4 * sizeof(TO));
        __builtin_memcpy(ot + h * odh + turn.b, o + 4, 4 * sizeof(TO));
        cur = nxt;
    }
}

// ---------------------------------------------------------------------------
// Cache.
// ---------------------------------------------------------------------------
struct KvArgs {
    uint8_t *cache;
    const int32_t *slots;
    int64_t slots_end;        // tokens the cache holds
    int page_shift, H, D;
};

// Largest magnitude of a row (as integer bits), in all of its lanes.
__device__ __forceinline__ uint32_t row_amax(const float (&x)[8], int lanes) {
    uint32_t am = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) am = max(am, __float_as_uint(x[j]) & 0x7fffffffu);
    for (int o = lanes / 2; o; o >>= 1) am = max(am, uint32_t(__shfl_xor(int(am), o)));
    return am;
}

// The tile that holds `slot` of head h.
__device__ __forceinline__ uint8_t *tile_of(const KvArgs &a, int slot, int h) {
    const int sh = a.page_shift - 4, page = slot >> a.page_shift, in = (slot >> 4) & ((1 << sh) - 1);
    return a.cache + (((int64_t(page) * a.H + h) << sh) + in) * kv_tile_bytes(a.D);
}

// Heads of a workgroup of the sixteen-token form.  Four compute an angle for
// more heads, two make more workgroups: 8192 tokens of 4 heads 11.6 and 11.8 us
// turned, 9.6 and 8.6 not; 1024 tokens of 8 heads 8.4 and 6.6.
constexpr int kWriteHeads = 2;

// One token a workgroup.
template <typename TI, Pairs P>
__global__ __launch_bounds__(256) void k_kv_write(const TI *__restrict__ k, int64_t kdt, int64_t kdh,
                                                  const TI *__restrict__ v, int64_t vdt, int64_t vdh, RopeArgs r, KvArgs a) {
    __shared__ double2 tab[128];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, D = a.D;
    const int64_t t = blockIdx.x;
    if (r.rot) angles<1>(r, t, t + 1, tab);
    __syncthreads();
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.slots_end) return;         // a token that is not kept
    const int lanes = row_lanes(D), rows = 64 / lanes, sub = lane & (lanes - 1), e0 = 8 * sub;
    Turn<P> turn;
    turn.place(r, sub);
    turn.set(tab, sub);
    const int in = slot & 15;
    // rows: the key heads, then the value heads; a wave's rows are of both kinds where the heads are few
    for (int i = lane / lanes + rows * wv; i < 2 * a.H; i += 4 * rows) {
        const bool is_v = i >= a.H;
        const int h = is_v ? i - a.H : i;
        const TI *row = is_v ? v + t * vdt + h * vdh : k + t * kdt + h * kdh;
        Raw<TI> raw;
        raw.load(row, is_v ? e0 : turn.a, is_v ? e0 + 4 : turn.b);
        float x[8];
        raw.values(x);
        if (!is_v) {
            if constexpr (P == ODD)
                turn.apply_odd(r, row, tab, x);
            else
                turn.apply(x);
        }
        const RowCode code(row_amax(x, lanes));
        const uint2 c = encode8(x, code);
        uint8_t *tile = tile_of(a, slot, h);
        if (is_v) {
            uint8_t *at = tile + 16 * D + (e0 >> 6) * 1024 + (in >> 2) * 256 + (e0 & 63) * 4 + (in & 3);
#pragma unroll
            for (int j = 0; j < 8; j++) at[4 * j] = uint8_t((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
        } else {
            *reinterpret_cast<uint32_t *>(tile + (turn.a >> 4) * 256 + in * 16 + (turn.a & 15)) = c.x;
            *reinterpret_cast<uint32_t *>(tile + (turn.b >> 4) * 256 + in * 16 + (turn.b & 15)) = c.y;
        }
        if (sub == 0) reinterpret_cast<float *>(tile + 32 * D + (is_v ? 64 : 0))[in] = code.scale();
    }
}

// Sixteen tokens of kWriteHeads heads a workgroup.  Codes pass through LDS so
// that what is neighbours in the cache is written together: a key's 16 bytes
// beside the next tokens', a value's four tokens as one dword (written a byte
// at a time, 32768 tokens of 4 heads of 128 took 60 us; so 24).
template <typename TI, Pairs P, int D>
__global__ __launch_bounds__(256) void k_kv_write16(const TI *__restrict__ k, int64_t kdt, int64_t kdh,
                                                    const TI *__restrict__ v, int64_t vdt, int64_t vdh, RopeArgs r, KvArgs a,
                                                    int64_t T) {
    constexpr int LANES = D / 8, PITCH = D + 16, ROWS = 256 / LANES;
    constexpr int PASSES = ROWS < 16 ? 16 / ROWS : 1, PARTS = ROWS > 16 ? ROWS / 16 : 1;
    __shared__ double2 tab[16 * (D / 2)];
    __shared__ __align__(16) uint8_t S[2 * kWriteHeads][16][PITCH];   // the keys of the heads, then the values
    __shared__ float S_d[2 * kWriteHeads][16];
    __shared__ int S_slot[16];
    const int tid = threadIdx.x, groups = (a.H + kWriteHeads - 1) / kWriteHeads;
    const int h0 = kWriteHeads * int(blockIdx.x % groups), heads = min(kWriteHeads, a.H - h0);
    const int64_t t0 = int64_t(blockIdx.x / groups) * 16;
    const int n = int(min(int64_t(16), T - t0));
    if (tid < 16) {
        const int slot = tid < n ? a.slots[t0 + tid] : -1;
        S_slot[tid] = slot < a.slots_end ? max(slot, -1) : -1;
    }
    const int sub = tid % LANES, e0 = 8 * sub, part = tid / LANES / 16, row = tid / LANES % 16;
    // One item is a token and head, keys and values; the next one's are loaded before this one's are used, and the first
    // before the angles are.
    struct Item {
        Raw<TI> k, v;
    };
    const int per_pass = (heads - part + PARTS - 1) / PARTS, items = per_pass > 0 ? PASSES * per_pass : 0;
    Turn<P> turn;
    turn.place(r, sub);
    auto key_row = [&](int pass, int h) {                             // past the last token: that one again, not stored
        return k + (t0 + min(row + ROWS * pass, n - 1)) * kdt + (h0 + h) * kdh;
    };
    auto fetch = [&](int i, Item &it) {
        const int pass = PASSES == 1 ? 0 : i / per_pass, h = part + PARTS * (i - pass * per_pass);
        it.k.load(key_row(pass, h), turn.a, turn.b);
        it.v.load8(v + (t0 + min(row + ROWS * pass, n - 1)) * vdt + (h0 + h) * vdh + e0);
    };
    Item cur, nxt;
    if (items) fetch(0, cur);
    nxt = cur;
    if (r.rot) angles<16>(r, t0, T, tab);
    __syncthreads();
    for (int i = 0; i < items; i++) {
        const int pass = PASSES == 1 ? 0 : i / per_pass, h = part + PARTS * (i - pass * per_pass), tok = row + ROWS * pass;
        const double2 *mine = tab + tok * (r.rot / 2);
        if (i + 1 < items) fetch(i + 1, nxt);
        if (i == 0 || (PASSES > 1 && i == pass * per_pass)) turn.set(mine, sub);
        float x[8];
        cur.k.values(x);
        if constexpr (P == ODD)
            turn.apply_odd(r, key_row(pass, h), mine, x);
        else
            turn.apply(x);
        const RowCode kc(row_amax(x, LANES));
        uint2 c = encode8(x, kc);
        *reinterpret_cast<uint32_t *>(&S[h][tok][turn.a]) = c.x;
        *reinterpret_cast<uint32_t *>(&S[h][tok][turn.b]) = c.y;
        cur.v.values(x);
        const RowCode vc(row_amax(x, LANES));
        c = encode8(x, vc);
        *reinterpret_cast<uint2 *>(&S[heads + h][tok][e0]) = c;
        if (sub == 0) {
            S_d[h][tok] = kc.scale();
            S_d[heads + h][tok] = vc.scale();
        }
        cur = nxt;
    }
    __syncthreads();
    // keys: 16 bytes of a token, the tokens side by side
    for (int u = tid; u < heads * 16 * (D / 16); u += 256) {
        const int tok = u % 16, c = u / 16 % (D / 16), which = u / D, slot = S_slot[tok];
        if (slot >= 0)
            *reinterpret_cast<uint4 *>(tile_of(a, slot, h0 + which) + c * 256 + (slot & 15) * 16) =
                *reinterpret_cast<const uint4 *>(&S[which][tok][16 * c]);
    }
    // values: where four tokens fill the four bytes of a dword, four dwords; else a byte at a time.  Fours begin at the
    // first token whose slot is a multiple of four.
    const int shift = -S_slot[0] & 3;
    uint32_t fours = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int j = shift + 4 * i, s = j + 3 < 16 ? S_slot[j] : -1;
        if (s >= 0 && !(s & 3) && S_slot[j + 1] == s + 1 && S_slot[j + 2] == s + 2 && S_slot[j + 3] == s + 3) fours |= 15u << j;
    }
    for (int u = tid; u < heads * D; u += 256) {           // four values of four tokens
        const int d = 4 * (u % (D / 4)), i = u / (D / 4) % 4, h = u / D, j = shift + 4 * i;
        if (!(fours >> j & 1)) continue;
        const int slot = S_slot[j];
        const uint32_t a0 = *reinterpret_cast<const uint32_t *>(&S[heads + h][j][d]), a1 = *reinterpret_cast<const uint32_t *>(&S[heads + h][j + 1][d]);
        const uint32_t a2 = *reinterpret_cast<const uint32_t *>(&S[heads + h][j + 2][d]), a3 = *reinterpret_cast<const uint32_t *>(&S[heads + h][j + 3][d]);
        const uint32_t p0 = __builtin_amdgcn_perm(a1, a0, 0x05010400u), p1 = __builtin_amdgcn_perm(a1, a0, 0x07030602u);
        const uint32_t p2 = __builtin_amdgcn_perm(a3, a2, 0x05010400u), p3 = __builtin_amdgcn_perm(a3, a2, 0x07030602u);
        const uint4 w = make_uint4(__builtin_amdgcn_perm(p2, p0, 0x05040100u), __builtin_amdgcn_perm(p2, p0, 0x07060302u),
                                   __builtin_amdgcn_perm(p3, p1, 0x05040100u), __builtin_amdgcn_perm(p3, p1, 0x07060302u));
        *reinterpret_cast<uint4 *>(tile_of(a, slot, h0 + h) + 16 * D + (d >> 6) * 1024 + ((slot & 15) >> 2) * 256 + (d & 63) * 4) = w;
    }
    if (fours != 0xffffu) {
        for (int u = tid; u < heads * 16 * D; u += 256) {
            const int d = u % D, tok = u / D % 16, h = u / (16 * D), slot = S_slot[tok];
            if (slot >= 0 && !(fours >> tok & 1))
                tile_of(a, slot, h0 + h)[16 * D + (d >> 6) * 1024 + ((slot & 15) >> 2) * 256 + (d & 63) * 4 + (slot & 3)] = S[heads + h][tok][d];
        }
    }
    for (int u = tid; u < 32 * heads; u += 256) {
        const int tok = u % 16, which = u / 16, slot = S_slot[tok];
        if (slot >= 0)
            reinterpret_cast<float *>(tile_of(a, slot, h0 + which % heads) + 32 * D + (which >= heads ? 64 : 0))[slot & 15] = S_d[which][tok];
    }
}

template <typename TO, int TOK>
__global__ __launch_bounds__(256) void k_kv_read(KvArgs a, TO *__restrict__ k, int64_t kdt, int64_t kdh,
                                                 TO *__restrict__ v, int64_t vdt, int64_t vdh, int64_t T) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, D = a.D;
    const int64_t t = int64_t(blockIdx.x) * TOK + (TOK > 1 ? wv : 0);
    if (t >= T) return;
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.slots_end) return;
    const int lanes = row_lanes(D), rows = 64 / lanes, e0 = 8 * (lane & (lanes - 1)), in = slot & 15;
    for (int i = lane / lanes + (TOK > 1 ? 0 : rows * wv); i < 2 * a.H; i += TOK > 1 ? rows : 4 * rows) {
        const bool is_v = i >= a.H;
        const int h = is_v ? i - a.H : i;
        const uint8_t *tile = tile_of(a, slot, h);
        const float d = reinterpret_cast<const float *>(tile + 32 * D + (is_v ? 64 : 0))[in];
        float x[8];
        if (is_v) {
            // the four tokens of a dword are neighbours: the other three are read by this workgroup's other waves, as a rule
            uint4 w[2];
            __builtin_memcpy(w, __builtin_assume_aligned(tile + 16 * D + (e0 >> 6) * 1024 + (in >> 2) * 256 + (e0 & 63) * 4, 16), 32);
            const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] = float(int8_t(u[j] >> (8 * (in & 3)))) * d;
            store8(v + t * vdt + h * vdh + e0, x);
        } else {
            const uint2 c = *reinterpret_cast<const uint2 *>(tile + (e0 >> 4) * 256 + in * 16 + (e0 & 15));
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] = float(int8_t((j < 4 ? c.x : c.y) >> (8 * (j & 3)))) * d;
            store8(k + t * kdt + h * kdh + e0, x);
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers.
// ---------------------------------------------------------------------------
// One token a workgroup of the rotation and of the read, until four of them
// still give every CU four (rope of 1024 x 28 x 128: 4.7 us against 5.3).
static bool few(int64_t T, int cu_count) { return T < 16 * int64_t(cu_count); }

static Pairs pairs_of(int layout, int rot) { return layout && rot ? SIDE : rot / 2 % 4 == 0 ? ENDS : ODD; }

template <typename TI, typename TO, Pairs P>
static void rope_laid(const TI *x, int64_t ldt, int64_t ldh, TO *out, int64_t odt, int64_t odh, const RopeArgs &r, int64_t T, int H,
                      int D, int cu_count, hipStream_t stream) {
    if (few(T, cu_count))
        k_rope<TI, TO, P, 1><<<dim3(unsigned(T)), 256, 0, stream>>>(x, ldt, ldh, out, odt, odh, r, T, H, D);
    else
        k_rope<TI, TO, P, 4><<<dim3(unsigned((T + 3) / 4)), 256, 0, stream>>>(x, ldt, ldh, out, odt, odh, r, T, H, D);
}

template <typename TI, typename TO>
static void rope_typed(const void *x, int64_t ldt, int64_t ldh, void *out, int64_t odt, int64_t odh, int layout, const RopeArgs &r,
                       int64_t T, int H, int D, int cu_count, hipStream_t stream) {
    const TI *xx = static_cast<const TI *>(x);
    TO *oo = static_cast<TO *>(out);
    const Pairs p = pairs_of(layout, r.rot);
    if (p == SIDE)
        rope_laid<TI, TO, SIDE>(xx, ldt, ldh, oo, odt, odh, r, T, H, D, cu_count, stream);
    else if (p == ENDS)
        rope_laid<TI, TO, ENDS>(xx, ldt, ldh, oo, odt, odh, r, T, H, D, cu_count, stream);
    else
        rope_laid<TI, TO, ODD>(xx, ldt, ldh, oo, odt, odh, r, T, H, D, cu_count, stream);
}

template <typename TI>
static void rope_from(const void *x, int64_t ldt, int64_t ldh, int out_type, void *out, int64_t odt, int64_t odh,
                      int layout, const RopeArgs &r, int64_t T, int H, int D, int cu_count, hipStream_t stream) {
    if (out_type == TYPE_F32)
        rope_typed<TI, float>(x, ldt, ldh, out, odt, odh, layout, r, T, H, D, cu_count, stream);
    else if (out_type == TYPE_BF16)
        rope_typed<TI, __bf16>(x, ldt, ldh, out, odt, odh, layout, r, T, H, D, cu_count, stream);
    else
        rope_typed<TI, _Float16>(x, ldt, ldh, out, odt, odh, layout, r, T, H, D, cu_count, stream);
}

hipError_t launch_rope(int type, const void *x, int64_t ldt, int64_t ldh, int out_type, void *out, int64_t odt, int64_t odh,
                       const int32_t *positions, const double *freqs, int rot, int layout, double mscale, int inverse,
                       int64_t T, int H, int D, int cu_count, hipStream_t stream) {
    const RopeArgs r{positions, freqs, mscale, rot, inverse};
    if (type == TYPE_F32)
        rope_from<float>(x, ldt, ldh, out_type, out, odt, odh, layout, r, T, H, D, cu_count, stream);
    else if (type == TYPE_BF16)
        rope_from<__bf16>(x, ldt, ldh, out_type, out, odt, odh, layout, r, T, H, D, cu_count, stream);
    else
        rope_from<_Float16>(x, ldt, ldh, out_type, out, odt, odh, layout, r, T, H, D, cu_count, stream);
    return hipGetLastError();
}

template <typename TI, Pairs P>
static void write_laid(const TI *kk, int64_t kdt, int64_t kdh, const TI *vv, int64_t vdt, int64_t vdh, const RopeArgs &r,
                       const KvArgs &a, int64_t T, int cu_count, hipStream_t stream) {
    // sixteen tokens a workgroup where every CU has one (1024 tokens of 8 heads of 128, turned: 8.4 -> 6.6 us), else one,
    // whose chain of loads is shorter (64 tokens of 4 heads: 4.1 us)
    const unsigned groups = unsigned(a.H + kWriteHeads - 1) / kWriteHeads;
    if ((T + 15) / 16 * groups < int64_t(cu_count)) {
        k_kv_write<TI, P><<<dim3(unsigned(T)), 256, 0, stream>>>(kk, kdt, kdh, vv, vdt, vdh, r, a);
        return;
    }
    // a launch holds fewer than 2^32 threads: slices of whole tokens
    const int64_t slice = ((int64_t(1) << 23) / groups) * 16;
    for (int64_t first = 0; first < T; first += slice) {
        const int64_t n = T - first < slice ? T - first : slice;
        RopeArgs rs = r;
        KvArgs as = a;
        rs.positions = r.positions ? r.positions + first : nullptr;
        as.slots = a.slots + first;
        const TI *ks = kk + first * kdt, *vs = vv + first * vdt;
        const dim3 grid(unsigned((n + 15) / 16) * groups);
        if (a.D == 64)
            k_kv_write16<TI, P, 64><<<grid, 256, 0, stream>>>(ks, kdt, kdh, vs, vdt, vdh, rs, as, n);
        else if (a.D == 128)
            k_kv_write16<TI, P, 128><<<grid, 256, 0, stream>>>(ks, kdt, kdh, vs, vdt, vdh, rs, as, n);
        else
            k_kv_write16<TI, P, 256><<<grid, 256, 0, stream>>>(ks, kdt, kdh, vs, vdt, vdh, rs, as, n);
    }
}

template <typename TI>
static void write_typed(const void *k, int64_t kdt, int64_t kdh, const void *v, int64_t vdt, int64_t vdh, int layout,
                        const RopeArgs &r, const KvArgs &a, int64_t T, int cu_count, hipStream_t stream) {
    const TI *kk = static_cast<const TI *>(k), *vv = static_cast<const TI *>(v);
    const Pairs p = pairs_of(layout, r.rot);             // nothing turned (rot 0): ENDS
    if (p == SIDE)
        write_laid<TI, SIDE>(kk, kdt, kdh, vv, vdt, vdh, r, a, T, cu_count, stream);
    else if (p == ENDS)
        write_laid<TI, ENDS>(kk, kdt, kdh, vv, vdt, vdh, r, a, T, cu_count, stream);
    else
        write_laid<TI, ODD>(kk, kdt, kdh, vv, vdt, vdh, r, a, T, cu_count, stream);
}

static KvArgs kv_args(void *cache, const int32_t *slots, int64_t n_pages, int page, int H, int D) {
    return KvArgs{static_cast<uint8_t *>(cache), slots, n_pages * page, __builtin_ctz(unsigned(page)), H, D};
}

hipError_t launch_kv_write(int type, const void *k, int64_t kdt, int64_t kdh, const void *v, int64_t vdt, int64_t vdh,
                           const int32_t *positions, const double *freqs, int rot, int layout, double mscale,
                           const int32_t *slots, int64_t T, void *cache, int64_t n_pages, int page, int H, int D, int cu_count,
                           hipStream_t stream) {
    const RopeArgs r{positions, freqs, mscale, rot, 0};
    const KvArgs a = kv_args(cache, slots, n_pages, page, H, D);
    if (type == TYPE_F32)
        write_typed<float>(k, kdt, kdh, v, vdt, vdh, layout, r, a, T, cu_count, stream);
    else if (type == TYPE_BF16)
        write_typed<__bf16>(k, kdt, kdh, v, vdt, vdh, layout, r, a, T, cu_count, stream);
    else
        write_typed<_Float16>(k, kdt, kdh, v, vdt, vdh, layout, r, a, T, cu_count, stream);
    return hipGetLastError();
}

template <typename TO>
static void read_typed(const KvArgs &a, void *k, int64_t kdt, int64_t kdh, void *v, int64_t vdt, int64_t vdh, int64_t T,
                       int cu_count, hipStream_t stream) {
    TO *kk = static_cast<TO *>(k), *vv = static_cast<TO *>(v);
    if (few(T, cu_count))
        k_kv_read<TO, 1><<<dim3(unsigned(T)), 256, 0, stream>>>(a, kk, kdt, kdh, vv, vdt, vdh, T);
    else
        k_kv_read<TO, 4><<<dim3(unsigned((T + 3) / 4)), 256, 0, stream>>>(a, kk, kdt, kdh, vv, vdt, vdh, T);
}

hipError_t launch_kv_read(int type, const void *cache, int64_t n_pages, int page, int H, int D, const int32_t *slots, int64_t T,
                          void *k, int64_t kdt, int64_t kdh, void *v, int64_t vdt, int64_t vdh, int cu_count,
                          hipStream_t stream) {
    const KvArgs a = kv_args(const_cast<void *>(cache), slots, n_pages, page, H, D);
    if (type == TYPE_F32)
        read_typed<float>(a, k, kdt, kdh, v, vdt, vdh, T, cu_count, stream);
    else if (type == TYPE_BF16)
        read_typed<__bf16>(a, k, kdt, kdh, v, vdt, vdh, T, cu_count, stream);
    else
        read_typed<_Float16>(a, k, kdt, kdh, v, vdt, vdh, T, cu_count, stream);
    return hipGetLastError();
}

}  // namespace mmq
