// kv_kernels.hip -- gfx950 kernels of the rotary positions and of the int8
// paged cache.
//
//   k_rope       pairs of a head's values turned by position times frequency
//   k_kv_write   keys (turned first, if asked) and values -> int8 codes and a
//                scale per token and head, written to their slots
//   k_kv_read    the values that slots hold
//
// All three are bound by memory and by the launch.  A workgroup takes four
// tokens (one wave each), or one token when there are few; a row (one head of
// one token) lies across D / 8 lanes of a wave, eight values a lane.
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
    int interleaved;          // pairs (2i, 2i+1), else (i, i + rot/2)
    int inverse;
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    T t[8];
    __builtin_memcpy(t, p, sizeof(t));                   // rows may start at any multiple of the type's size
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = float(t[i]);
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    T t[8];
#pragma unroll
    for (int i = 0; i < 8; i++) t[i] = T(v[i]);
    __builtin_memcpy(p, t, sizeof(t));
}

// Cosine and sine (times mscale) of every pair of the workgroup's tokens.
// position * frequency reaches a million radians, where fp32 has no digits of
// the angle left: 64 bits, in half turns, so that the reduction is exact.
// One angle serves all heads of its token.
template <int TOK>
__device__ __forceinline__ void angles(const RopeArgs &r, int64_t t0, int64_t T, double2 *tab) {
    const int pairs = r.rot / 2;
    for (int i = threadIdx.x; i < TOK * pairs; i += 256) {
        const int k = i / pairs, p = i - k * pairs;
        if (t0 + k >= T) break;
        double s, c;
        sincospi(double(r.positions[t0 + k]) * (r.freqs[p] * 0.318309886183790671538), &s, &c);
        tab[i] = make_double2(c * r.mscale, (r.inverse ? -s : s) * r.mscale);
    }
}

// What a lane keeps of its eight values' pairs: factors of the value itself
// and of its partner.
struct Turn {
    double c[8], s[8];
    __device__ __forceinline__ void set(const RopeArgs &r, const double2 *tab, int e0) {
        const int half = r.rot / 2;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int e = e0 + i;
            c[i] = 1.0;
            s[i] = 0.0;
            if (e < r.rot) {
                const int p = r.interleaved ? e >> 1 : e < half ? e : e - half;
                const bool first = r.interleaved ? !(e & 1) : e < half;
                const double2 a = tab[p];
                c[i] = a.x;
                s[i] = first ? -a.y : a.y;
            }
        }
    }
    // Two products and a sum in 64 bits, rounded to fp32 once.
    __device__ __forceinline__ void apply(const RopeArgs &r, int e0, float (&v)[8], const float (&partner)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (e0 + i < r.rot) v[i] = float(double(v[i]) * c[i] + double(partner[i]) * s[i]);
    }
};

// The partners of row[e0 .. e0 + 7]; only those below rot are used.
template <typename T>
__device__ __forceinline__ void partners(const RopeArgs &r, const T *row, int e0, const float (&v)[8], float (&p)[8]) {
    if (r.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i++) p[i] = v[i ^ 1];
        return;
    }
    const int half = r.rot / 2;
    if (half % 8 == 0) {
        if (e0 < r.rot)
            load8(row + (e0 < half ? e0 + half : e0 - half), p);
        else
#pragma unroll
            for (int i = 0; i < 8; i++) p[i] = 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int e = e0 + i;
            p[i] = e < r.rot ? float(row[e < half ? e + half : e - half]) : 0.0f;
        }
    }
}

// Lanes that share a row: a power of two, so that a row lies within a wave
// (turned in place, every lane's loads are then before any lane's stores).
__device__ __forceinline__ int row_lanes(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : 64; }

// ---------------------------------------------------------------------------
// Rotary positions.
// ---------------------------------------------------------------------------
template <typename TI, typename TO, int TOK>
__global__ __launch_bounds__(256) void k_rope(const TI *x, int64_t ldt, int64_t ldh, TO *out, int64_t odt, int64_t odh,
                                              RopeArgs r, int64_t T, int H, int D) {
    __shared__ double2 tab[TOK * kRopeMaxDim / 2];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int64_t t0 = int64_t(blockIdx.x) * TOK, t = t0 + (TOK > 1 ? wv : 0);
    angles<TOK>(r, t0, T, tab);
    __syncthreads();
    const int lanes = row_lanes(D), rows = 64 / lanes, e0 = 8 * (lane & (lanes - 1));
    if (t >= T || e0 >= D) return;
    Turn turn;
    turn.set(r, tab + (TOK > 1 ? wv * (r.rot / 2) : 0), e0);
    const TI *xt = x + t * ldt;
    TO *ot = out + t * odt;
    for (int h = lane / lanes + (TOK > 1 ? 0 : rows * wv); h < H; h += TOK > 1 ? rows : 4 * rows) {
        float v[8], p[8];
        load8(xt + h * ldh + e0, v);
        partners(r, xt + h * ldh, e0, v, p);
        turn.apply(r, e0, v, p);
        store8(ot + h * odh + e0, v);
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

// The tile that holds `slot` of head h.
__device__ __forceinline__ uint8_t *tile_of(const KvArgs &a, int slot, int h) {
    const int sh = a.page_shift - 4, page = slot >> a.page_shift, in = (slot >> 4) & ((1 << sh) - 1);
    return a.cache + (((int64_t(page) * a.H + h) << sh) + in) * kv_tile_bytes(a.D);
}

template <typename TI, int TOK>
__global__ __launch_bounds__(256) void k_kv_write(const TI *__restrict__ k, int64_t kdt, int64_t kdh,
                                                  const TI *__restrict__ v, int64_t vdt, int64_t vdh, RopeArgs r, KvArgs a,
                                                  int64_t T) {
    __shared__ double2 tab[TOK * 128];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, D = a.D;
    const int64_t t0 = int64_t(blockIdx.x) * TOK, t = t0 + (TOK > 1 ? wv : 0);
    if (r.rot) angles<TOK>(r, t0, T, tab);
    __syncthreads();
    if (t >= T) return;
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.slots_end) return;         // a token that is not kept
    const int lanes = row_lanes(D), rows = 64 / lanes, sub = lane & (lanes - 1), e0 = 8 * sub;
    Turn turn;
    turn.set(r, tab + (TOK > 1 ? wv * (r.rot / 2) : 0), e0);
    const int in = slot & 15;
    // rows: the key heads, then the value heads; a wave's rows are of both kinds where the heads are few
    for (int i = lane / lanes + (TOK > 1 ? 0 : rows * wv); i < 2 * a.H; i += TOK > 1 ? rows : 4 * rows) {
        const bool is_v = i >= a.H;
        const int h = is_v ? i - a.H : i;
        float x[8];
        if (is_v) {
            load8(v + t * vdt + h * vdh + e0, x);
        } else {
            const TI *row = k + t * kdt + h * kdh;
            load8(row + e0, x);
            if (r.rot) {
                float p[8];
                partners(r, row, e0, x, p);
                turn.apply(r, e0, x, p);
            }
        }
        uint32_t am = 0;
#pragma unroll
        for (int j = 0; j < 8; j++) am = max(am, __float_as_uint(x[j]) & 0x7fffffffu);
        for (int o = lanes / 2; o; o >>= 1) am = max(am, uint32_t(__shfl_xor(int(am), o)));
        const RowCode code(am);
        const uint2 c = encode8(x, code);
        uint8_t *tile = tile_of(a, slot, h);
        if (is_v) {
            uint8_t *at = tile + 16 * D + (e0 >> 6) * 1024 + (in >> 2) * 256 + (e0 & 63) * 4 + (in & 3);
#pragma unroll
            for (int j = 0; j < 8; j++) at[4 * j] = uint8_t((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
        } else {
            *reinterpret_cast<uint2 *>(tile + (e0 >> 4) * 256 + in * 16 + (e0 & 15)) = c;
        }
        if (sub == 0) reinterpret_cast<float *>(tile + 32 * D + (is_v ? 64 : 0))[in] = code.scale();
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
// Launchers.  Four tokens a workgroup where that still gives every CU one.
// ---------------------------------------------------------------------------
static bool few(int64_t T, int cu_count) { return T < 4 * int64_t(cu_count); }

template <typename TI, typename TO>
static void rope_typed(const void *x, int64_t ldt, int64_t ldh, void *out, int64_t odt, int64_t odh, const RopeArgs &r,
                       int64_t T, int H, int D, int cu_count, hipStream_t stream) {
    const TI *xx = static_cast<const TI *>(x);
    TO *oo = static_cast<TO *>(out);
    if (few(T, cu_count))
        k_rope<TI, TO, 1><<<dim3(unsigned(T)), 256, 0, stream>>>(xx, ldt, ldh, oo, odt, odh, r, T, H, D);
    else
        k_rope<TI, TO, 4><<<dim3(unsigned((T + 3) / 4)), 256, 0, stream>>>(xx, ldt, ldh, oo, odt, odh, r, T, H, D);
}

template <typename TI>
static void rope_from(const void *x, int64_t ldt, int64_t ldh, int out_type, void *out, int64_t odt, int64_t odh,
                      const RopeArgs &r, int64_t T, int H, int D, int cu_count, hipStream_t stream) {
    if (out_type == TYPE_F32)
        rope_typed<TI, float>(x, ldt, ldh, out, odt, odh, r, T, H, D, cu_count, stream);
    else if (out_type == TYPE_BF16)
        rope_typed<TI, __bf16>(x, ldt, ldh, out, odt, odh, r, T, H, D, cu_count, stream);
    else
        rope_typed<TI, _Float16>(x, ldt, ldh, out, odt, odh, r, T, H, D, cu_count, stream);
}

hipError_t launch_rope(int type, const void *x, int64_t ldt, int64_t ldh, int out_type, void *out, int64_t odt, int64_t odh,
                       const int32_t *positions, const double *freqs, int rot, int layout, double mscale, int inverse,
                       int64_t T, int H, int D, int cu_count, hipStream_t stream) {
    const RopeArgs r{positions, freqs, mscale, rot, layout, inverse};
    if (type == TYPE_F32)
        rope_from<float>(x, ldt, ldh, out_type, out, odt, odh, r, T, H, D, cu_count, stream);
    else if (type == TYPE_BF16)
        rope_from<__bf16>(x, ldt, ldh, out_type, out, odt, odh, r, T, H, D, cu_count, stream);
    else
        rope_from<_Float16>(x, ldt, ldh, out_type, out, odt, odh, r, T, H, D, cu_count, stream);
    return hipGetLastError();
}

template <typename TI>
static void write_typed(const void *k, int64_t kdt, int64_t kdh, const void *v, int64_t vdt, int64_t vdh, const RopeArgs &r,
                        const KvArgs &a, int64_t T, int cu_count, hipStream_t stream) {
    const TI *kk = static_cast<const TI *>(k), *vv = static_cast<const TI *>(v);
    if (few(T, cu_count))
        k_kv_write<TI, 1><<<dim3(unsigned(T)), 256, 0, stream>>>(kk, kdt, kdh, vv, vdt, vdh, r, a, T);
    else
        k_kv_write<TI, 4><<<dim3(unsigned((T + 3) / 4)), 256, 0, stream>>>(kk, kdt, kdh, vv, vdt, vdh, r, a, T);
}

static KvArgs kv_args(void *cache, const int32_t *slots, int64_t n_pages, int page, int H, int D) {
    return KvArgs{static_cast<uint8_t *>(cache), slots, n_pages * page, __builtin_ctz(unsigned(page)), H, D};
}

hipError_t launch_kv_write(int type, const void *k, int64_t kdt, int64_t kdh, const void *v, int64_t vdt, int64_t vdh,
                           const int32_t *positions, const double *freqs, int rot, int layout, double mscale,
                           const int32_t *slots, int64_t T, void *cache, int64_t n_pages, int page, int H, int D, int cu_count,
                           hipStream_t stream) {
    const RopeArgs r{positions, freqs, mscale, rot, layout, 0};
    const KvArgs a = kv_args(cache, slots, n_pages, page, H, D);
    if (type == TYPE_F32)
        write_typed<float>(k, kdt, kdh, v, vdt, vdh, r, a, T, cu_count, stream);
    else if (type == TYPE_BF16)
        write_typed<__bf16>(k, kdt, kdh, v, vdt, vdh, r, a, T, cu_count, stream);
    else
        write_typed<_Float16>(k, kdt, kdh, v, vdt, vdh, r, a, T, cu_count, stream);
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
