// i8_kernels.hip -- gfx950 kernels of the per-token / per-channel int8
// operators.
//
//   k_quantize_i8   rows of fp32 / bf16 / fp16 (or silu(gate) * up) -> int8
//                   codes and one fp32 scale per row
//   k_gemm_i8       int8 x int8 -> fp32 / bf16 / fp16 with a scale per row
//                   (token) and per column (channel), dense or grouped by
//                   expert
//
// With one scale per row of each operand the integer sum runs over all of K:
//     out[m,n] = xs[m] * ws[n] * sum_k xq[m,k] * wq[n,k]
// so the matrix core accumulates int32 from the first to the last k-step and
// the scales are applied once per output element.  Integer sums are exact in
// any order: how K is split never changes a result.
#include <hip/hip_runtime.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include "i8_plan.hpp"

namespace mmq {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct I8Args {
    const uint8_t *x;         // codes, row pitch ldx
    const float *xs;
    const uint8_t *w;         // codes, row pitch ldw; experts N * ldw apart
    const float *ws;
    const float *bias;        // or null
    const int32_t *rows;      // grouped: row of x that each routed row reads, or null
    const int32_t *offsets;   // grouped: E + 1 group bounds
    void *out;                // row pitch ldo
    int64_t M, N, K, T;       // M: output rows; T: rows of x
    int64_t ldx, ldw, ldo;
    int E;                    // 0: dense
};

template <typename T> __device__ __forceinline__ float to_f32(T v) { return float(v); }

// ---------------------------------------------------------------------------
// Row quantizer
// ---------------------------------------------------------------------------
template <typename T, bool SILU>
__global__ __launch_bounds__(256) void k_quantize_i8(const T *__restrict__ x, const T *__restrict__ up, int64_t ldx,
                                                     int8_t *__restrict__ q, int64_t ldq, float *__restrict__ scale,
                                                     int K) {
    const int64_t row = blockIdx.x;
    const T *xr = x + row * ldx;
    const T *ur = SILU ? up + row * ldx : nullptr;
    auto value = [&](int k) {
        const float v = to_f32(xr[k]);
        if constexpr (SILU) return v / (1.0f + expf(-v)) * to_f32(ur[k]);
        return v;
    };
    // the largest magnitude as integer bits: NaN > infinity > any finite
    uint32_t am = 0;
    for (int k = threadIdx.x; k < K; k += 256) am = max(am, __float_as_uint(value(k)) & 0x7fffffffu);
    __shared__ uint32_t part[4];
    for (int o = 32; o; o >>= 1) am = max(am, uint32_t(__shfl_xor(int(am), o)));
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = am;
    __syncthreads();
    am = max(max(part[0], part[1]), max(part[2], part[3]));
    const bool finite = am < 0x7f800000u;
    const float d = __uint_as_float(am) / 127.0f;
    float id = (finite && d != 0.0f) ? 1.0f / d : 0.0f;
    if (__builtin_isinf(id)) id = 0.0f;
    const int Kp = (K + 15) / 16 * 16;
    for (int k = threadIdx.x; k < Kp; k += 256) {
        int c = 0;
        if (k < K && finite) c = min(127, max(-127, int(roundf(value(k) * id))));
        q[row * ldq + k] = int8_t(c);
    }
    if (threadIdx.x == 0) scale[row] = finite ? d : __uint_as_float(0x7fc00000u);
}

// ---------------------------------------------------------------------------
// GEMM
// ---------------------------------------------------------------------------

// The group that tile `tile` of a grouped launch belongs to: its expert and
// its rows [row, end).  Expert e has ceil(len_e / TM) tiles; a wave scans the
// experts 64 at a time.  False past the last tile.  Bounds are clamped to
// [0, M], so no offsets make the kernel leave its buffers.
template <int TM>
__device__ __forceinline__ bool find_group(const int32_t *__restrict__ offsets, int E, int M, int tile, int &e,
                                           int &row, int &end) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        int b = 0, t = 0;
        if (e0 + lane < E) {
            b = min(max(offsets[e0 + lane], 0), M);
            t = min(max(offsets[e0 + lane + 1], 0), M);
        }
        const int n = t > b ? (t - b + TM - 1) / TM : 0;
        int upto = n;
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned long long hit = __ballot(before + upto > tile);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            e = __builtin_amdgcn_readfirstlane(e0 + l);
            row = __builtin_amdgcn_readlane(b, l) + (tile - before - __builtin_amdgcn_readlane(upto - n, l)) * TM;
            end = __builtin_amdgcn_readlane(t, l);
            return true;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

template <typename O, bool GROUPED>
__global__ __launch_bounds__(256) void k_gemm_i8(I8Args a, int tiles_n) {
    constexpr int TM = 128, TN = 128, TK = 64, P = TK + 16;   // padded rows in LDS
    __shared__ __align__(16) uint8_t sx[TM * P], sw[TN * P];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int tm = blockIdx.x / tiles_n, tn = blockIdx.x % tiles_n;
    int e = 0, row0 = tm * TM, end = int(a.M);
    if (GROUPED && !find_group<TM>(a.offsets, a.E, int(a.M), tm, e, row0, end)) return;
    const int64_t n0 = int64_t(tn) * TN;
    const uint8_t *w = a.w + int64_t(e) * a.N * a.ldw;
    const int K = int(a.K);

    // each thread stages 2 x 16 bytes of each operand per k-step
    int64_t xo[2], wo[2];
    for (int i = 0; i < 2; i++) {
        const int r = (tid + 256 * i) / 4;
        const int rr = min(row0 + r, end - 1);
        int64_t src = rr;
        if (GROUPED && a.rows) {
            src = a.rows[rr];
            src = src < 0 || src >= a.T ? 0 : src;
        }
        xo[i] = src * a.ldx;
        wo[i] = (n0 + r < a.N ? n0 + r : a.N - 1) * a.ldw;
    }
    const int kc = (tid & 3) * 16;
    i32x16 acc[2][2] = {};
    const int wm = (wv >> 1) * 64, wn = (wv & 1) * 64;
    for (int k = 0; k < K; k += TK) {
        i32x4 vx[2], vw[2];
        for (int i = 0; i < 2; i++) {
            const bool in = k + kc < K;
            vx[i] = in ? *reinterpret_cast<const i32x4 *>(a.x + xo[i] + k + kc) : i32x4{};
            vw[i] = in ? *reinterpret_cast<const i32x4 *>(w + wo[i] + k + kc) : i32x4{};
        }
        __syncthreads();
        for (int i = 0; i < 2; i++) {
            const int r = (tid + 256 * i) / 4;
            *reinterpret_cast<i32x4 *>(sx + r * P + kc) = vx[i];
            *reinterpret_cast<i32x4 *>(sw + r * P + kc) = vw[i];
        }
        __syncthreads();
        for (int ks = 0; ks < TK; ks += 32) {
            i32x4 fx[2], fw[2];
            for (int i = 0; i < 2; i++) {
                fx[i] = *reinterpret_cast<const i32x4 *>(sx + (wm + 32 * i + (lane & 31)) * P + ks + 16 * (lane >> 5));
                fw[i] = *reinterpret_cast<const i32x4 *>(sw + (wn + 32 * i + (lane & 31)) * P + ks + 16 * (lane >> 5));
            }
            for (int i = 0; i < 2; i++)
                for (int j = 0; j < 2; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fx[i], fw[j], acc[i][j], 0, 0, 0);
        }
    }
    O *out = static_cast<O *>(a.out);
    for (int j = 0; j < 2; j++) {
        const int64_t n = n0 + wn + 32 * j + (lane & 31);
        if (n >= a.N) continue;
        const float s = a.ws[int64_t(e) * a.N + n];
        const float bias = a.bias ? a.bias[n] : 0.0f;
        for (int i = 0; i < 2; i++)
            for (int r = 0; r < 16; r++) {
                const int m = row0 + wm + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                if (m >= end) continue;
                int src = m;
                if (GROUPED && a.rows) {
                    src = a.rows[m];
                    if (src < 0 || src >= a.T) continue;
                }
                float y = float(acc[i][j][r]) * a.xs[src] * s;
                if (a.bias) y += bias;
                out[int64_t(m) * a.ldo + n] = O(y);
            }
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
template <bool SILU>
static hipError_t launch_rows(int type, const void *x, const void *up, int64_t ldx, void *q, int64_t ldq, float *scale,
                              int64_t M, int64_t K, hipStream_t stream) {
    int8_t *qq = static_cast<int8_t *>(q);
    const dim3 grid((unsigned)M);
    if (type == TYPE_F32)
        k_quantize_i8<float, SILU><<<grid, 256, 0, stream>>>((const float *)x, (const float *)up, ldx, qq, ldq, scale, int(K));
    else if (type == TYPE_BF16)
        k_quantize_i8<__bf16, SILU><<<grid, 256, 0, stream>>>((const __bf16 *)x, (const __bf16 *)up, ldx, qq, ldq, scale, int(K));
    else
        k_quantize_i8<_Float16, SILU><<<grid, 256, 0, stream>>>((const _Float16 *)x, (const _Float16 *)up, ldx, qq, ldq, scale, int(K));
    return hipGetLastError();
}

// `up` null: quantize x; else silu(x) * up.
hipError_t launch_quantize_i8(int type, const void *x, const void *up, int64_t ldx, void *q, int64_t ldq, float *scale,
                              int64_t M, int64_t K, hipStream_t stream) {
    return up ? launch_rows<true>(type, x, up, ldx, q, ldq, scale, M, K, stream)
              : launch_rows<false>(type, x, up, ldx, q, ldq, scale, M, K, stream);
}

template <typename O>
static hipError_t launch_type(const I8Plan &p, const I8Args &a, hipStream_t stream) {
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n));
    if (a.E)
        k_gemm_i8<O, true><<<grid, 256, 0, stream>>>(a, int(p.tiles_n));
    else
        k_gemm_i8<O, false><<<grid, 256, 0, stream>>>(a, int(p.tiles_n));
    return hipGetLastError();
}

hipError_t launch_gemm_i8(const I8Plan &p, int type, const void *x, int64_t ldx, const float *xs, int64_t T,
                          const int32_t *rows, const int32_t *offsets, int experts, const void *w, int64_t ldw,
                          const float *ws, const float *bias, void *out, int64_t ldo, int64_t M, int64_t N, int64_t K,
                          hipStream_t stream) {
    const I8Args a{static_cast<const uint8_t *>(x), xs, static_cast<const uint8_t *>(w), ws, bias, rows, offsets, out,
                   M, N, K, T, ldx, ldw, ldo, experts};
    if (type == TYPE_F32) return launch_type<float>(p, a, stream);
    if (type == TYPE_BF16) return launch_type<__bf16>(p, a, stream);
    return launch_type<_Float16>(p, a, stream);
}

}  // namespace mmq
