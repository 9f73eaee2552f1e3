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

// A raw buffer whose lanes carry their own 32-bit offsets: every offset used
// stays below kBufBytes (checked before the launch), and a lane with nothing
// to fetch is sent to kNowhere, which reads as zero.
constexpr uint32_t kBufBytes = 0xfffff000u, kNowhere = 0xfffff800u;
static_assert(int64_t(kBufBytes) == kI8BufBytes, "plan and kernel disagree");
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t wide_rsrc(const uint8_t *base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), (short)0, int(kBufBytes), 0x00020000);
}
// 16 bytes per lane, global memory to LDS without registers: lane i's bytes
// land at lds + 16 i.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint8_t *lds, uint32_t off, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)lds, 16, int(off), soff, 0, 0);
}
__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off, int soff) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, int(off), soff, 0));
}

// This wave's DMA has landed, and after the barrier every wave's has.  (The
// barrier alone orders LDS traffic but does not wait for DMA.)
__device__ __forceinline__ void dma_barrier() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// Workgroups are dealt to the 8 XCDs in turn, and each XCD has an L2 of its
// own: hand every XCD a contiguous run of tiles instead, which walks bands of
// kBand row tiles column by column, so that the tiles in flight on an XCD
// share operand rows in its L2.
constexpr int kBand = 8;
__device__ __forceinline__ void tile_of_block(int tiles_m, int tiles_n, int &tm, int &tn) {
    const int n = gridDim.x, per = n / 8, rem = n % 8, xcd = blockIdx.x % 8;
    const int t = xcd * per + min(xcd, rem) + blockIdx.x / 8;
    const int size = kBand * tiles_n, b = t / size, r = t % size, h = min(kBand, tiles_m - b * kBand);
    tm = b * kBand + r % h;
    tn = r / h;
}

// Row of x that output row m reads; -1: the row is not to be written.
template <bool GROUPED>
__device__ __forceinline__ int source_row(const I8Args &a, int m) {
    if (!GROUPED || !a.rows) return m;
    const int t = a.rows[m];
    return uint32_t(t) < uint32_t(a.T) ? t : -1;
}

// The definition's roundings: fp32 sum, times xs, times ws, plus bias, then
// one to the output type.
template <typename O>
__device__ __forceinline__ O scaled(int sum, float xs, float ws, float bias, bool has_bias) {
    float y = float(sum) * xs * ws;
    if (has_bias) y += bias;
    return O(y);
}

// ---------------------------------------------------------------------------
// Tile kernel: BM x BN outputs per workgroup of WM x WN waves.
//
// Each k-step stages 128 bytes of every row of both operands by DMA into one
// of two LDS buffers.  A 32-byte sub-step of a wave's tile takes AI + BJ
// fragment reads (ds_read_b128: row lane % 32, 16-byte half lane / 32) and
// AI * BJ v_mfma_i32_32x32x32_i8.  The pipeline runs one sub-step ahead in
// registers and two k-steps ahead in memory: while the matrix core works on
// sub-step s the fragments of s + 1 are read; the step's barrier stands
// before its last sub-step, whose fragments are in registers by then, so the
// buffer is free for step ks + 2's DMA and the next step's first fragments
// load under the last sub-step's products.  The interleaving of reads, DMA
// and products is pinned with scheduling groups (left alone, the compiler
// sinks the reads behind the products: 8192 x 8192 x 8192 466 us against 450).
//
// LDS rows are 128 bytes; the eight 16-byte chunks of row r are stored at
// chunk ^ ((r / 2) % 8), so the 16 lanes that a ds_read_b128 serves at once
// (16 rows, one chunk) cover all 64 banks.  A DMA instruction writes 1 KiB of
// LDS in lane order, eight rows; choosing each lane's source chunk realises
// the order.  Rows past an operand's end repeat its last row (never stored);
// chunks past K read as zero.
//
// A = weights, B = activations, so a lane's accumulator registers hold four
// consecutive columns of one output row.  The epilogue scales them, passes
// each 32-row slab through LDS and stores 16 bytes per lane, 128 contiguous
// bytes per row.
// ---------------------------------------------------------------------------
template <int BM, int BN, int WM, int WN, typename O, bool GROUPED>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_i8_tile(I8Args a, int tiles_m, int tiles_n) {
    constexpr int W = WM * WN, AI = BM / WM / 32, BJ = BN / WN / 32, BK = 128;
    constexpr int UA = BM / 8 / W, UB = BN / 8 / W;      // DMA instructions per wave and k-step
    constexpr int OFF_W = BM * BK;
    static_assert(UA * 8 * W == BM && UB * 8 * W == BN && (UA == 1 || UA % 2 == 0) && (UB == 1 || UB % 2 == 0), "staging map");
    static_assert((BM + BN) * BK >= W * 4096 && (BM + BN) * BK >= (2 * BM + 2 * BN) * 4, "the epilogue reuses the buffers");
    // two variables: the compiler then sees that reads of one do not wait for DMA into the other
    __shared__ __align__(16) uint8_t S0[(BM + BN) * BK], S1[(BM + BN) * BK];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_of_block(tiles_m, tiles_n, tm, tn);
    int e = 0, row0 = tm * BM, end = int(a.M);
    if (GROUPED && !find_group<BM>(a.offsets, a.E, int(a.M), tm, e, row0, end)) return;
    const int n0 = tn * BN, K = int(a.K), N = int(a.N);
    const bool gather = GROUPED && a.rows;

    const __amdgpu_buffer_rsrc_t rx = wide_rsrc(a.x + (gather ? 0 : int64_t(row0) * a.ldx));
    const __amdgpu_buffer_rsrc_t rw = wide_rsrc(a.w + (int64_t(e) * a.N + n0) * a.ldw);
    // lane -> row lane / 8 of its instruction's eight, stored chunk lane % 8
    const int chunk = 16 * ((lane & 7) ^ (lane >> 4));   // of an even instruction; an odd one's differs in bit 6
    uint32_t va[UA], vb[UB];
#pragma unroll
    for (int u = 0; u < UA; u++) {
        const int r = min((wv * UA + u) * 8 + (lane >> 3), end - row0 - 1);
        const uint32_t src = gather ? uint32_t(max(source_row<GROUPED>(a, row0 + r), 0)) : uint32_t(r);
        va[u] = src * uint32_t(a.ldx) + (chunk ^ (((wv * UA + u) & 1) * 64));
    }
#pragma unroll
    for (int u = 0; u < UB; u++)
        vb[u] = uint32_t(min((wv * UB + u) * 8 + (lane >> 3), N - n0 - 1)) * uint32_t(a.ldw) +
                (chunk ^ (((wv * UB + u) & 1) * 64));
    const int steps = (K + BK - 1) / BK;
    auto load = [&](int ks, uint8_t *S) {                // past the last step: fetches nothing
        const int k0 = ks * BK;
        const bool in0 = k0 + chunk < K, in1 = k0 + (chunk ^ 64) < K;
#pragma unroll
        for (int u = 0; u < UA; u++)
            dma16(rx, S + (wv * UA + u) * 1024, (((wv * UA + u) & 1) ? in1 : in0) ? va[u] : kNowhere, k0);
#pragma unroll
        for (int u = 0; u < UB; u++)
            dma16(rw, S + OFF_W + (wv * UB + u) * 1024, (((wv * UB + u) & 1) ? in1 : in0) ? vb[u] : kNowhere, k0);
    };

    i32x16 acc[AI][BJ] = {};
    const int wm = (wv / WN) * (BM / WM), wn = (wv % WN) * (BN / WN), h = lane >> 5;
    const int a_off = (wm + (lane & 31)) * BK, b_off = OFF_W + (wn + (lane & 31)) * BK;
    int co[4];                                           // sub-step s: this lane's chunk
#pragma unroll
    for (int s = 0; s < 4; s++) co[s] = 16 * ((2 * s + h) ^ ((lane >> 1) & 7));
    i32x4 fa[2][AI], fb[2][BJ];
    auto frags = [&](const uint8_t *S, int s, int p) {
#pragma unroll
        for (int j = 0; j < BJ; j++) fb[p][j] = *reinterpret_cast<const i32x4 *>(S + b_off + co[s] + 32 * BK * j);
#pragma unroll
        for (int i = 0; i < AI; i++) fa[p][i] = *reinterpret_cast<const i32x4 *>(S + a_off + co[s] + 32 * BK * i);
    };
    auto mma = [&](int p) {
#pragma unroll
        for (int i = 0; i < AI; i++)
#pragma unroll
            for (int j = 0; j < BJ; j++)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[p][j], fa[p][i], acc[i][j], 0, 0, 0);
    };
    // scheduling groups: 0x008 products, 0x100 LDS reads, 0x010 memory instructions
    constexpr int NR = AI + BJ, NM = AI * BJ, REST = NM > NR ? NM - NR : 1;
    constexpr int QR = (NR + 1) / 2, QD = NM > QR ? NM - QR : 1, VP = (UA + UB + QD - 1) / QD;
    auto step = [&](int ks, uint8_t *cur, const uint8_t *nxt) {
#pragma unroll
        for (int s = 0; s < 3; s++) {
            frags(cur, s + 1, (s + 1) & 1);
            mma(s & 1);
#pragma unroll
            for (int q = 0; q < NR; q++) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, REST, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        dma_barrier();                                   // step ks + 1 has landed; `cur` is in registers
        frags(nxt, 0, 0);
        load(ks + 2, cur);
        mma(1);
#pragma unroll
        for (int q = 0; q < NM; q++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (q < QR)
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            else
                __builtin_amdgcn_sched_group_barrier(0x010, VP, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    load(0, S0);
    load(1, S1);
    dma_barrier();
    int ks = 0;
    if (row0 + wm < end) {
        frags(S0, 0, 0);
        for (; ks + 1 < steps; ks += 2) {
            step(ks, S0, S1);
            step(ks + 1, S1, S0);
        }
        if (ks < steps) step(ks, S0, S1);
    } else {                                             // no rows of this wave's tile exist: staging only
        for (; ks < steps; ks++) {
            dma_barrier();
            load(ks + 2, ks & 1 ? S1 : S0);
        }
    }
    dma_barrier();

    float *sxs = reinterpret_cast<float *>(S1), *sws = sxs + BM, *sbias = sws + BN;
    int *sdst = reinterpret_cast<int *>(sbias + BN);     // output row of each tile row, -1: none
    for (int r = tid; r < BM; r += 64 * W) {
        const int m = row0 + r, src = m < end ? source_row<GROUPED>(a, m) : -1;
        sdst[r] = src < 0 ? -1 : m;
        sxs[r] = src < 0 ? 0.0f : a.xs[src];
    }
    const bool has_bias = a.bias != nullptr;
    for (int r = tid; r < BN; r += 64 * W) {
        sws[r] = n0 + r < N ? a.ws[int64_t(e) * a.N + n0 + r] : 0.0f;
        if (has_bias) sbias[r] = n0 + r < N ? a.bias[n0 + r] : 0.0f;
    }
    __syncthreads();
    if (row0 + wm >= end) return;
    // GJ sub-tiles side by side fill 128-byte slab rows of CH chunks, stored swizzled
    constexpr int GJ = sizeof(O) == 2 && BJ % 2 == 0 ? 2 : 1, CH = GJ * 2 * int(sizeof(O)), PER = 16 / int(sizeof(O));
    uint8_t *slab = S0 + wv * 4096;
    O *out = static_cast<O *>(a.out);
    const int ml = lane & 31;
#pragma unroll
    for (int i = 0; i < AI; i++) {
        const float xs = sxs[wm + 32 * i + ml];
#pragma unroll
        for (int jj = 0; jj < BJ / GJ; jj++) {
#pragma unroll
            for (int g = 0; g < GJ; g++)
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const int j = jj * GJ + g, c = wn + 32 * j + 8 * q + 4 * h;
                    struct alignas(4 * sizeof(O)) { O v[4]; } o;
#pragma unroll
                    for (int r = 0; r < 4; r++)
                        o.v[r] = scaled<O>(acc[i][j][4 * q + r], xs, sws[c + r], has_bias ? sbias[c + r] : 0.0f, has_bias);
                    const int at = sizeof(O) == 2 ? 16 * ((4 * g + q) ^ (ml & (CH - 1))) + 8 * h
                                                  : 16 * ((2 * q + h) ^ (ml & (CH - 1)));
                    __builtin_memcpy(__builtin_assume_aligned(slab + ml * CH * 16 + at, 4 * sizeof(O)), &o, sizeof(o));
                }
#pragma unroll
            for (int it = 0; it < CH / 2; it++) {
                const int row = it * (64 / CH) + lane / CH, c = lane % CH;
                const i32x4 v = *reinterpret_cast<const i32x4 *>(slab + row * CH * 16 + 16 * (c ^ (row & (CH - 1))));
                const int dst = sdst[wm + 32 * i + row], n = n0 + wn + 32 * GJ * jj + c * PER;
                if (dst >= 0) {
                    O *o = out + int64_t(dst) * a.ldo + n;
                    if (n + PER <= N)
                        __builtin_memcpy(o, &v, 16);     // rows may start at any multiple of the type's size
                    else {
                        const O *ov = reinterpret_cast<const O *>(&v);
#pragma unroll
                        for (int q = 0; q < PER; q++)
                            if (n + q < N) o[q] = ov[q];
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Few-rows kernel: 16 * MB rows of x against 16 * NB weight rows per
// workgroup, bound by the weight stream.
//
// The eight waves split K: wave w takes the 128-byte units w, w + 8, ... of
// every row, each as two v_mfma_i32_16x16x64_i8 per block pair, fragments
// loaded straight into registers (lane: row lane % 16, 16 bytes lane / 16):
// nothing of the weights is used twice, so LDS would only add a trip.  The
// waves' int32 sums are added through LDS, exactly.
// ---------------------------------------------------------------------------
template <int MB, int NB, int DEPTH, typename O, bool GROUPED>
__global__ __launch_bounds__(512) void k_i8_rows(I8Args a, int tiles_m, int tiles_n) {
    constexpr int W = 8, BM = 16 * MB, BN = 16 * NB;
    __shared__ __align__(16) int part[W][MB * NB][4][64];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tn = blockIdx.x % tiles_n, tm = blockIdx.x / tiles_n;
    int e = 0, row0 = tm * BM, end = int(a.M);
    if (GROUPED && !find_group<BM>(a.offsets, a.E, int(a.M), tm, e, row0, end)) return;
    const int n0 = tn * BN, K = int(a.K), N = int(a.N);
    const bool gather = GROUPED && a.rows;
    const __amdgpu_buffer_rsrc_t rx = wide_rsrc(a.x + (gather ? 0 : int64_t(row0) * a.ldx));
    const __amdgpu_buffer_rsrc_t rw = wide_rsrc(a.w + (int64_t(e) * a.N + n0) * a.ldw);
    const int kc = 16 * (lane >> 4);
    uint32_t vx[MB], vw[NB];
#pragma unroll
    for (int j = 0; j < NB; j++) vw[j] = uint32_t(min(16 * j + (lane & 15), N - n0 - 1)) * uint32_t(a.ldw) + kc;
#pragma unroll
    for (int i = 0; i < MB; i++) {
        const int r = min(16 * i + (lane & 15), end - row0 - 1);
        vx[i] = (gather ? uint32_t(max(source_row<GROUPED>(a, row0 + r), 0)) : uint32_t(r)) * uint32_t(a.ldx) + kc;
    }
    i32x4 acc[MB][NB] = {};
    const int units = (K + 127) / 128;
    for (int u0 = wv; u0 < units; u0 += W * DEPTH) {
        i32x4 fw[DEPTH][2][NB], fx[DEPTH][2][MB];
#pragma unroll
        for (int d = 0; d < DEPTH; d++)
#pragma unroll
            for (int p = 0; p < 2; p++) {
                const int k0 = (u0 + d * W) * 128 + 64 * p;
                const bool in = k0 + kc < K;
#pragma unroll
                for (int j = 0; j < NB; j++) fw[d][p][j] = load16(rw, in ? vw[j] : kNowhere, k0);
#pragma unroll
                for (int i = 0; i < MB; i++) fx[d][p][i] = load16(rx, in ? vx[i] : kNowhere, k0);
            }
#pragma unroll
        for (int d = 0; d < DEPTH; d++)
#pragma unroll
            for (int p = 0; p < 2; p++)
#pragma unroll
                for (int i = 0; i < MB; i++)
#pragma unroll
                    for (int j = 0; j < NB; j++)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[d][p][j], fx[d][p][i], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < MB; i++)
#pragma unroll
        for (int j = 0; j < NB; j++)
#pragma unroll
            for (int r = 0; r < 4; r++) part[wv][i * NB + j][r][lane] = acc[i][j][r];
    __syncthreads();
    // register r of lane l: row (of x) l % 16, column 4 * (l / 16) + r
    const bool has_bias = a.bias != nullptr;
    O *out = static_cast<O *>(a.out);
    for (int o = tid; o < BM * BN; o += 512) {
        const int mr = o / BN, nr = o % BN, m = row0 + mr, n = n0 + nr;
        if (m >= end || n >= N) continue;
        const int src = source_row<GROUPED>(a, m);
        if (src < 0) continue;
        const int l = (mr & 15) + 16 * ((nr & 15) >> 2), r = nr & 3, b = (mr >> 4) * NB + (nr >> 4);
        int sum = 0;
#pragma unroll
        for (int w = 0; w < W; w++) sum += part[w][b][r][l];
        out[int64_t(m) * a.ldo + n] = scaled<O>(sum, a.xs[src], a.ws[int64_t(e) * a.N + n], has_bias ? a.bias[n] : 0.0f, has_bias);
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

template <typename O, bool GROUPED>
static void launch_kernel(const I8Plan &p, const I8Args &a, hipStream_t stream) {
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n));
    const int tm = int(p.tiles_m), tn = int(p.tiles_n);
    switch (p.kernel) {
    case I8_TILE_256x256: k_i8_tile<256, 256, 2, 4, O, GROUPED><<<grid, 512, 0, stream>>>(a, tm, tn); break;
    case I8_TILE_128x256: k_i8_tile<128, 256, 2, 4, O, GROUPED><<<grid, 512, 0, stream>>>(a, tm, tn); break;
    case I8_TILE_128x128: k_i8_tile<128, 128, 2, 4, O, GROUPED><<<grid, 512, 0, stream>>>(a, tm, tn); break;
    case I8_TILE_64x128: k_i8_tile<64, 128, 2, 2, O, GROUPED><<<grid, 256, 0, stream>>>(a, tm, tn); break;
    case I8_ROWS_16: k_i8_rows<1, 1, 4, O, GROUPED><<<grid, 512, 0, stream>>>(a, tm, tn); break;
    case I8_ROWS_32: k_i8_rows<2, 1, 2, O, GROUPED><<<grid, 512, 0, stream>>>(a, tm, tn); break;
    case I8_ROWS_64: k_i8_rows<4, 1, 2, O, GROUPED><<<grid, 512, 0, stream>>>(a, tm, tn); break;
    }
}

template <typename O>
static hipError_t launch_type(const I8Plan &p, const I8Args &a, hipStream_t stream) {
    if (a.E)
        launch_kernel<O, true>(p, a, stream);
    else
        launch_kernel<O, false>(p, a, stream);
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
