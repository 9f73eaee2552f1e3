// i8_kernels.hip -- gfx950 kernels of the per-token / per-channel int8
// operators.
//
//   k_quantize_i8   rows of fp32 / bf16 / fp16 (or silu(gate) * up) -> int8
//                   codes and one fp32 scale per row
//   k_i8_tile       int8 x int8 -> fp32 / bf16 / fp16 with a scale per row
//                   (token) and per column (channel), dense or grouped by
//                   expert, in tiles of 64 x 128 to 256 x 256 outputs
//   k_i8_rows       the same for few rows or few tiles, down to one token
//
// With one scale per row of each operand the integer sum runs over all of K:
//     out[m,n] = xs[m] * ws[n] * sum_k xq[m,k] * wq[n,k]
// so the matrix core accumulates int32 from the first to the last k-step and
// the scales are applied once per output element.  Integer sums are exact in
// any order: how K is split never changes a result.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "i8_codes.hpp"
#include "i8_plan.hpp"
#include "wave_scan.hpp"

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

// ---------------------------------------------------------------------------
// Row quantizer, bound by memory: a row is read once, held in registers as
// eight-value chunks while its largest magnitude is found, and written as
// codes, eight bytes a lane.  THREADS threads share a row; each holds CH
// chunks, and rows of more than THREADS * CH chunks are read again from the
// cache instead.  Measured at 2048 rows of 18944 bf16 (117 MB; a copy moves
// 5.2 TB/s here): 26.3 us = 4.4 TB/s, of which ~4 us is the launch and its
// ends; 512 threads of five chunks 27.3, and 163 for the first form, which
// read the row twice, a value a lane.  silu(gate) * up of two such (194 MB):
// 43.1 us = 4.5 TB/s against 48.8.
// ---------------------------------------------------------------------------
constexpr int kChunk = 8;

// Chunk c of a row of K values, zeros past its end.  Rows may start at any
// multiple of the type's size.
template <typename T>
__device__ __forceinline__ void load_chunk(const T *row, int c, int K, float (&v)[kChunk]) {
    T t[kChunk];
    if (kChunk * (c + 1) <= K)
        __builtin_memcpy(t, row + kChunk * c, sizeof(t));
    else
#pragma unroll
        for (int i = 0; i < kChunk; i++) t[i] = kChunk * c + i < K ? row[kChunk * c + i] : T(0.0f);
#pragma unroll
    for (int i = 0; i < kChunk; i++) v[i] = float(t[i]);
}

// v = silu(v) * u = v / (1 + exp(-v)) * u.  exp(-v) = 2^t * 2^lo with t =
// -v * log2(e) rounded to fp32 and lo what the rounding and the constant left
// out (2^lo = 1 + lo * ln 2 to fp32: |lo| < 2^-15): an ulp or two of error.
// The exponential takes v limited to 200 in magnitude, past which it is 0
// beside the 1, or the result is: the largest v would make t infinite and lo
// NaN.  The quotient is the hardware's reciprocal with a residual correction:
// half an ulp.  Where exp(-v) nears the largest number the 1 is far below its
// last bit: v * exp(v), the exponential scaled by 2^64 to stay a normal number.
// A chunk of gates below 86 in magnitude needs neither that nor the limit
// (which would change none of its values), and skips both: 2048 x 18944 bf16
// over eight inputs in turn 45.3 us against 46.4.  Which form a value takes
// depends on its own gate only.  With expf and a full divide everywhere:
// 8192 x 2047 bf16 19.4 us against 17.7.
__device__ __forceinline__ void silu_mul(float (&v)[kChunk], const float (&u)[kChunk]) {
    constexpr float L = 1.44269502162933349609375f, L_LO = 1.92596299112661746887e-8f, LN2 = 0.693147182464599609375f;
    constexpr float FAR = 86.0f, LIMIT = 200.0f;
    auto near = [](float g, float c) {           // c: g within the limit
        const float t = -c * L, lo = fmaf(-c, L_LO, fmaf(-c, L, -t)), x = __builtin_amdgcn_exp2f(t);
        const float s = 1.0f + fmaf(x, lo * LN2, x), r = __builtin_amdgcn_rcpf(s), y = g * r;
        return fmaf(fmaf(-s, y, g), r, y);
    };
    auto far = [](float g, float c) {
        const float t = c * L, lo = fmaf(c, L_LO, fmaf(c, L, -t)), x = __builtin_amdgcn_exp2f(t + 64.0f);
        return g * fmaf(x, lo * LN2, x) * 0x1p-64f;
    };
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunk; i++) most = fmaxf(most, fabsf(v[i]));
    if (most < FAR) {
#pragma unroll
        for (int i = 0; i < kChunk; i++) v[i] = near(v[i], v[i]) * u[i];
    } else {
#pragma unroll
        for (int i = 0; i < kChunk; i++) {
            const float g = v[i];
            v[i] = (g > -FAR ? near(g, fminf(g, LIMIT)) : far(g, fmaxf(g, -LIMIT))) * u[i];
        }
    }
}

template <typename T, bool SILU, int THREADS, int CH>
__global__ __launch_bounds__(THREADS < 256 ? 256 : THREADS) void k_quantize_i8(
    const T *__restrict__ x, const T *__restrict__ up, int64_t ldx, int8_t *__restrict__ q, int64_t ldq,
    float *__restrict__ scale, int64_t first, int M, int K) {
    constexpr int ROWS = THREADS < 256 ? 256 / THREADS : 1;
    const int tid = threadIdx.x % THREADS, chunks = (K + 15) / 16 * 2;   // codes are padded to a multiple of 16
    const int64_t row = first + int64_t(blockIdx.x) * ROWS + threadIdx.x / THREADS;
    if (ROWS > 1 && row >= M) return;                                    // whole waves: a row's threads are one
    const T *xr = x + row * ldx, *ur = SILU ? up + row * ldx : nullptr;
    // the largest magnitude as integer bits: NaN > infinity > any finite
    uint32_t am = 0;
    auto largest = [&](const float (&v)[kChunk]) {
#pragma unroll
        for (int i = 0; i < kChunk; i++) am = max(am, __float_as_uint(v[i]) & 0x7fffffffu);
    };
    float v[CH][kChunk];
    auto values = [&](int c, float (&w)[kChunk]) {
        load_chunk(xr, c, K, w);
        if constexpr (SILU) {
            float u[kChunk];
            load_chunk(ur, c, K, u);
            silu_mul(w, u);
        }
    };
#pragma unroll
    for (int i = 0; i < CH; i++)
        if (tid + i * THREADS < chunks) {
            values(tid + i * THREADS, v[i]);
            largest(v[i]);
        }
    for (int c = tid + CH * THREADS; c < chunks; c += THREADS) {
        float w[kChunk];
        values(c, w);
        largest(w);
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) am = max(am, uint32_t(__shfl_xor(int(am), o)));
    if constexpr (THREADS > 64) {
        __shared__ uint32_t part[THREADS / 64];
        if (tid % 64 == 0) part[tid / 64] = am;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 64; w++) am = max(am, part[w]);
    }
    const RowCode code(am);
    auto store = [&](int c, const float (&w)[kChunk]) {
        *reinterpret_cast<uint2 *>(q + row * ldq + kChunk * c) = encode8(w, code);
    };
#pragma unroll
    for (int i = 0; i < CH; i++)
        if (tid + i * THREADS < chunks) store(tid + i * THREADS, v[i]);
    for (int c = tid + CH * THREADS; c < chunks; c += THREADS) {
        float w[kChunk];
        values(c, w);
        store(c, w);
    }
    if (tid == 0) scale[row] = code.scale();
}

// ---------------------------------------------------------------------------
// GEMM
// ---------------------------------------------------------------------------

// The group that tile `tile` of a grouped launch belongs to: its expert and
// its rows [row, end).  A wave scans the experts 64 at a time; false past the
// last tile.  Offsets are clamped to [0, M], and a group starts no earlier
// than any before it ended, so whatever the offsets say, tiles lie within the
// buffers and there are at most M / TM + E of them.
template <int TM>
__device__ __forceinline__ bool find_group(const int32_t *__restrict__ offsets, int E, int M, int tile, int &e,
                                           int &row, int &end) {
    const int lane = threadIdx.x & 63;
    int before = 0, seen = min(max(offsets[0], 0), M);
    for (int e0 = 0; e0 < E; e0 += 64) {
        int t = 0;
        if (e0 + lane < E) t = min(max(offsets[e0 + lane + 1], 0), M);
        t = max(scan_max(t), seen);
        const int b = lane_before(t, seen);
        const int n = (t - b + TM - 1) / TM, upto = scan_sum(n);
        const unsigned long long hit = __ballot(before + upto > tile);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            e = __builtin_amdgcn_readfirstlane(e0 + l);
            row = __builtin_amdgcn_readlane(b, l) + (tile - before - __builtin_amdgcn_readlane(upto - n, l)) * TM;
            end = __builtin_amdgcn_readlane(t, l);
            return true;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
        seen = __builtin_amdgcn_readlane(t, 63);
    }
    return false;
}

// A raw buffer whose lanes carry their own 32-bit offsets: every offset used
// stays below kBufBytes (checked before the launch), and a lane with nothing
// to fetch is sent to kNowhere, which reads as zero.
constexpr uint32_t kBufBytes = 0xfffff000u, kNowhere = 0xfffff800u;
static_assert(int64_t(kBufBytes) == kI8BufBytes, "plan and kernel disagree");
typedef __attribute__((address_space(3))) void lds_void;

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
// Tile kernel: BM x BN outputs per tile, WM x WN waves, NS stages in LDS.
//
// A k-step is 128 bytes of every row of both operands, brought to LDS by DMA
// NS steps ahead.  The matrix instruction is v_mfma_i32_32x32x32_i8 with
// A = weights and B = activations, so that a lane's accumulator registers
// hold four consecutive columns of one output row.
//
// What bounds it.  Built without its products the kernel moves tiles at
// 12-14 TB/s out of the L2s, of which a quarter misses them; without its DMA
// it runs at 3.6 POP/s; both together, at the full chip's power-limited clock
// (1.7-2.0 GHz under this load), it reaches 2.2-2.3 (8192 x 18944 x 3584) to
// 2.6 (8192 x 8192 x 8192).  So the schedule has to keep loads in flight all
// the time and let no wave wait for LDS:
//
//  - A step's products run in two phases, first half of the tile's rows, then
//    the second, and the weights' fragments of the whole step stay in
//    registers between them.  The weights' and the first rows' buffers are
//    therefore free half a step before the second rows': their DMA for step
//    ks + NS goes out half a step earlier, which makes NS - 1/2 steps of
//    lead out of NS buffers (8192 x 18944 x 3584: 543 -> 521 us; one
//    256 x 256 tile per CU, K = 18944: 222 -> 176 us).
//  - A cluster is one 32-byte sub-step of one phase.  The fragments of the
//    next cluster are read behind the products of this one, and the DMA
//    instructions are spread over the clusters after the barrier that frees
//    their buffer.  The order is written out and pinned (left alone, the
//    compiler sinks the reads behind the products).
//  - DMA is issued and counted by hand.  The compiler cannot tell which LDS
//    buffer an LDS read depends on and would drain every DMA before it.
//    vmcnt retires in order, every step issues the same number of DMA
//    instructions (past the last step they fetch nothing), so "all but the
//    youngest (NS - 1) * U" names exactly the group a phase needs.
//  - Workgroups stay: each walks the tiles of its share, and the next tile's
//    first steps are under way while the last tile is scaled and written.  The
//    first products wait for their loads only, not for the stores issued
//    since, whose number is known: a tile that ends early writes its last row
//    from every lane past it (ragged groups: 512 rows over 128 experts in
//    256 x 256 tiles 101 -> 88 us, 12008 skewed rows 74.6 -> 71.1).
//
// LDS rows are 128 bytes; the eight 16-byte chunks of row r are stored at
// chunk ^ ((r / 2) % 8), so the 16 lanes that a ds_read_b128 serves at once
// (16 rows, one chunk) cover all 64 banks; choosing each DMA lane's source
// chunk realises the order.  Rows past an operand's end repeat its last row
// (never stored); chunks past K read as zero.
//
// The epilogue scales the accumulators, passes 32-row slabs through LDS and
// stores 16 bytes per lane, 128 contiguous bytes per row (stored straight
// from the registers, 32 bytes per row, 2048 x 3584 x 3584 took 35.1 us
// instead of 31.5).  A slab lies where the wave's own DMA of the last stage
// goes, and that stage is requested after it.
// ---------------------------------------------------------------------------

// 16 (4) bytes per lane from `r` + off + soff to LDS byte address lds + 16 i
// (4 i) of lane i.  The LDS address is the wave's, not the lane's.
__device__ __forceinline__ void dma16(i32x4 r, uint32_t lds, uint32_t off, int soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(off),
                 "s"(r), "s"(soff)
                 : "memory", "m0");
}
__device__ __forceinline__ void dma4(i32x4 r, uint32_t lds, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(r)
                 : "memory", "m0");
}
// All but this wave's N youngest memory instructions are done, and its LDS
// reads; after the barrier that holds for every wave.
template <int N>
__device__ __forceinline__ void wait_dma() {
    static_assert(N < 64, "vmcnt holds six bits");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
// Such a buffer's descriptor, in scalar registers.
__device__ __forceinline__ i32x4 wide_words(const void *base) {
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    i32x4 r{__builtin_amdgcn_readfirstlane(int(uint32_t(b))),
            __builtin_amdgcn_readfirstlane(int(uint32_t(b >> 32) & 0xffffu)), int(kBufBytes), 0x00020000};
    // a memory instruction reads a scalar register at least five wait states
    // after a vector instruction wrote it; the compiler does not see that the
    // assembly below is one
    asm volatile("s_nop 4" : "+s"(r));
    return r;
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return uint32_t(reinterpret_cast<uintptr_t>((lds_void *)p));
}

template <int N, typename F>
__device__ __forceinline__ void unrolled(F f) {
    if constexpr (N > 0) {
        unrolled<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}
template <int V> using constant = std::integral_constant<int, V>;

// Row tiles of every expert, by the rule of find_group: start[e] becomes the
// first tile of expert e, the sum is returned.  kLate marks an expert whose
// rows start behind its own offset, at the end of a group before it: there
// the offsets decrease.
constexpr int kLate = INT32_MIN, kTile = INT32_MAX;
template <int TM, int THREADS>
__device__ __forceinline__ int scan_groups(const I8Args &a, int *start, int *part) {
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, M = int(a.M);
    int tiles = 0, seen = min(max(a.offsets[0], 0), M);
    for (int e0 = 0; e0 < a.E; e0 += THREADS) {
        const int e = e0 + tid;
        int own = 0, t = 0;                                        // the group's offset and the one behind it
        if (e < a.E) {
            own = min(max(a.offsets[e], 0), M);
            t = min(max(a.offsets[e + 1], 0), M);
        }
        t = scan_max(t);
        if (lane == 63) part[wv] = t;
        __syncthreads();
        int last = seen, most = seen;                              // of the waves before this one, and of all
#pragma unroll
        for (int w = 0; w < THREADS / 64; w++) {
            if (w < wv) last = max(last, part[w]);
            most = max(most, part[w]);
        }
        t = max(t, last);
        const int b = lane_before(t, last);
        const int n = (t - b + TM - 1) / TM, upto = scan_sum(n);
        __syncthreads();
        if (lane == 63) part[wv] = upto;
        __syncthreads();
        int before = tiles, sum = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 64; w++) {
            if (w < wv) before += part[w];
            sum += part[w];
        }
        if (e < a.E) start[e] = (before + upto - n) | (b != own ? kLate : 0);
        tiles += sum;
        seen = most;
        __syncthreads();
    }
    return __builtin_amdgcn_readfirstlane(tiles);
}
// Where the rows of a late expert start: at the largest offset up to its own.
__device__ __forceinline__ int late_row(const I8Args &a, int e) {
    int t = 0;
    for (int i = threadIdx.x & 63; i <= e; i += 64) t = max(t, min(max(a.offsets[i], 0), int(a.M)));
    return __builtin_amdgcn_readlane(scan_max(t), 63);
}
// The expert of row tile `tile`: the last e with start[e] <= tile (of equal
// starts only the last has tiles).  64-way search by one wave.
__device__ __forceinline__ int group_of(const int *start, int E, int tile) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = E;
    while (n > 1) {
        const int stride = (n + 63) / 64;
        const bool ok = lane * stride < n && (start[lo + lane * stride] & kTile) <= tile;
        const int c = __popcll(__ballot(ok)) - 1;
        lo += c * stride;
        n = min(stride, n - c * stride);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Workgroups are dealt to the 8 XCDs in turn, and each XCD has an L2 of its
// own: every XCD gets a contiguous run of tiles, which walks bands of kBand
// row tiles column by column, so that the tiles in flight on an XCD share
// operand rows in its L2.  Measured at 8192 x 18944 x 3584 (256 x 256 /
// 128 x 256 tiles): bands of 4 527 / 577 us, 6 512 / 554, 8 524 / 593,
// 16 527 / 593.
constexpr int kBand = 6;

template <int BM, int BN, int WM, int WN, int NS, int OCC, typename O, bool GROUPED>
__global__ __launch_bounds__(64 * WM * WN, OCC) void k_i8_tile(I8Args a, int tiles_m, int tiles_n) {
    constexpr int W = WM * WN, AI = BM / WM / 32, BJ = BN / WN / 32, BK = 128, SUB = BK / 32;
    constexpr int UA = BM / 8 / W, UB = BN / 8 / W, U = UA + UB;   // DMA instructions (8 rows) per wave and step
    constexpr int AH = AI / 2, UH = UA / 2, G1 = UB + UH;          // ... of phase 0: the weights and half the rows
    constexpr int HW = BM / WM / 2;                                // rows of a wave's tile in one half
    constexpr int OFF_W = BM * BK, STAGE = (BM + BN) * BK, SCALES = BM + 2 * BN;
    static_assert(UA * 8 * W == BM && UB * 8 * W == BN && AI % 2 == 0 && UA % 2 == 0, "staging map");
    __shared__ __align__(1024) uint8_t S[NS * STAGE];
    __shared__ __align__(16) float scales[2][SCALES];              // xs, ws, bias of this tile and the next
    __shared__ int start[GROUPED ? kI8MaxExperts : 1], part[W];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = int(a.K), N = int(a.N), steps = (K + BK - 1) / BK;
    const bool gather = GROUPED && a.rows, has_bias = a.bias != nullptr;
    const uint32_t lds0 = lds_address(S), lds_scales = lds_address(scales);
    const int wm = (wv / WN) * 2 * HW, wn = (wv % WN) * (BN / WN), h = lane >> 5, ml = lane & 31;

    if (GROUPED) tiles_m = scan_groups<BM, 64 * W>(a, start, part);
    // this workgroup's tiles: every nb-th of its XCD's share
    const int total = tiles_m * tiles_n, xcd = blockIdx.x % 8, nb = (int(gridDim.x) - xcd + 7) / 8;
    int t = xcd * (total / 8) + min(xcd, total % 8) + blockIdx.x / 8;
    const int t_end = (xcd + 1) * (total / 8) + min(xcd + 1, total % 8);
    if (t >= t_end) return;

    // What follows from the lane number outside the products is computed for
    // every tile where the accumulators leave no room to keep it: kept, it
    // spilled, and every reload waited for the DMA and the stores under way
    // (8192 x 18944 x 3584 510 -> 495 us; smaller tiles are 1-2 % faster with it
    // kept).
    auto lane_anew = [&]() {
        int l = lane;
        if (AI * BJ >= 8) asm volatile("" : "+v"(l));
        return l;
    };
    // source chunk of this lane in DMA instruction u of an operand
    auto chunk_of = [](int lane, int u) { return 16 * ((lane & 7) ^ (((u * 8 + (lane >> 3)) >> 1) & 7)); };
    int row0, end, e, n0, stored;          // stored: bit i, this lane's row of sub-tile i exists
    i32x4 rx, rw;
    uint32_t va[UA], vb[UB];
    auto setup = [&]() {                   // tile t
        const int lane = lane_anew(), ml = lane & 31;
        const int size = kBand * tiles_n, b = t / size, r = t % size, hb = min(kBand, tiles_m - b * kBand);
        const int tm = b * kBand + r % hb;
        n0 = (r / hb) * BN;
        e = 0;
        row0 = tm * BM;
        end = int(a.M);
        if (GROUPED) {
            typedef const __attribute__((address_space(4))) int *scalar_ints;
            const scalar_ints off = (scalar_ints)a.offsets;
            e = group_of(start, a.E, tm);
            const int first = __builtin_amdgcn_readfirstlane(start[e]);
            row0 = (first & kLate ? late_row(a, e) : min(max(off[e], 0), end)) + (tm - (first & kTile)) * BM;
            end = min(max(off[e + 1], 0), end);
        }
        rx = wide_words(a.x + (gather ? 0 : int64_t(row0) * a.ldx));
        rw = wide_words(a.w + (int64_t(e) * N + n0) * a.ldw);
#pragma unroll
        for (int u = 0; u < UA; u++) {     // LDS holds the halves one after the other
            const int rh = (wv * UH + u % UH) * 8 + (lane >> 3);
            const int r = min((rh / HW) * 2 * HW + (u / UH) * HW + rh % HW, end - row0 - 1);
            const uint32_t src = gather ? uint32_t(max(source_row<GROUPED>(a, row0 + r), 0)) : uint32_t(r);
            va[u] = src * uint32_t(a.ldx) + chunk_of(lane, wv * UH + u % UH);
        }
#pragma unroll
        for (int u = 0; u < UB; u++)
            vb[u] = uint32_t(min((wv * UB + u) * 8 + (lane >> 3), N - n0 - 1)) * uint32_t(a.ldw) + chunk_of(lane, wv * UB + u);
        stored = 0;
#pragma unroll
        for (int i = 0; i < AI; i++) {
            const int m = row0 + wm + 32 * i + ml;
            if (m < end && source_row<GROUPED>(a, m) >= 0) stored |= 1 << i;
        }
    };
    // Instruction u of a step: UB of the weights, UH of the first rows, UH of
    // the second.  Chunks past K, and so whole steps past the last, fetch
    // nothing.
    auto load1 = [&](int u, int k0, int stage) {
        if (u < UB) {
            const bool in = k0 + chunk_of(lane, wv * UB + u) < K;
            dma16(rw, lds0 + stage * STAGE + OFF_W + (wv * UB + u) * 1024, in ? vb[u < UB ? u : 0] : kNowhere, k0);
        } else {
            const int v = u - UB;
            const bool in = k0 + chunk_of(lane, wv * UH + v % UH) < K;
            dma16(rx, lds0 + stage * STAGE + (v / UH) * (OFF_W / 2) + (wv * UH + v % UH) * 1024,
                  in ? va[v >= 0 && v < UA ? v : 0] : kNowhere, k0);
        }
    };
    auto load = [&](int ks, int stage, int u0, int u1) {
#pragma unroll
        for (int u = 0; u < U; u++)
            if (u >= u0 && u < u1) load1(u, ks * BK, stage);
    };
    auto load_scales = [&](int parity) {   // 64 values an instruction, dealt to the waves
        const i32x4 rs = wide_words(a.xs + (gather ? 0 : row0)), rv = wide_words(a.ws + int64_t(e) * N + n0);
        const i32x4 rb = wide_words(a.bias + n0);
        const uint32_t base = lds_scales + parity * SCALES * 4;
        const int lane = lane_anew();
        for (int g = wv; g < BM / 64; g += W) {
            const int r = g * 64 + lane, src = row0 + r >= end ? -1 : gather ? source_row<GROUPED>(a, row0 + r) : r;
            dma4(rs, base + g * 256, src < 0 ? kNowhere : uint32_t(src) * 4);
        }
        for (int g = W - 1 - wv; g < BN / 64; g += W) {
            const uint32_t off = n0 + g * 64 + lane < N ? uint32_t(g * 64 + lane) * 4 : kNowhere;
            dma4(rv, base + BM * 4 + g * 256, off);
            if (has_bias) dma4(rb, base + (BM + BN) * 4 + g * 256, off);
        }
    };

    i32x16 acc[AI][BJ];
    const int a_off = ((wv / WN) * HW + ml) * BK, b_off = OFF_W + (wn + ml) * BK;
    int co[SUB];                           // this lane's chunk of sub-step s: row lane % 32, half lane / 32
#pragma unroll
    for (int s = 0; s < SUB; s++) co[s] = 16 * ((2 * s + h) ^ ((lane >> 1) & 7));
    i32x4 fa[2][AH], fb[SUB][BJ];
    auto frag_b = [&](int j, int stage, int s) {
        fb[s][j] = *reinterpret_cast<const i32x4 *>(S + stage * STAGE + b_off + co[s] + 32 * BK * j);
    };
    auto frag_a = [&](int i, int stage, int half, int s, int p) {
        fa[p][i] = *reinterpret_cast<const i32x4 *>(S + stage * STAGE + half * (OFF_W / 2) + a_off + co[s] + 32 * BK * i);
    };
    // Products of row half HALF and sub-step SS; behind them the reads of the
    // next cluster's fragments (stage rstage) and DMA instructions D0 .. D1-1
    // of the step at k0 into dstage.
    auto cluster = [&](auto half_, auto s_, int rstage, auto d0_, auto d1_, int k0, int dstage) {
        constexpr int HALF = decltype(half_)::value, SS = decltype(s_)::value, P = SS & 1;
        constexpr int D0 = decltype(d0_)::value, ND = decltype(d1_)::value - D0, NM = AH * BJ;
        constexpr int NSUB = (SS + 1) % SUB, NHALF = SS + 1 < SUB ? HALF : 1 - HALF;
        constexpr int NB = NHALF == 0 ? BJ : 0, NR = AH + NB;      // phase 1 has the weights in registers
#pragma unroll
        for (int q = 0; q < NM; q++) {
            i32x16 &c = acc[HALF * AH + q / BJ][q % BJ];
            c = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[SS][q % BJ], fa[P][q / BJ], c, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < NR; r++)
                if (r * NM / NR == q) {                            // b0 a0 a1 .. b1 ..: as the products need them
                    const int ra = r - (NB ? 1 : 0);
                    if (NB && r == 0)
                        frag_b(0, rstage, NSUB);
                    else if (ra < AH)
                        frag_a(ra, rstage, NHALF, NSUB, 1 - P);
                    else
                        frag_b(r - AH, rstage, NSUB);
                }
#pragma unroll
            for (int d = 0; d < ND; d++)
                if (d * NM / (ND > 0 ? ND : 1) == q) load1(D0 + d, k0, dstage);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto step = [&](int ks, auto stage_) {
        constexpr int STG = decltype(stage_)::value, NXT = (STG + 1) % NS;
        const int k2 = (ks + NS) * BK;
        unrolled<SUB - 1>([&](auto s) { cluster(constant<0>{}, s, STG, constant<0>{}, constant<0>{}, 0, 0); });
        // the second rows have landed; the weights and the first rows are in registers
        wait_dma<(NS - 1) * U>();
        constexpr int D1 = (G1 + 3) / 4, D2 = D1 + (G1 - D1 + 2) / 3, D3 = D2 + (G1 - D2 + 1) / 2;
        cluster(constant<0>{}, constant<3>{}, STG, constant<0>{}, constant<D1>{}, k2, STG);
        cluster(constant<1>{}, constant<0>{}, STG, constant<D1>{}, constant<D2>{}, k2, STG);
        cluster(constant<1>{}, constant<1>{}, STG, constant<D2>{}, constant<D3>{}, k2, STG);
        cluster(constant<1>{}, constant<2>{}, STG, constant<D3>{}, constant<G1>{}, k2, STG);
        // the next step's weights and first rows have landed; the second rows are in registers
        wait_dma<(NS - 1) * U>();
        cluster(constant<1>{}, constant<3>{}, NXT, constant<G1>{}, constant<U>{}, k2, STG);
    };

    constexpr int PER = 16 / int(sizeof(O)), STORES = AI * BJ * 32 * 32 / (64 * PER);   // 16-byte stores per wave and tile
    constexpr int RB = UB >= 4 && BJ * 32 * sizeof(O) >= 128 ? 128 : 64, CH = RB / 16;  // slab row: bytes, chunks
    constexpr int CW = RB / int(sizeof(O));                                             // and columns
    static_assert(32 * RB <= UB * 1024, "a slab fits the wave's own DMA destination");
    setup();
    unrolled<NS>([&](auto i) { load(i, i, 0, U); });
    load_scales(0);
    // Younger than the loads of stage 0 are those of the other stages and, from
    // the second tile on, at least the stores of `behind` 32-row sub-tiles.
    int behind = 0;
    for (int parity = 0;; parity ^= 1) {
        bool waited = false;
        unrolled<AI>([&](auto i) {
            if (behind == i + 1) {
                wait_dma<(NS - 1) * U + (i + 1) * (STORES / AI)>();
                waited = true;
            }
        });
        if (!waited) wait_dma<(NS - 1) * U>();
        const bool active = row0 + wm < end;
        if (active) {
#pragma unroll
            for (int i = 0; i < AI; i++)
#pragma unroll
                for (int j = 0; j < BJ; j++) acc[i][j] = i32x16{};
#pragma unroll
            for (int j = 0; j < BJ; j++) frag_b(j, 0, 0);
#pragma unroll
            for (int i = 0; i < AH; i++) frag_a(i, 0, 0, 0, 0);
            int ks = 0;
            for (; ks + NS <= steps; ks += NS) unrolled<NS>([&](auto i) { step(ks + i, i); });
            unrolled<NS - 1>([&](auto i) {
                if (ks + i < steps) step(ks + i, i);
            });
        } else {                           // no rows of this wave's tile exist: staging only
            for (int ks = 0; ks < steps; ks++) {
                wait_dma<(NS - 1) * U>();
                load(ks + NS, ks % NS, 0, G1);
                wait_dma<(NS - 1) * U>();
                load(ks + NS, ks % NS, G1, U);
            }
        }
        wait_dma<0>();
        const int o_row = row0 + wm, o_n = n0 + wn, o_rows = min(end - o_row, 32 * AI), o_stored = stored;
        t += nb;
        const bool more = t < t_end;
        if (more) {
            setup();
            unrolled<NS - 1>([&](auto i) { load(i, i, 0, U); });
            load_scales(parity ^ 1);
        }
        behind = 0;
        if (active) {
            const int ln = lane_anew(), ml = ln & 31, h = ln >> 5;
            const float *sxs = scales[parity], *sws = sxs + BM, *sbias = sws + BN;
            O *out = static_cast<O *>(a.out) + int64_t(o_row) * a.ldo + o_n;
            const int n_left = N - o_n;
            // every row there is to write and every column: lanes past the
            // last row write that row again, so that each store is issued
            int rows_here = 0;
#pragma unroll
            for (int i = 0; i < AI; i++) rows_here |= 32 * i + ml < o_rows ? 1 << i : 0;
            const bool whole = __all(o_stored == rows_here) && BJ * 32 <= n_left;
            if (whole) behind = (o_rows + 31) / 32;
            uint8_t *slab = S + (NS - 1) * STAGE + OFF_W + wv * UB * 1024;
#pragma unroll
            for (int i = 0; i < AI; i++) {
                if (32 * i >= o_rows) break;
                const float xs = sxs[wm + 32 * i + ml];
#pragma unroll
                for (int cc = 0; cc < BJ * 32 / CW; cc++) {
                    asm volatile("" ::: "memory");                 // the scales are read again, not kept in registers
#pragma unroll
                    for (int g = 0; g < CW / 8; g++) {             // eight columns, four in each half of the wave
                        const int j = (cc * CW + 8 * g) / 32, q = (cc * CW / 8 + g) % 4, c = wn + 32 * j + 8 * q + 4 * h;
                        struct alignas(4 * sizeof(O)) { O v[4]; } o;
#pragma unroll
                        for (int r = 0; r < 4; r++)
                            o.v[r] = scaled<O>(acc[i][j][4 * q + r], xs, sws[c + r], has_bias ? sbias[c + r] : 0.0f, has_bias);
                        const int at = sizeof(O) == 2 ? 16 * (g ^ (ml & (CH - 1))) + 8 * h : 16 * ((2 * g + h) ^ (ml & (CH - 1)));
                        __builtin_memcpy(__builtin_assume_aligned(slab + ml * RB + at, 4 * sizeof(O)), &o, sizeof(o));
                    }
#pragma unroll
                    for (int it = 0; it < CH / 2; it++) {
                        const int row = min(it * (64 / CH) + ln / CH, o_rows - 1 - 32 * i), ck = ln % CH, n = cc * CW + ck * PER;
                        const i32x4 v = *reinterpret_cast<const i32x4 *>(slab + row * RB + 16 * (ck ^ (row & (CH - 1))));
                        O *p = out + int64_t(32 * i + row) * a.ldo + n;
                        if (whole)
                            __builtin_memcpy(p, &v, 16);           // rows may start at any multiple of the type's size
                        else if (__shfl(o_stored, row) >> i & 1) {
                            if (n + PER <= n_left)
                                __builtin_memcpy(p, &v, 16);
                            else {
                                const O *ov = reinterpret_cast<const O *>(&v);
#pragma unroll
                                for (int r = 0; r < PER; r++)
                                    if (n + r < n_left) p[r] = ov[r];
                            }
                        }
                    }
                }
            }
        }
        if (!more) break;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");         // the slab has been read
        load(NS - 1, NS - 1, 0, U);
    }
}

// ---------------------------------------------------------------------------
// Rows kernel: 16 * MB rows of x against 16 * NB weight rows per workgroup,
// for products too small to fill the device with tiles, down to one row,
// where the weight stream is all there is.
//
// The four waves split K: wave w takes the 128-byte units w, w + 4, ... of
// every row, each as two v_mfma_i32_16x16x64_i8 per pair of blocks, through a
// ring of two units in LDS of its own: no wave waits for another before the
// int32 sums are added, exactly, at the end.  The units come by DMA, eight
// rows of 128 bytes an instruction.  (Fragments loaded straight into
// registers touch 16 rows an instruction, which the address unit serves at
// 16 B/clk per CU instead of 53: 16 x 18944 x 3584 17.5 us against 13.0,
// 16 x 3584 x 18944 19.5 against 11.9.)  Rows of x that do not exist fetch
// nothing.  Two units per wave keep three to five workgroups on a CU; four
// units and eight waves, which leave one, were slower (18.7 us and 12.1).
// LDS chunks are swizzled as in the tile kernel.
// ---------------------------------------------------------------------------
template <int MB, int NB, typename O, bool GROUPED>
__global__ __launch_bounds__(256) void k_i8_rows(I8Args a, int tiles_n) {
    constexpr int W = 4, NS = 2, BM = 16 * MB, BN = 16 * NB;
    constexpr int D = 2 * (MB + NB), UNIT = D * 1024;      // DMA instructions and bytes of a unit
    static_assert(NS * UNIT >= MB * NB * 1024, "the sums reuse the ring");
    __shared__ __align__(1024) uint8_t S[W * NS * UNIT];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tn = blockIdx.x % tiles_n, tm = blockIdx.x / tiles_n;
    int e = 0, row0 = tm * BM, end = int(a.M);
    if (GROUPED && !find_group<BM>(a.offsets, a.E, int(a.M), tm, e, row0, end)) return;
    const int n0 = tn * BN, K = int(a.K), N = int(a.N), units = (K + 127) / 128;
    const bool gather = GROUPED && a.rows;
    const i32x4 rx = wide_words(a.x + (gather ? 0 : int64_t(row0) * a.ldx));
    const i32x4 rw = wide_words(a.w + (int64_t(e) * a.N + n0) * a.ldw);
    int ch[2];                                             // source chunk of even and odd instructions
#pragma unroll
    for (int p = 0; p < 2; p++) ch[p] = 16 * ((lane & 7) ^ ((p * 4 + (lane >> 4)) & 7));
    uint32_t off[D];                                       // 2 NB instructions of the weights, then 2 MB of x
#pragma unroll
    for (int d = 0; d < D; d++) {
        const int r = (d < 2 * NB ? d : d - 2 * NB) * 8 + (lane >> 3);
        if (d < 2 * NB)
            off[d] = uint32_t(min(r, N - n0 - 1)) * uint32_t(a.ldw) + ch[d & 1];
        else {
            const int src = row0 + r >= end ? -1 : gather ? source_row<GROUPED>(a, row0 + r) : r;
            off[d] = src < 0 ? kNowhere : uint32_t(src) * uint32_t(a.ldx) + ch[d & 1];
        }
    }
    const uint32_t ring = lds_address(S) + wv * NS * UNIT;
    auto load = [&](int u, int slot) {                     // past the last unit: fetches nothing
        const int k0 = u * 128;
        const bool in0 = k0 + ch[0] < K, in1 = k0 + ch[1] < K;
#pragma unroll
        for (int d = 0; d < D; d++)
            dma16(d < 2 * NB ? rw : rx, ring + slot * UNIT + d * 1024, (d & 1 ? in1 : in0) ? off[d] : kNowhere, k0);
    };
    i32x4 acc[MB][NB] = {};
    const uint8_t *mine = S + wv * NS * UNIT + (lane & 15) * 128;
    int co[2];                                             // fragment: row lane % 16, 16 bytes lane / 16 of each half
#pragma unroll
    for (int p = 0; p < 2; p++) co[p] = 16 * ((4 * p + (lane >> 4)) ^ ((lane >> 1) & 7));
#pragma unroll
    for (int i = 0; i < NS; i++) load(wv + i * W, i);
    int slot = 0;
    for (int u = wv; u < units; u += W, slot ^= 1) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 1) * D) : "memory");
        const uint8_t *s = mine + slot * UNIT;
        i32x4 fw[2][NB], fx[2][MB];
#pragma unroll
        for (int p = 0; p < 2; p++) {
#pragma unroll
            for (int j = 0; j < NB; j++) fw[p][j] = *reinterpret_cast<const i32x4 *>(s + j * 2048 + co[p]);
#pragma unroll
            for (int i = 0; i < MB; i++) fx[p][i] = *reinterpret_cast<const i32x4 *>(s + (NB + i) * 2048 + co[p]);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); // the slot is in registers
        load(u + NS * W, slot);
#pragma unroll
        for (int p = 0; p < 2; p++)
#pragma unroll
            for (int i = 0; i < MB; i++)
#pragma unroll
                for (int j = 0; j < NB; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[p][j], fx[p][i], acc[i][j], 0, 0, 0);
    }
    wait_dma<0>();
    int *part = reinterpret_cast<int *>(S);
#pragma unroll
    for (int i = 0; i < MB; i++)
#pragma unroll
        for (int j = 0; j < NB; j++)
            reinterpret_cast<i32x4 *>(part)[(wv * MB * NB + i * NB + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    // register r of lane l: row (of x) l % 16, column 4 * (l / 16) + r
    const bool has_bias = a.bias != nullptr;
    O *out = static_cast<O *>(a.out);
#pragma unroll
    for (int o = tid; o < BM * BN; o += 64 * W) {
        const int mr = o / BN, nr = o % BN, m = row0 + mr, n = n0 + nr;
        if (m >= end || n >= N) continue;
        const int src = source_row<GROUPED>(a, m);
        if (src < 0) continue;
        const int l = (mr & 15) + 16 * ((nr & 15) >> 2), r = nr & 3, b = (mr >> 4) * NB + (nr >> 4);
        int sum = 0;
#pragma unroll
        for (int w = 0; w < W; w++) sum += part[((w * MB * NB + b) * 64 + l) * 4 + r];
        out[int64_t(m) * a.ldo + n] =
            scaled<O>(sum, a.xs[src], a.ws[int64_t(e) * a.N + n], has_bias ? a.bias[n] : 0.0f, has_bias);
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
template <typename T, bool SILU>
static hipError_t launch_rows(const void *x, const void *up, int64_t ldx, void *q, int64_t ldq, float *scale, int64_t M,
                              int64_t K, hipStream_t stream) {
    const T *xx = static_cast<const T *>(x), *uu = static_cast<const T *>(up);
    int8_t *qq = static_cast<int8_t *>(q);
    const int m = int(M), k = int(K);
    // a launch holds fewer than 2^32 threads: at most kSlice rows each
    constexpr int64_t kSlice = int64_t(1) << 21;
    for (int64_t first = 0; first < M; first += kSlice) {
        const unsigned n = unsigned(M - first < kSlice ? M - first : kSlice);
        // threads per row: a wave up to 2048 values, else as many as hold the
        // row in three or four chunks
        if (K <= 64 * 4 * kChunk)
            k_quantize_i8<T, SILU, 64, 4><<<dim3((n + 3) / 4), 256, 0, stream>>>(xx, uu, ldx, qq, ldq, scale, first, m, k);
        else if (K <= 256 * 4 * kChunk)
            k_quantize_i8<T, SILU, 256, 4><<<dim3(n), 256, 0, stream>>>(xx, uu, ldx, qq, ldq, scale, first, m, k);
        else
            k_quantize_i8<T, SILU, 1024, 3><<<dim3(n), 1024, 0, stream>>>(xx, uu, ldx, qq, ldq, scale, first, m, k);
    }
    return hipGetLastError();
}

// `up` null: quantize x; else silu(x) * up.
hipError_t launch_quantize_i8(int type, const void *x, const void *up, int64_t ldx, void *q, int64_t ldq, float *scale,
                              int64_t M, int64_t K, hipStream_t stream) {
    if (type == TYPE_F32)
        return up ? launch_rows<float, true>(x, up, ldx, q, ldq, scale, M, K, stream)
                  : launch_rows<float, false>(x, up, ldx, q, ldq, scale, M, K, stream);
    if (type == TYPE_BF16)
        return up ? launch_rows<__bf16, true>(x, up, ldx, q, ldq, scale, M, K, stream)
                  : launch_rows<__bf16, false>(x, up, ldx, q, ldq, scale, M, K, stream);
    return up ? launch_rows<_Float16, true>(x, up, ldx, q, ldq, scale, M, K, stream)
              : launch_rows<_Float16, false>(x, up, ldx, q, ldq, scale, M, K, stream);
}

template <typename O, bool GROUPED>
static void launch_kernel(const I8Plan &p, const I8Args &a, hipStream_t stream) {
    const dim3 grid((unsigned)p.workgroups);
    const int tm = int(p.tiles_m), tn = int(p.tiles_n);
    switch (p.kernel) {
    case I8_TILE_256x256: k_i8_tile<256, 256, 2, 4, 2, 2, O, GROUPED><<<grid, 512, 0, stream>>>(a, tm, tn); break;
    case I8_TILE_128x256: k_i8_tile<128, 256, 2, 4, 3, 2, O, GROUPED><<<grid, 512, 0, stream>>>(a, tm, tn); break;
    case I8_TILE_128x128: k_i8_tile<128, 128, 2, 2, 2, 2, O, GROUPED><<<grid, 256, 0, stream>>>(a, tm, tn); break;
    case I8_TILE_64x128: k_i8_tile<64, 128, 1, 4, 2, 3, O, GROUPED><<<grid, 256, 0, stream>>>(a, tm, tn); break;
    case I8_ROWS_16x16: k_i8_rows<1, 1, O, GROUPED><<<grid, 256, 0, stream>>>(a, tn); break;
    case I8_ROWS_16x32: k_i8_rows<1, 2, O, GROUPED><<<grid, 256, 0, stream>>>(a, tn); break;
    case I8_ROWS_32x32: k_i8_rows<2, 2, O, GROUPED><<<grid, 256, 0, stream>>>(a, tn); break;
    case I8_ROWS_32x64: k_i8_rows<2, 4, O, GROUPED><<<grid, 256, 0, stream>>>(a, tn); break;
    case I8_ROWS_64x64: k_i8_rows<4, 4, O, GROUPED><<<grid, 256, 0, stream>>>(a, tn); break;
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
