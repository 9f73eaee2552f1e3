"""The per-token / per-channel int8 operators on the GPU against plain
implementations in 64 bits.

Tolerances.  The integer sum is exact; the definition then rounds to fp32 at
the conversion, at each of the two scale products and at the bias, and once to
the output type, so an output is within 3 u |y| + u |y + b| + h |out| of the
exact value (u = 2^-24, h = half a step of the type), to first order; 4 u and
5 u below leave room for the products of those terms.  The same roundings done
on the host in fp32 give the same bits, and that is asserted too.  Codes and
scales of the plain quantizer are fp32 arithmetic by definition and must be
equal; the bound for silu(gate) * up is derived where it is used."""
import numpy as np
import pytest
import torch

import block_quantized_int8_q8_amd as mmq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
U = 2.0 ** -24


def gen(seed):
    return torch.Generator().manual_seed(seed)


def codes(rows, K, seed, lo=-128, pitch=None):
    """int8 codes [rows, K] on the GPU, as a slice of wider rows if `pitch`."""
    full = torch.randint(lo, 128, (rows, pitch or K), generator=gen(seed), dtype=torch.int8)
    return full.to(DEV)[:, :K]


def scales(n, seed):
    return (torch.rand(n, generator=gen(seed)) * 0.05 + 1e-3).to(DEV)


def in_fp32(acc64, xs, ws, bias, dtype):
    """The definition's roundings, on the host: acc64 [M, N] exact integers."""
    y = acc64.to(F32) * xs[:, None] * ws
    if bias is not None:
        y = y + bias
    return y.to(dtype)


def check(out, acc64, xs, ws, bias, dtype):
    out, xs, ws = out.cpu(), xs.cpu(), ws.cpu()
    bias = None if bias is None else bias.cpu()
    y = acc64 * xs.double()[:, None] * ws.double()
    full = y if bias is None else y + bias.double()
    h = torch.finfo(dtype).eps / 2
    bound = 4 * U * y.abs() + 5 * U * full.abs() + h * full.abs() * (1 + 2 * h)
    if dtype == F16:
        bound = bound + 2.0 ** -25           # half the subnormal step
    over = full.abs() >= torch.finfo(dtype).max * (1 - h)
    assert bool(((out.double() - full).abs() <= bound)[~over].all())
    assert torch.equal(out, in_fp32(acc64, xs, ws, bias, dtype))


def exact_sum(xq, wq):
    return torch.matmul(xq.cpu().double(), wq.cpu().double().t())     # integers below 2^53: exact


# ---------------------------------------------------------------------------
# dense products
# ---------------------------------------------------------------------------
SHAPES = [(1, 1, 16), (1, 16, 16), (1, 33, 48), (1, 3584, 3584), (2, 65, 80), (3, 129, 128), (5, 512, 784), (7, 31, 1040),
          (8, 1000, 512), (9, 100, 2064), (13, 515, 3584), (16, 16, 64), (17, 64, 144), (31, 257, 272), (32, 96, 4096),
          (33, 47, 1008), (48, 200, 640), (63, 640, 256), (64, 64, 64), (65, 130, 400), (96, 1024, 512), (100, 1, 512),
          (127, 129, 160), (128, 128, 128), (129, 383, 528), (160, 2048, 336), (192, 70, 3200), (200, 1536, 768),
          (255, 257, 256), (256, 256, 272), (257, 600, 1024), (300, 2000, 96), (384, 512, 3584), (509, 768, 496),
          (512, 4608, 128), (700, 900, 112), (1000, 1030, 144), (1024, 768, 640), (2049, 385, 192), (2048, 3584, 64)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K):
    dtype = TYPES[(M + N + K // 16) % 3]
    xq, wq, xs, ws = codes(M, K, M), codes(N, K, N + 1), scales(M, 2), scales(N, 3)
    bias = torch.randn(N, generator=gen(4)).to(DEV) if (M + N) % 2 else None
    out = mmq.gemm_i8(xq, xs, wq, ws, bias=bias, dtype=dtype)
    assert out.shape == (M, N) and out.dtype == dtype
    check(out, exact_sum(xq, wq), xs, ws, bias, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K,px,pw,po", [(1, 100, 48, 64, 96, 101), (5, 70, 144, 160, 400, 77), (40, 129, 80, 80, 112, 131),
                                            (130, 260, 192, 4096, 208, 260), (300, 515, 272, 288, 272, 1031),
                                            (600, 1025, 128, 256, 144, 1025)])
def test_gemm_pitches_leave_the_rest_untouched(M, N, K, px, pw, po, dtype):
    """Rows with a pitch in every operand: columns between them are neither
    used (they hold codes too) nor written; the output rows start at any
    alignment of the type."""
    xq, wq, xs, ws = codes(M, K, 1, pitch=px), codes(N, K, 2, pitch=pw), scales(M, 3), scales(N, 4)
    flat = torch.full((M * po + 9,), -77.0, dtype=dtype, device=DEV)
    out = flat[1:1 + M * po].view(M, po)[:, :N]
    got = mmq.gemm_i8(xq, xs, wq, ws, out=out)
    assert got.data_ptr() == out.data_ptr()
    check(out, exact_sum(xq, wq), xs, ws, None, dtype)
    rest = torch.ones(flat.shape, dtype=torch.bool, device=DEV)
    rest[1:1 + M * po].view(M, po)[:, :N] = False
    assert bool((flat[rest] == -77.0).all())


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_gemm_longest_rows_and_extreme_codes(M):
    """K = 131056 of -128 * -128 is 2147221504, the largest sum there is."""
    K, N = mmq.I8_MAX_K, 40
    xq = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    wq = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    wq[1::2] = 127
    one = torch.ones(max(M, N), device=DEV)
    out = mmq.gemm_i8(xq, one[:M], wq, one[:N])
    want = torch.where(torch.arange(N) % 2 == 0, 16384.0 * K, -128.0 * 127.0 * K).to(F32)
    assert torch.equal(out.cpu(), want.expand(M, N))


@pytest.mark.parametrize("M", [2, 64, 300])
def test_gemm_nan_and_infinite_scales_stay_in_their_row_and_column(M):
    N, K = 200, 256
    xq, wq, xs, ws = codes(M, K, 1, lo=1), codes(N, K, 2, lo=1), scales(M, 3), scales(N, 4)
    xs[1], ws[7], ws[150] = float("nan"), float("inf"), 0.0
    out = mmq.gemm_i8(xq, xs, wq, ws).cpu()
    assert bool(out[1].isnan().all()) and bool((out[0, 7] == float("inf")).all()) and float(out[0, 150]) == 0.0
    keep = [n for n in range(N) if n not in (7, 150)]
    rest = [m for m in range(M) if m != 1]
    assert bool(out[rest][:, keep].isfinite().all())


def test_gemm_beyond_32_bit_offsets():
    """Codes of 4.3 GB and an output of more than 2^31 bytes' offset: the
    last rows are checked against the same rows multiplied by themselves."""
    M, N, K, pitch = 140_000, 40, 128, 32_768
    big = torch.zeros((M, pitch), dtype=torch.int8, device=DEV)
    xq = big[:, :K]
    xq[-300:] = codes(300, K, 5)
    wq, xs, ws = codes(N, K, 6), scales(M, 7), scales(N, 8)
    store = torch.empty((M, 16_384), dtype=BF16, device=DEV)
    out = mmq.gemm_i8(xq, xs, wq, ws, out=store[:, :N])
    check(out[-300:], exact_sum(xq[-300:], wq), xs[-300:], ws, None, BF16)
    assert bool((out[:-300] == 0).all())


def kernel_of(M, N, K, E=0):
    ok, desc = mmq.plan_i8(M, N, K, E, torch.cuda.get_device_properties(0).multi_processor_count)
    assert ok, desc
    return desc.split(" threads")[0]


# last k-steps of every length behind a long K (a step's offset then passes
# the distance by which "nowhere" lies past a buffer's end), with the kernel
# that runs each
TAILS = [(300, 4000, 3600), (600, 1500, 2064), (700, 2100, 2096), (900, 3000, 4112), (1500, 2500, 3264), (2000, 3000, 2160),
         (2500, 4000, 3504), (4000, 4100, 2064), (5000, 9000, 2128), (40, 600, 5008), (100, 2000, 4144), (200, 2000, 2192)]


def test_gemm_long_k_tails_on_every_kernel():
    seen = set()
    for M, N, K in TAILS:
        seen.add(kernel_of(M, N, K))
        xq, wq, xs, ws = codes(M, K, M), codes(N, K, N), scales(M, 2), scales(N, 3)
        out = mmq.gemm_i8(xq, xs, wq, ws)
        acc = torch.matmul(xq.double(), wq.double().t())          # integers below 2^53: exact on the GPU as well
        assert torch.equal(out, acc.float() * xs[:, None] * ws), (M, N, K)
    for tile in ("256x256", "128x256", "128x128", "64x128"):
        assert f"kernel=tile tile={tile}" in seen, seen
    for tile in ("32x32", "32x64", "64x64"):
        assert f"kernel=rows tile={tile}" in seen, seen


# ---------------------------------------------------------------------------
# grouped products
# ---------------------------------------------------------------------------
def offsets_of(lengths, first=0):
    return torch.tensor([first] + list(first + np.cumsum(lengths)), dtype=torch.int32)


def check_grouped(out, xq, xs, wq, ws, off, rows, dtype, fill):
    off = off.tolist()
    R = out.shape[0]
    T = xq.shape[0]
    out, xq, xs, wq, ws = out.cpu(), xq.cpu(), xs.cpu(), wq.cpu(), ws.cpu()
    rows = torch.arange(R) if rows is None else rows.cpu().long()
    written = torch.zeros(R, dtype=torch.bool)
    for e in range(len(off) - 1):
        r = torch.arange(off[e], off[e + 1])
        if len(r):
            r = r[(rows[r] >= 0) & (rows[r] < T)]
        if not len(r):
            continue
        written[r] = True
        t = rows[r]
        check(out[r], exact_sum(xq[t], wq[e]), xs[t], ws[e], None, dtype)
    assert bool((out[~written] == fill).all())


GROUPS = [
    ("one expert", [37], 0, 0), ("all in the last", [0, 0, 0, 150], 0, 0), ("all in the first", [300, 0, 0], 0, 0),
    ("nothing", [0, 0, 0], 0, 5), ("single rows", [1] * 9, 0, 0), ("ragged", [3, 0, 129, 64, 1, 0, 257, 31, 16, 128], 0, 0),
    ("rows before and behind", [5, 0, 70, 2], 11, 19), ("decode", [1, 0, 0, 2, 0, 1, 3, 0, 1, 0, 0, 0, 8], 0, 0),
    ("many experts", [(i * 7) % 5 for i in range(300)], 0, 3), ("2048 experts", [int(i % 41 == 0) * 3 for i in range(2048)], 2, 0),
    ("one long", [2, 900, 0, 3], 0, 0), ("multiples", [128, 256, 64, 0, 128], 0, 0),
    ("past 64", [0] * 63 + [5, 6, 0, 40] + [0] * 60 + [17], 0, 0),
]


@pytest.mark.parametrize("gather", [False, True], ids=["inplace", "gather"])
@pytest.mark.parametrize("name,lengths,first,behind", GROUPS, ids=[g[0].replace(" ", "_") for g in GROUPS])
@pytest.mark.parametrize("N,K", [(48, 80), (197, 272)])
def test_grouped(name, lengths, first, behind, gather, N, K):
    E, R = len(lengths), first + sum(lengths) + behind
    dtype = TYPES[(E + N + R) % 3]
    T = max(1, R // 3) if gather else R
    off = offsets_of(lengths, first)
    xq, xs = codes(T, K, R), scales(T, 1)
    wq = codes(E * N, K, E).view(E, N, K)
    ws = scales(E * N, 2).view(E, N)
    rows = torch.randint(0, T, (R,), generator=gen(R + 3), dtype=torch.int32) if gather else None
    out = torch.full((R, N), -5.0, dtype=dtype, device=DEV)
    mmq.grouped_gemm_i8(xq, xs, wq, ws, off.to(DEV), rows=None if rows is None else rows.to(DEV), out=out)
    check_grouped(out, xq, xs, wq, ws, off, rows, dtype, -5.0)


# (lengths, first, behind, N, K): groups whose sizes and number make the planner take tiles
TILED = [([700, 0, 300, 1, 0, 900, 130, 64], 3, 9, 2100, 208), ([1] * 200 + [4000] + [0] * 50 + [257], 0, 40, 1030, 400),
         ([(i * 37) % 23 for i in range(2048)], 5, 0, 130, 80), ([0] * 1024 + [9000] + [0] * 1000 + [77], 0, 0, 520, 2064),
         ([128] * 64, 0, 0, 1536, 512), ([5000], 0, 3, 4000, 96), ([3000, 5000, 2, 4000], 0, 0, 5000, 144),
         ([600 + 40 * i for i in range(17)], 0, 0, 2048, 160)]


@pytest.mark.parametrize("gather", [False, True], ids=["inplace", "gather"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_grouped_tiles(gather, dtype):
    seen = set()
    for lengths, first, behind, N, K in TILED:
        E, R = len(lengths), first + sum(lengths) + behind
        seen.add(kernel_of(R, N, K, E))
        T = R // 5 if gather else R
        off = offsets_of(lengths, first)
        xq, xs, wq, ws = codes(T, K, R), scales(T, 1), codes(E * N, K, E).view(E, N, K), scales(E * N, 2).view(E, N)
        rows = torch.randint(0, T, (R,), generator=gen(R), dtype=torch.int32) if gather else None
        if gather:
            rows[first + 1], rows[R // 2] = -7, T
        out = torch.full((R, N), -5.0, dtype=dtype, device=DEV)
        mmq.grouped_gemm_i8(xq, xs, wq, ws, off.to(DEV), rows=None if rows is None else rows.to(DEV), out=out)
        src = torch.arange(R, device=DEV) if rows is None else rows.to(DEV).long()
        want = torch.full((R, N), -5.0, dtype=dtype, device=DEV)
        for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
            if b > a:
                t = src[a:b].clamp(0, T - 1)
                y = torch.matmul(xq[t].double(), wq[e].double().t()).float() * xs[t][:, None] * ws[e]
                good = (src[a:b] >= 0) & (src[a:b] < T)
                want[a:b] = torch.where(good[:, None], y.to(dtype), want[a:b])
        assert torch.equal(out, want), (lengths[:8], E, N, K)
    for tile in ("256x256", "128x256", "128x128", "64x128"):
        assert f"kernel=tile tile={tile}" in seen, seen


@pytest.mark.parametrize("seed", range(6))
def test_grouped_tiles_bad_offsets_stay_within_the_buffers(seed):
    """Offsets in any order and far out of range, on the tile kernels: what is
    around the output stays as it was."""
    E, R, N, K = 40, 9000, 1100, 96
    off = torch.randint(-2 ** 31, 2 ** 31 - 1, (E + 1,), generator=gen(seed)) if seed % 2 else torch.randint(-500, R + 500, (E + 1,), generator=gen(seed))
    assert "kernel=tile" in kernel_of(R, N, K, E)
    xq, xs, wq, ws = codes(R, K, 1), scales(R, 2), codes(E * N, K, 3).view(E, N, K), scales(E * N, 4).view(E, N)
    store = torch.full((R + 600, N), 3.0, dtype=BF16, device=DEV)
    mmq.grouped_gemm_i8(xq, xs, wq, ws, off.to(torch.int32).to(DEV), out=store[300:300 + R])
    assert bool((store[:300] == 3.0).all()) and bool((store[300 + R:] == 3.0).all())


@pytest.mark.parametrize("lengths", [[4, 9, 3], [40, 150, 30]], ids=["few", "many"])
def test_grouped_skips_rows_whose_index_is_out_of_range(lengths):
    R, T, N, K = sum(lengths), 6, 65, 96
    rows = torch.arange(R, dtype=torch.int32) % T
    rows[3], rows[7], rows[R - 1] = -1, T, 2 ** 31 - 1
    off = offsets_of(lengths)
    xq, xs, wq, ws = codes(T, K, 1), scales(T, 2), codes(3 * N, K, 3).view(3, N, K), scales(3 * N, 4).view(3, N)
    out = torch.full((R, N), 9.0, dtype=F32, device=DEV)
    mmq.grouped_gemm_i8(xq, xs, wq, ws, off.to(DEV), rows=rows.to(DEV), out=out)
    check_grouped(out, xq, xs, wq, ws, off, rows, F32, 9.0)


@pytest.mark.parametrize("off", [[-5, 3, 40, 10 ** 6], [7, 2, 9, 30], [0, 50, 10, 20]], ids=["clamped", "decreasing", "overlap"])
def test_grouped_bad_offsets_stay_within_the_buffers(off):
    """Guard rows around the output stay as they were, whatever the offsets
    say (the kernel clamps them to 0..R before it forms an address)."""
    R, N, K = 40, 70, 64
    xq, xs, wq, ws = codes(R, K, 1), scales(R, 2), codes(3 * N, K, 3).view(3, N, K), scales(3 * N, 4).view(3, N)
    store = torch.full((R + 200, N), 3.0, dtype=F32, device=DEV)
    out = store[100:100 + R]
    mmq.grouped_gemm_i8(xq, xs, wq, ws, torch.tensor(off, dtype=torch.int32, device=DEV), out=out)
    assert bool((store[:100] == 3.0).all()) and bool((store[100 + R:] == 3.0).all())
    if off[0] == -5:     # clamped to 0, 3, 40, 40: a good grouping
        check_grouped(out, xq, xs, wq, ws, torch.tensor([0, 3, 40, 40]), None, F32, 3.0)


def test_grouped_rows_with_pitches_and_odd_output():
    lengths, N, K = [6, 0, 140, 33], 75, 112
    R = sum(lengths)
    off = offsets_of(lengths)
    xq, xs = codes(R, K, 1, pitch=320), scales(R, 2)
    wq, ws = codes(4 * N, K, 3).view(4, N, K), scales(4 * N, 4).view(4, N)
    store = torch.full((R, N + 6), 2.0, dtype=BF16, device=DEV)
    mmq.grouped_gemm_i8(xq, xs, wq, ws, off.to(DEV), out=store[:, 3:3 + N])
    check_grouped(store[:, 3:3 + N], xq, xs, wq, ws, off, None, BF16, 2.0)
    assert bool((store[:, :3] == 2.0).all()) and bool((store[:, 3 + N:] == 2.0).all())


def test_grouped_equals_dense_bit_for_bit():
    lengths, N, K = [130, 5, 0, 400], 384, 768
    off = offsets_of(lengths).tolist()
    R = sum(lengths)
    xq, xs, wq, ws = codes(R, K, 1), scales(R, 2), codes(4 * N, K, 3).view(4, N, K), scales(4 * N, 4).view(4, N)
    out = mmq.grouped_gemm_i8(xq, xs, wq, ws, torch.tensor(off, dtype=torch.int32, device=DEV), dtype=BF16)
    for e in range(4):
        a, b = off[e], off[e + 1]
        if b > a:
            assert torch.equal(out[a:b], mmq.gemm_i8(xq[a:b], xs[a:b], wq[e], ws[e], dtype=BF16))


@pytest.mark.parametrize("R", [40, 5000])
def test_grouped_weights_beyond_4_gib(R):
    """Experts whose matrices lie past 2^32 bytes, on the rows and the tile kernel."""
    E, N, K = 300, 4096, 4096
    wq = torch.zeros((E, N, K), dtype=torch.int8, device=DEV)
    ws = torch.ones((E, N), device=DEV)
    for e in (0, E - 1):
        wq[e], ws[e] = codes(N, K, e), scales(N, e + 1)
    off = torch.full((E + 1,), R // 2, dtype=torch.int32, device=DEV)
    off[0], off[E] = 0, R
    assert ("rows" if R == 40 else "tile") in kernel_of(R, N, K, E)
    xq, xs = codes(R, K, 1), scales(R, 2)
    out = mmq.grouped_gemm_i8(xq, xs, wq, ws, off)
    for e, a, b in ((0, 0, R // 2), (E - 1, R // 2, R)):
        acc = torch.matmul(xq[a:b].double(), wq[e].double().t())
        assert torch.equal(out[a:b], acc.float() * xs[a:b, None] * ws[e])


# ---------------------------------------------------------------------------
# row quantizers
# ---------------------------------------------------------------------------
def exact_quantize(v32):
    """Codes and scales from fp32 values, every rounding of the definition made once from 64 bits."""
    v = v32.double()
    d = (v.abs().amax(1) / 127).float().double()
    inv = torch.where(d > 0, 1 / d, torch.zeros_like(d)).float().double()
    inv[inv.isinf()] = 0.0
    y = (v * inv[:, None]).float().double()
    q = torch.where(y < 0, torch.ceil(y - 0.5), torch.floor(y + 0.5)).clamp(-127, 127)
    return q.to(torch.int8), d.float()


ROWS = [(1, 1), (1, 16), (3, 15), (2, 17), (1, 3584), (5, 100), (4, 255), (3, 256), (2, 1000), (3, 1024), (2, 2047), (7, 2048),
        (64, 768), (2, 4096), (3, 4097), (2, 8191), (2, 18944), (1, 32768), (2, 32783), (1, 65536), (1, 131056), (300, 512)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", ROWS)
def test_quantize(M, K, dtype):
    x = (torch.randn((M, K), generator=gen(M * 7 + K)) * 3).to(dtype)
    q, s = mmq.quantize_i8(x.to(DEV))
    Kp = -(-K // 16) * 16
    assert q.shape == (M, Kp) and s.shape == (M,)
    wq, ws = exact_quantize(x.float())
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(q.cpu()[:, :K], wq) and bool((q[:, K:] == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K,px,first,pq", [(40, 41, 1, 64), (100, 333, 3, 128), (256, 264, 8, 272), (3000, 3001, 0, 3024),
                                           (5000, 5010, 2, 8192)])
def test_quantize_pitches_and_alignment(K, px, first, pq, dtype):
    M = 5
    full = torch.randn((M, px + first), generator=gen(K)).to(dtype).to(DEV)
    x = full[:, first:first + K]
    store = torch.full((M, pq), 99, dtype=torch.int8, device=DEV)
    Kp = -(-K // 16) * 16
    q, s = mmq.quantize_i8(x, q=store[:, :Kp])
    wq, ws = exact_quantize(x.cpu().float())
    assert torch.equal(s.cpu(), ws) and torch.equal(q.cpu()[:, :K], wq)
    assert bool((q[:, K:] == 0).all()) and bool((store[:, Kp:] == 99).all())


def test_quantize_special_rows():
    """Zero rows, rows whose reciprocal scale overflows, ties, the largest
    finite values, and rows with an infinity or NaN."""
    K = 300
    x = torch.zeros((9, K))
    x[1, 5] = 1e-38                                       # d is denormal, 1/d overflows: all codes 0
    x[2] = torch.randn(K, generator=gen(1)) * 1e37
    x[3, :4] = torch.tensor([127.0, 0.5, -1.5, 2.5])      # d = 1: exact ties go away from zero
    x[4, 0], x[4, 299] = 3.4e38, -3.4e38
    x[5, 7] = float("nan")
    x[6, 0], x[6, 1] = float("inf"), 1.0
    x[7, 299] = float("-inf")
    x[8] = -2.0
    q, s = mmq.quantize_i8(x.to(DEV))
    q, s = q.cpu(), s.cpu()
    good = [0, 1, 2, 3, 4, 8]
    wq, ws = exact_quantize(x[good])
    assert torch.equal(q[good][:, :K], wq) and torch.equal(s[good], ws)
    assert q[3, :4].tolist() == [127, 1, -2, 3] and bool((q[8, :K] == -127).all()) and bool((q[1] == 0).all())
    assert bool(s[[5, 6, 7]].isnan().all()) and bool((q[[5, 6, 7]] == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", ROWS)
def test_silu_mul_quantize(M, K, dtype):
    """h = silu(g) * u in fp32: exp within an ulp (2 u), the sum 1 + e, the
    quotient and the product within u each, so h is within 5 u |h|, doubled
    below for the products of those; the scale takes u more.  A code is then
    within half a step of h / d, plus 127 times the relative errors of h, d
    and 1/d (12 + 2 + 2 u at most)."""
    gu = (torch.randn((M, 2 * K), generator=gen(M + 3 * K)) * 2).to(dtype)
    t = gu.to(DEV)
    q, s = mmq.silu_mul_quantize_i8(t[:, :K], t[:, K:])
    g, u = gu[:, :K].double(), gu[:, K:].double()
    h = g / (1 + torch.exp(-g)) * u
    d = h.abs().amax(1) / 127
    assert bool(((s.cpu().double() - d).abs() <= 11 * U * d).all())
    step = s.cpu().double()[:, None]
    err = (q.cpu()[:, :K].double() * step - h).abs()
    assert bool((err <= step * (0.5 + 127 * 16 * U)).all())
    assert bool((q[:, K:] == 0).all())


def test_quantize_beyond_32_bit_offsets():
    """2.3 * 10^9 values: the last rows like the same rows alone."""
    M, K = 70_001, 32_768
    x = torch.zeros((M, K), dtype=BF16, device=DEV)
    x[-3:] = torch.randn((3, K), generator=gen(1)).to(BF16).to(DEV)
    q, s = mmq.quantize_i8(x)
    wq, ws = mmq.quantize_i8(x[-3:].clone())
    assert torch.equal(q[-3:], wq) and torch.equal(s[-3:], ws) and bool(ws.gt(0).all())
    assert bool((s[:-3] == 0).all()) and bool((q[:-3] == 0).all())


def test_silu_mul_special_rows():
    K = 40
    g, u = torch.randn((6, K), generator=gen(1)), torch.randn((6, K), generator=gen(2))
    g[0] = -200.0                 # exp overflows: silu is -0
    g[1, 3] = 1000.0              # silu(g) = g
    g[2, 1] = float("nan")
    u[3, 2] = float("inf")
    g[4, 39] = float("-inf")      # -inf / inf: NaN
    g[5] = 0.0
    q, s = mmq.silu_mul_quantize_i8(g.to(DEV), u.to(DEV))
    q, s = q.cpu(), s.cpu()
    assert float(s[0]) == 0.0 and float(s[5]) == 0.0 and bool((q[[0, 2, 3, 4, 5]] == 0).all())
    assert bool(s[2:5].isnan().all())
    assert abs(float(s[1]) - max(abs(1000.0 * float(u[1, 3])), 0) / 127) <= 11 * U * float(s[1]) or q[1].abs().max() == 127


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def moe_layer(x, w1, s1, w2, s2, ids, out=None):
    """A token's experts: quantize, gate/up by expert, silu * up, down by expert."""
    E, topk = w1.shape[0], ids.shape[1]
    order = torch.sort(ids.reshape(-1), stable=True).indices
    off = torch.zeros(E + 1, dtype=torch.int32, device=x.device)
    off[1:] = torch.bincount(ids.reshape(-1), minlength=E).cumsum(0)
    rows = (order // topk).to(torch.int32)
    return off, rows, run_layer(x, w1, s1, w2, s2, off, rows, out)


def run_layer(x, w1, s1, w2, s2, off, rows, out=None):
    F = w2.shape[2]
    xq, xs = mmq.quantize_i8(x)
    gu = mmq.grouped_gemm_i8(xq, xs, w1, s1, off, rows=rows, dtype=BF16)
    hq, hs = mmq.silu_mul_quantize_i8(gu[:, :F], gu[:, F:])
    return mmq.grouped_gemm_i8(hq, hs, w2, s2, off, dtype=BF16, out=out)


@pytest.mark.parametrize("T", [1, 5, 70, 600])
def test_expert_layer_end_to_end(T):
    """The four operators in a row, each stage against 64 bits on the codes
    the stage before it made, and the layer captured in a graph and replayed
    with new inputs against the eager calls, bit for bit."""
    E, topk, H, F = 16, 4, 256, 192
    x = torch.randn((T, H), generator=gen(T)).to(BF16).to(DEV)
    w1, s1 = mmq.quantize_i8((0.1 * torch.randn((E * 2 * F, H), generator=gen(1))).to(DEV))
    w2, s2 = mmq.quantize_i8((0.1 * torch.randn((E * H, F), generator=gen(2))).to(DEV))
    w1, s1, w2, s2 = w1.view(E, 2 * F, H), s1.view(E, 2 * F), w2.view(E, H, F), s2.view(E, H)
    ids = torch.stack([torch.randperm(E, generator=gen(100 + t))[:topk] for t in range(T)]).to(DEV)
    off, rows, y = moe_layer(x, w1, s1, w2, s2, ids)
    xq, xs = mmq.quantize_i8(x)
    wq, ws = exact_quantize(x.float().cpu())
    assert torch.equal(xq.cpu(), wq) and torch.equal(xs.cpu(), ws)
    gu = mmq.grouped_gemm_i8(xq, xs, w1, s1, off, rows=rows, dtype=BF16)
    check_grouped(gu, xq, xs, w1, s1, off.cpu(), rows, BF16, 0.0)
    hq, hs = mmq.silu_mul_quantize_i8(gu[:, :F], gu[:, F:])
    check_grouped(y, hq, hs, w2, s2, off.cpu(), None, BF16, 0.0)

    static = x.clone()
    out = torch.zeros_like(y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_layer(static, w1, s1, w2, s2, off, rows, out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run_layer(static, w1, s1, w2, s2, off, rows, out)
    for i in range(4):
        new = torch.randn((T, H), generator=gen(50 + i)).to(BF16).to(DEV)
        static.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run_layer(new, w1, s1, w2, s2, off, rows)), i


def test_two_streams_at_once():
    """Calls that overlap in time share nothing: no workspace, no state."""
    M, N, K = 200, 600, 1024
    ins = [(codes(M, K, i), scales(M, i), codes(N, K, 9 + i), scales(N, 9 + i)) for i in range(2)]
    want = [mmq.gemm_i8(*t) for t in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(want[0]) for _ in range(20)] for _ in range(2)]
    for j in range(20):
        for i in range(2):
            mmq.gemm_i8(*ins[i], out=outs[i][j], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_inputs_of_a_call_on_another_stream_are_kept_until_it_ran():
    """The call waits on its stream behind a long product; its inputs are
    dropped at once and their memory is written by the current stream."""
    M, N, K = 300, 500, 4096
    wq, ws = codes(N, K, 1), scales(N, 2)
    side = torch.cuda.Stream()
    big = torch.randn((8192, 8192), device=DEV)
    xq, xs = codes(M, K, 3), scales(M, 4)
    want = mmq.gemm_i8(xq, xs, wq, ws)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(4):
            big @ big
    out = mmq.gemm_i8(xq, xs, wq, ws, stream=side)
    del xq, xs
    junk = [torch.full((M, K), 1, dtype=torch.int8, device=DEV) for _ in range(4)] + [torch.zeros(M, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and len(junk) == 8


def test_tensors_of_a_gpu_that_is_not_current(monkeypatch):
    """Each call makes the tensors' GPU current for itself (here the first
    answer of the device query is another one)."""
    c = mmq._c()
    real, entered = c.current_device, []
    device = c.device

    def make_current(dev):
        entered.append(dev)
        return device(dev)

    xq, xs, wq, ws = codes(5, 64, 1), scales(5, 2), codes(9, 64, 3), scales(9, 4)
    x = torch.randn((5, 64), device=DEV)
    off = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    calls = [lambda: mmq.gemm_i8(xq, xs, wq, ws), lambda: mmq.quantize_i8(x)[0], lambda: mmq.silu_mul_quantize_i8(x, x)[0],
             lambda: mmq.grouped_gemm_i8(xq, xs, wq[None], ws[None], off)]
    for f in calls:
        want = f()
        answers = iter([real() + 1])
        monkeypatch.setattr(c, "current_device", lambda: next(answers, real()))
        monkeypatch.setattr(c, "device", make_current)
        assert torch.equal(f(), want) and entered.pop() == xq.device
        monkeypatch.undo()


def test_no_rows():
    z = torch.empty((0, 64), dtype=BF16, device=DEV)
    q, s = mmq.quantize_i8(z)
    assert q.shape == (0, 64) and s.shape == (0,)
    wq, ws = codes(10, 64, 1), scales(10, 2)
    assert mmq.gemm_i8(q, s, wq, ws).shape == (0, 10)
    off = torch.zeros(2, dtype=torch.int32, device=DEV)
    assert mmq.grouped_gemm_i8(q, s, wq[None], ws[None], off).shape == (0, 10)


def test_binding_refuses_what_does_not_fit():
    xq, xs, wq, ws = codes(4, 64, 1), scales(4, 2), codes(8, 64, 3), scales(8, 4)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    bad = [
        lambda: mmq.gemm_i8(xq, xs[:3], wq, ws), lambda: mmq.gemm_i8(xq, xs, wq, ws[:7]),
        lambda: mmq.gemm_i8(xq, xs, codes(8, 48, 1), ws), lambda: mmq.gemm_i8(xq.float(), xs, wq, ws),
        lambda: mmq.gemm_i8(xq.cpu(), xs, wq, ws), lambda: mmq.gemm_i8(xq, xs.cpu(), wq, ws),
        lambda: mmq.gemm_i8(xq, xs, wq.cpu(), ws), lambda: mmq.gemm_i8(xq, xs.double(), wq, ws),
        lambda: mmq.gemm_i8(xq, xs, wq, ws, bias=ws[:4]), lambda: mmq.gemm_i8(xq, xs, wq, ws, dtype=torch.float64),
        lambda: mmq.gemm_i8(xq, xs, wq, ws, out=torch.empty((4, 9), device=DEV)),
        lambda: mmq.gemm_i8(xq, xs, wq, ws, dtype=BF16, out=torch.empty((4, 8), device=DEV)),
        lambda: mmq.gemm_i8(xq, xs, wq, ws, out=torch.empty((8, 4), device=DEV).t()),
        lambda: mmq.gemm_i8(xq.t(), xs, wq, ws), lambda: mmq.gemm_i8(xq[:1].expand(4, 64), xs, wq, ws),
        lambda: mmq.gemm_i8(xq, scales(8, 1)[::2], wq, ws),
        lambda: mmq.quantize_i8(xq), lambda: mmq.quantize_i8(xs), lambda: mmq.quantize_i8(torch.zeros((2, 64))),
        lambda: mmq.quantize_i8(torch.zeros((2, 64), device=DEV), q=xq),
        lambda: mmq.quantize_i8(torch.zeros((4, 64), device=DEV), scale=xs[:3]),
        lambda: mmq.silu_mul_quantize_i8(torch.zeros((2, 64), device=DEV), torch.zeros((2, 32), device=DEV)),
        lambda: mmq.silu_mul_quantize_i8(torch.zeros((2, 64), device=DEV), torch.zeros((2, 128), device=DEV)[:, :64]),
        lambda: mmq.silu_mul_quantize_i8(torch.zeros((2, 64), device=DEV), torch.zeros((2, 64), device=DEV, dtype=BF16)),
        lambda: mmq.grouped_gemm_i8(xq, xs, wq, ws, off), lambda: mmq.grouped_gemm_i8(xq, xs, wq[None], ws, off),
        lambda: mmq.grouped_gemm_i8(xq, xs, wq[None], ws[None], off.long()),
        lambda: mmq.grouped_gemm_i8(xq, xs, wq[None], ws[None], off[:1]),
        lambda: mmq.grouped_gemm_i8(xq, xs, wq[None], ws[None], off, rows=torch.zeros(3, dtype=torch.int64, device=DEV)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(mmq.MMQError):
        mmq.gemm_i8(codes(4, 40, 1), xs, codes(8, 40, 2), ws)
