"""Every kernel of the per-token int8 products, with every output type, with
and without a bias, dense and grouped.  The planner's choice is asserted, so
that a kernel whose shape moves to another one is missed here, not silently.
The sum is exact and the roundings after it are fixed, so results are
compared bit for bit with the definition's fp32 arithmetic on the exact sum
(a product of integers in 64 bits)."""
import re

import pytest
import torch

import block_quantized_int8_q8_amd as mmq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]

# kernel, M, N: columns that end inside a tile, and tiles for more than one round of workgroups
DENSE = [("rows 16x16", 13, 67), ("rows 16x32", 20, 4110), ("rows 32x32", 33, 4110), ("rows 32x64", 130, 3050),
         ("rows 64x64", 300, 3050), ("tile 64x128", 33100, 70), ("tile 128x128", 8300, 2070), ("tile 128x256", 8300, 2690),
         ("tile 256x256", 6000, 4110)]
# kernel, routed rows, N, experts
GROUPED = [("rows 16x16", 60, 70, 5), ("rows 16x32", 60, 1100, 130), ("rows 32x32", 3000, 70, 5), ("rows 32x64", 2000, 197, 3),
           ("rows 64x64", 3400, 197, 3), ("tile 64x128", 1500, 1100, 5), ("tile 128x128", 3000, 2100, 40),
           ("tile 128x256", 5000, 4100, 5), ("tile 256x256", 12000, 4100, 5)]
# kernel, M, N at the longest K
LONGEST = [("rows 16x16", 13, 67), ("rows 16x32", 300, 333), ("rows 32x32", 300, 700), ("rows 32x64", 300, 1450),
           ("rows 64x64", 300, 3050), ("tile 64x128", 1100, 1030), ("tile 128x128", 2100, 1030), ("tile 128x256", 2100, 2070),
           ("tile 256x256", 2100, 4110)]


def planned(kernel, M, N, K, E=0, rounds=False):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    ok, desc = mmq.plan_i8(M, N, K, E, cus)
    assert ok, desc
    f = re.match(r"kernel=(\w+) tile=(\w+) .*tiles=(\d+)x(\d+) workgroups=(\d+)", desc)
    assert f"{f[1]} {f[2]}" == kernel, desc
    assert not rounds or f[1] == "rows" or int(f[3]) * int(f[4]) > int(f[5]), desc


def operands(M, N, K, seed, E=1, px=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    xq = torch.randint(-128, 128, (M, px or K), generator=g, device=DEV, dtype=torch.int8)[:, :K]
    wq = torch.randint(-128, 128, (E, N, K), generator=g, device=DEV, dtype=torch.int8)
    xs = torch.rand(M, generator=g, device=DEV) * 0.01 + 1e-3
    ws = torch.rand((E, N), generator=g, device=DEV) * 0.01 + 1e-3
    return g, xq, xs, wq, ws


def defined(xq, xs, wq, ws, bias, dtype):
    y = torch.matmul(xq.double(), wq.double().t()).float() * xs[:, None] * ws
    return (y if bias is None else y + bias).to(dtype)


@pytest.mark.parametrize("with_bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kernel,M,N", DENSE, ids=[d[0].replace(" ", "_") for d in DENSE])
def test_dense(kernel, M, N, dtype, with_bias):
    K = 208
    planned(kernel, M, N, K, rounds=True)
    g, xq, xs, wq, ws = operands(M, N, K, M)
    bias = torch.randn(N, generator=g, device=DEV) if with_bias else None
    out = mmq.gemm_i8(xq, xs, wq[0], ws[0], bias=bias, dtype=dtype)
    assert torch.equal(out, defined(xq, xs, wq[0], ws[0], bias, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kernel,M,N", DENSE, ids=[d[0].replace(" ", "_") for d in DENSE])
def test_dense_into_a_slice_of_columns(kernel, M, N, dtype):
    """Output rows with a pitch, at an odd element of the storage, and codes
    with a pitch: the columns around the output stay as they were."""
    K = 144
    planned(kernel, M, N, K)
    g, xq, xs, wq, ws = operands(M, N, K, N, px=K + 48)
    bias = torch.randn(N, generator=g, device=DEV)
    pitch = N + 7
    flat = torch.full((M * pitch + 3,), -77.0, dtype=dtype, device=DEV)
    inside = flat[1:1 + M * pitch].view(M, pitch)
    out = inside[:, 3:3 + N]
    mmq.gemm_i8(xq, xs, wq[0], ws[0], bias=bias, out=out)
    assert torch.equal(out, defined(xq, xs, wq[0], ws[0], bias, dtype))
    assert bool((inside[:, :3] == -77.0).all()) and bool((inside[:, 3 + N:] == -77.0).all())
    assert float(flat[0]) == -77.0 and bool((flat[1 + M * pitch:] == -77.0).all())


@pytest.mark.parametrize("kernel,M,N", LONGEST, ids=[d[0].replace(" ", "_") for d in LONGEST])
def test_longest_rows_of_extreme_codes(kernel, M, N):
    """131056 products of -128 * -128 come to 2147221504, the largest sum there is."""
    K = mmq.I8_MAX_K
    planned(kernel, M, N, K)
    xq = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    wq = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    wq[1::2] = 127
    one = torch.ones(max(M, N), device=DEV)
    out = mmq.gemm_i8(xq, one[:M], wq, one[:N])
    even = torch.arange(N, device=DEV) % 2 == 0
    want = torch.where(even, torch.tensor(16384.0 * K, device=DEV), torch.tensor(-128.0 * 127.0 * K, device=DEV))
    assert torch.equal(out, want.expand(M, N))


@pytest.mark.parametrize("gather", [False, True], ids=["inplace", "gather"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kernel,R,N,E", GROUPED, ids=[d[0].replace(" ", "_") for d in GROUPED])
def test_grouped(kernel, R, N, E, dtype, gather):
    K = 208
    planned(kernel, R, N, K, E)
    T = max(1, R // 3) if gather else R
    g, xq, xs, wq, ws = operands(T, N, K, R, E)
    rows = torch.randint(-1, T + 1, (R,), generator=g, device=DEV, dtype=torch.int32) if gather else None
    cuts = torch.randint(2, R - 1, (E - 1,), generator=g, device=DEV).sort().values.tolist()
    off = [2] + cuts + [R - 1]                              # two rows before the groups and one behind them
    out = torch.full((R, N), -5.0, dtype=dtype, device=DEV)
    want = out.clone()
    mmq.grouped_gemm_i8(xq, xs, wq, ws, torch.tensor(off, dtype=torch.int32, device=DEV), rows=rows, out=out)
    src = torch.arange(R, device=DEV) if rows is None else rows.long()
    for e, (a, b) in enumerate(zip(off, off[1:])):
        r = torch.arange(a, b, device=DEV)
        r = r[(src[r] >= 0) & (src[r] < T)]
        want[r] = defined(xq[src[r]], xs[src[r]], wq[e], ws[e], None, dtype)
    assert torch.equal(out, want)


@pytest.mark.parametrize("K", [3, 2049])
def test_quantizers_of_more_rows_than_one_launch_holds(K):
    """Rows 2^21 and on are another launch's: the last rows, and those around
    the border, like the same rows alone; no row is left out."""
    M = (1 << 21) + 5
    x = torch.full((M, K), 0.5, dtype=torch.bfloat16, device=DEV)
    picks = torch.tensor([0, (1 << 21) - 1, 1 << 21, M - 1], device=DEV)
    x[picks] = torch.randn((4, K), generator=torch.Generator(device=DEV).manual_seed(K), device=DEV).to(torch.bfloat16)
    rest = torch.ones(M, dtype=torch.bool, device=DEV)
    rest[picks] = False
    for call in (mmq.quantize_i8, lambda t: mmq.silu_mul_quantize_i8(t, t)):
        q, s = call(x)
        want, scale = call(x[picks])
        assert torch.equal(q[picks], want) and torch.equal(s[picks], scale)
        want, scale = call(x[1:2])
        assert bool((s[rest] == scale).all()) and bool((q[:, :K].amin(1)[rest] == 127).all())
        assert bool((q[:, K:] == 0).all())
        del q, s, want
