"""silu(gate) * up of the per-token int8 form over the whole range of finite
gates, against 64 bits.

Bounds.  u = 2^-24.  A value h = silu(g) * up is within 10 u |h| of the exact
one (the exponential within 2 u, the sum, the quotient and the product u each,
doubled for the products of those); where silu(g) itself is subnormal its
rounding, 2^-150, adds up to 2^-149 |up|, doubled likewise.  A row's scale
takes u more for the division by 127.  A code is within half a step of h / d,
plus 127 times the relative errors of h, d and 1 / d."""
import pytest
import torch

import block_quantized_int8_q8_amd as mmq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24


def check(g, u):
    """Quantize silu(g) * u of the CPU tensors on the GPU and compare."""
    K = g.shape[1]
    q, s = mmq.silu_mul_quantize_i8(g.to(DEV), u.to(DEV))
    q, s = q.cpu(), s.cpu().double()
    g, u = g.double(), u.double()
    h = g * torch.sigmoid(g) * u
    tiny = 2.0 ** -149 * u.abs()
    d = h.abs().amax(1) / 127
    assert bool(s.isfinite().all()), s
    assert bool(((s - d).abs() <= 11 * U * d + tiny.amax(1) / 127).all()), (s, d)
    err = (q[:, :K].double() * s[:, None] - h).abs()
    assert bool((err <= s[:, None] * (0.5 + 127 * 16 * U) + tiny).all())
    assert bool((q[:, K:] == 0).all())


@pytest.mark.parametrize("K", [24, 2100, 9000])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_largest_finite_gates(K, dtype):
    """The largest and lowest finite gates beside ordinary ones: silu(g) is g,
    or -0 (the lowest value is what masks are filled with)."""
    big = torch.finfo(dtype).max
    small = 2.0 ** (-14 if dtype == F16 else -126)
    rows = [(s * f * big, up) for s in (1, -1) for f in (1.0, 0.875, 0.703125, 0.5) for up in (0.25, -0.5, small)]
    gen = torch.Generator().manual_seed(K)
    g, u = torch.randn((len(rows), K), generator=gen).to(dtype), torch.randn((len(rows), K), generator=gen).to(dtype)
    for i, (gate, up) in enumerate(rows):
        at = (5 * i) % K
        g[i, at], u[i, at] = gate, up
    g[-1], u[-1] = -big, 1.0
    g[-1, K // 2] = 1.5
    assert bool(g.isfinite().all()) and bool(u.isfinite().all())
    check(g, u)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_a_value_does_not_depend_on_its_neighbours(dtype):
    """The same gate and up beside zeros, and beside gates of every size: the
    value that sets the scale has the same bits."""
    M, K = 4096, 16
    gen = torch.Generator().manual_seed(3)
    g, u = torch.zeros((M, K)), torch.full((M, K), 2.0 ** -20)
    g[:, 3] = torch.rand(M, generator=gen) * 140 - (70 if dtype != F16 else 10)
    u[:, 3] = 1 + torch.rand(M, generator=gen)
    g, u = g.to(dtype), u.to(dtype)
    want = mmq.silu_mul_quantize_i8(g.to(DEV), u.to(DEV))[1]
    assert bool(want.gt(0).all())
    for gate in (-90.0, -1000.0, float(torch.finfo(dtype).min)):
        g[:, 6] = gate
        assert torch.equal(mmq.silu_mul_quantize_i8(g.to(DEV), u.to(DEV))[1], want), gate


# (gates lo..hi, |up| to): exp(-gate) nears the largest number, and the result is what is small
FAR = [(-80.0, -86.5, 2.0 ** 40), (-85.5, -89.0, 2.0 ** 60), (-87.0, -97.0, 2.0 ** 100), (-95.0, -104.0, 2.0 ** 120),
       (-86.0, -103.0, 2.0 ** 127)]


@pytest.mark.parametrize("among", ["alone", "ordinary", "large"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lo,hi,top", FAR)
def test_far_negative_gates_with_large_ups(lo, hi, top, dtype, among):
    """Gates whose silu is tiny or subnormal with an up so large that they set
    the scale: every value of the row, or one to three of each eight beside
    ordinary or large positive gates."""
    M, K = 64, 72
    if dtype == F16:
        top = 2.0 ** 15
        hi = max(hi, -96.0)
    gen = torch.Generator().manual_seed(int(-10 * hi))
    far = lo + (hi - lo) * torch.rand((M, K), generator=gen)
    big = top * (1 + torch.rand((M, K), generator=gen)) / 2 * torch.where(torch.rand((M, K), generator=gen) < 0.5, -1.0, 1.0)
    if among == "alone":
        g, u = far, big
    else:
        here = (torch.arange(K) % 8)[None, :] < torch.randint(1, 4, (M, 1), generator=gen)
        near = torch.randn((M, K), generator=gen) * 2 if among == "ordinary" else 50 + 50 * torch.rand((M, K), generator=gen)
        # so small that the far gates' values set the scale, about half of the time
        least = 100 * float(torch.exp(torch.tensor(hi, dtype=torch.float64))) * top / 100
        small = least * torch.exp(4 * torch.randn((M, K), generator=gen))
        g, u = torch.where(here, far, near), torch.where(here, big, small)
    check(g.to(dtype), u.to(dtype))


def test_a_large_gate_sets_the_scale():
    """silu(1000) = 1000 beside ordinary gates: scale and codes of the row."""
    gen = torch.Generator().manual_seed(1)
    g, u = torch.randn((3, 40), generator=gen), torch.randn((3, 40), generator=gen)
    g[0, 3], g[1, 0], g[2, 39] = 1000.0, 87.0, -87.0
    check(g, u)
    s = mmq.silu_mul_quantize_i8(g.to(DEV), u.to(DEV))[1]
    want = 1000.0 * float(u[0, 3].abs()) / 127
    assert abs(float(s[0]) - want) <= 4 * U * want
