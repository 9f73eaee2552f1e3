"""Attention over values whose sizes differ as much as fp32 allows.

The reference forms every weight w and sum in fp64.  The bound, with u = 2^-24,
h half a step of q's type, N keys, s a value's scale, t scores in units of log2:
  - a score as in tests/test_gpu_attention.py, 2 D u A + 4 u |t| + u max|t|; the
    scale stands in the exponent, t + log2 s, so rounding it, the logarithm, the
    difference to the reference and its halves add 4 u 121 and 80 u at most;
    2^x and the reciprocal of s 4u each, and in the sum 2^-16 beside values past
    2^121, whose terms are subnormal.  Counted twice, for the weights and for
    their sum, which is scaled in two halves where a reference moves and where
    shares meet, 6u each time, counted as 100 u;
  - w s rounds to 16 bits: h of itself (h^2 where it is held in two parts), or in fp16 2^-31 of the row's largest at
    worst, times codes of 127 and N: N 2^-24 of the largest product;
  - a scale counts as 2^-100, or 2^-108 of the largest of its sequence, at least,
    so values are off by 127 times that (zeros are not, their codes are 0);
  - keys whose w s is below 2^-118 of their row's largest may be lost, from the
    sum too;
  - sums over N keys, 3 N u; the quotient and the output's own rounding."""
import math

import pytest
import torch

from tests.test_gpu_attention import BF16, DEV, F16, F32, U, Batch, gen, heads, kvcache

pytestmark = pytest.mark.gpu


def check(bt, out, window=0, every=1, parts=1):
    (kc, kd), (vc, vd) = kvcache.unpack(bt.cache, bt.D)
    h16, i, scale = (torch.finfo(bt.q.dtype).eps / 2) ** parts, 0, bt.D ** -0.5 * math.log2(math.e)
    for b, (n, N) in enumerate(zip(bt.new, bt.lens_h)):
        slot = bt.slots[b].to(DEV)
        pos, key = torch.arange(N - n, N, device=DEV)[:, None], torch.arange(N, device=DEV)[None]
        seen = (key <= pos) & (key > pos - (window or N))
        for head in range(0, bt.q.shape[1], every):
            g = head // bt.G
            c, s, q = kc[slot, g].double(), vd[slot, g].double(), bt.q[i:i + n, head].double()
            f = scale * kd[slot, g].double()
            t, A = (q @ c.t()) * f, (q.abs() @ c.abs().t()) * f
            w = torch.softmax(torch.where(seen, t, -math.inf) * math.log(2), 1)
            least = max(2.0 ** -100, 2.0 ** -108 * float(s.max()))
            V = vc[slot, g].double() * s[:, None]
            want, ws = w @ V, w * s.clamp_min(least)
            top = ws.amax(1, keepdim=True)
            lost = torch.where(ws < 2.0 ** -118 * top, w, 0.0)
            big = torch.where(seen, t.abs(), 0.0).amax(1, keepdim=True)
            e = w * (math.log(2) * U * (2 * bt.D * A + 4 * t.abs() + big + 564) + 8 * U + 2.0 ** -16 * (s.max() > 2.0 ** 114)) + lost
            bound = 2 * (e @ V.abs() + e.sum(1, keepdim=True) * want.abs()) + (h16 + (3 * N + 100) * U) * (w @ V.abs()) \
                + (N + 100) * U * want.abs() + N * 2.0 ** -24 * top + 127 * least
            h = torch.finfo(out.dtype).eps / 2
            bound = bound * (1 + 2 * h) + h * want.abs() + (2.0 ** -25 if out.dtype == F16 else 0.0)
            got = out[i:i + n, head].double()
            off = (got - want).abs()
            assert bool(torch.isfinite(got).all()) and bool((off <= bound).all()), (b, head, float((off / bound).max()))
        i += n


ROWS = [([1], [700]), ([1, 1], [2000, 90]), ([100], [700]), ([300], [300])]


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("large", [1e12, 1e22, 1e30, 2e38])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,lens", ROWS)
def test_rows_of_zeros_beside_large_values(new, lens, D, large, t):
    """All scores alike, and values that are zero or large by turns: the zeros take their half of the weights."""
    def v(total):
        x = heads(total, 2, D, F32, 41).abs().clamp(0.5, 1.0) * large
        x[torch.arange(total, device=DEV) % 2 == 0] = 0.0
        return x
    for far in (False, True):
        def k(total):
            x = torch.zeros((total, 2, D), device=DEV)
            return x if not far else x + (torch.arange(total, device=DEV) > 350)[:, None, None] * 0.5
        bt = Batch(new, lens, 8, 2, D, 16, t, k=k, v=v)
        check(bt, bt.run(dtype=F32))


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("small", [0.0, 1e-37, 1e-32, 1e-24])
@pytest.mark.parametrize("new,Hq,Hkv", [(1, 4, 1), (70, 4, 1), (128, 512, 64)])
def test_many_small_values_ahead_of_ordinary_ones(new, Hq, Hkv, small, t):
    """Ninety thousand keys of next to no value, whose scores lie just below where the reference would move, and
    ordinary values behind them: the sum stays finite, and keeps all of the weights.  (The many heads leave each
    workgroup all of the keys.)"""
    n = 90000

    def k(total):
        x = torch.zeros((total, Hkv, 64), device=DEV)
        x[64:] = 1.0
        return x

    def v(total):
        x = heads(total, Hkv, 64, F32, 42)
        x[:n - 3000] *= small
        return x
    bt = Batch([new], [n], Hq, Hkv, 64, 256, t, k=k, v=v)
    bt.q[:] = 5.19 / 8.0                                             # 5.19 e-folds: 7.49 in units of log2
    check(bt, bt.run(dtype=F32), every=max(Hq // 4 - 1, 1))


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("lo,hi", [(-90, 90), (-60, 120), (-120, 0), (0, 120)])
@pytest.mark.parametrize("new,lens", ROWS + [([3, 60], [5000, 900])])
def test_values_of_any_size(new, lens, lo, hi, t):
    """Every key's values of a size of its own, zeros among them, in no order: under a window some rows see small ones
    only."""
    def v(total):
        e = torch.rand(total, generator=gen(43), device=DEV) * (hi - lo) + lo
        e[torch.rand(total, generator=gen(44), device=DEV) < 0.2] = -200.0
        return torch.exp2(e)[:, None, None] * heads(total, 2, 64, F32, 45).clamp(-3.0, 3.0)

    def k(total):
        return heads(total, 2, 64, F32, 46)
    bt = Batch(new, lens, 8, 2, 64, 16, t, k=k, v=v)
    check(bt, bt.run(dtype=F32))
    check(bt, bt.run(dtype=F32, window=5), window=5)
