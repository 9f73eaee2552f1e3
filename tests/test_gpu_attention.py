"""Attention over the int8 paged cache against the definition in 64 bits.

The reference takes codes and scales from the cache's bytes by the documented
layout and forms every score, weight and sum in fp64.  Caches are filled with
0xff bytes first, so that every slot not written holds codes of -1 and NaN
scales: what is not seen must have no effect.

Tolerance of an output element, with u = 2^-24, h = half a step of q's type,
w_t the exact weights, t = scores in units of log2, A_t = the score's sum of
magnitudes in the same units, N keys:
  - a score: its D products are exact in fp32 (8 by 8 or 11 by 8 bits), each
    addition of the matrix core is taken to cost up to 2u of the magnitudes,
    three scalings u each, the difference to the reference u (|t| + |m|), so
    |dt| <= 2 D u A + 3 u |t| + u (|t| + max|t| + 80); the 80 bounds how far m
    may stand from max t.  exp2 of the hardware: 1 ulp, counted as 4u.
    e_t = ln 2 |dt| + 4u is the relative error of p_t, counted twice below for
    the terms of second order.
  - the weight of a value: p_t times its scale, u, rounded to q's type, h
    (fp16: below 2^-14 by 2^-25 at most; its largest is at least 2^6, so that
    is 2^-31 of the largest product of weight and scale, times codes of 127; a
    row of zeros takes part in that largest with a scale of at most 2^-40).
  - numbers below 2^-126 may be taken as 0, by exp2 and by the matrix core: a
    weight of p_t / p_max below 2^-118 (the reference stands up to 2^8 from the
    maximum) is lost, N 2^-118 of the largest value at most (a first form
    without this term was off by 4e-40 where one weight was all there was).
    A value's scale below 2^-100 may count as that: 127 * 2^-100 < 2^-93.
  - sums over N keys: N u, twice for the matrix core, of the magnitudes; the
    shares' factors and the quotient, 8u.
  - the output's own rounding."""
import math

import pytest
import torch

import block_quantized_int8_q8_amd as mmq
from tests import kvcache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def heads(T, H, D, t, seed):
    g = gen(seed)
    x = torch.randn((T, H, D), generator=g, device=DEV)
    return (x * torch.exp(0.4 * torch.randn((H, D), generator=g, device=DEV))).to(t)


def poisoned(n_pages, page, H, D):
    cache = mmq.kv_cache(n_pages, page, H, D, device=DEV)
    cache.fill_(0xff)
    return cache


class Batch:
    """Sequences of `lens` tokens, the last `new` of them new, on shuffled pages of a poisoned cache."""

    def __init__(self, new, lens, Hq, Hkv, D, page, t, seed=1, k=None, v=None, behind=0, spare=3, max_pages=None, qscale=1.0):
        self.new, self.lens_h, self.D, self.page, self.G = new, lens, D, page, Hq // Hkv
        B = len(lens)
        need = [-(-max(n, 0) // page) for n in lens]
        n_pages = sum(need) + spare
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed))
        width = max(need + [1]) if max_pages is None else max_pages
        table = torch.full((B, width), -7, dtype=torch.int32)         # no page where none is needed
        slots, at = [], 0
        for b, n in enumerate(lens):
            mine = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = mine[:width].to(torch.int32)
            tok = torch.arange(max(n, 0))
            slots.append(mine[tok // page] * page + tok % page if n > 0 else tok)
        self.slots = slots
        flat = torch.cat(slots).to(torch.int32).to(DEV)
        total = flat.numel()
        self.k = heads(total, Hkv, D, t, seed + 10) if k is None else k(total)
        self.v = heads(total, Hkv, D, self.k.dtype, seed + 11) if v is None else v(total).to(self.k.dtype)
        self.cache = poisoned(n_pages, page, Hkv, D)
        if total:
            mmq.kv_write(self.k, self.v, self.cache, flat)
        self.table = table.to(DEV)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.offsets = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(DEV)
        self.q = (heads(sum(new) + behind, Hq, D, F32, seed + 12) * qscale).to(t)

    def run(self, **kw):
        return mmq.attention_i8(self.q, self.cache, self.table, self.lens, self.offsets, **kw)


def reference(bt, scale, window=0, table=None):
    """Exact outputs and their bounds without the output's rounding, [rows of the sequences, Hq, D] in 64 bits."""
    (kc, kd), (vc, vd) = kvcache.unpack(bt.cache, bt.D)
    P = bt.cache.shape[0]
    table = (bt.table if table is None else table).cpu()
    h16 = torch.finfo(bt.q.dtype).eps / 2
    outs, bounds, i = [], [], 0
    for b, (n, length) in enumerate(zip(bt.new, bt.lens_h)):
        length = min(max(length, 0), table.shape[1] * bt.page)
        tok = torch.arange(length)
        page = table[b].long()[tok // bt.page]
        there = ((page >= 0) & (page < P)).to(DEV)
        slot = (page.clamp(0, P - 1) * bt.page + tok % bt.page).to(DEV)
        q = bt.q[i:i + n].double()
        i += n
        pos = torch.arange(length - n, length, device=DEV)[:, None]
        key = torch.arange(length, device=DEV)[None]
        seen = (key <= pos) & there[None]
        if window:
            seen &= key > pos - window
        o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
        e = torch.zeros_like(o)
        for h in range(q.shape[1] if length and n else 0):
            g = h // bt.G
            c, d, w_c, w_d = kc[slot, g].double(), kd[slot, g].double(), vc[slot, g].double(), vd[slot, g].double()
            d, w_d = torch.where(there, d, 0.0), torch.where(there, w_d, 0.0)
            f = scale * d * math.log2(math.e)
            t = (q[:, h] @ c.t()) * f
            A = (q[:, h].abs() @ c.abs().t()) * f.abs()
            ts = torch.where(seen, t, -math.inf)
            m = ts.amax(1, keepdim=True)
            none = torch.isinf(m) & (m < 0)
            w = torch.where(seen, torch.exp2(torch.where(seen, t, 0.0) - torch.where(none, 0.0, m)), 0.0)
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
            V = w_c * w_d[:, None]
            V = torch.where(seen.any(0)[:, None], V, 0.0)             # not seen by any row: may be NaN
            wv = w @ V
            big = torch.where(seen, t.abs(), 0.0).amax(1, keepdim=True)
            eps = math.log(2) * (2 * bt.D * U * A + 3 * U * t.abs() + U * (t.abs() + big + 80)) + 4 * U
            eps = torch.where(seen, eps, 0.0)
            N = length
            mag = w @ V.abs()
            bound = 2 * ((w * eps) @ V.abs() + (w * eps).sum(1, keepdim=True) * wv.abs()) + (h16 * (1 + 2 * h16) + 3 * N * U + 9 * U) * mag \
                + N * U * wv.abs() + N * 2.0 ** -118 * V.abs().amax() + 2.0 ** -93
            if bt.q.dtype == F16:
                bound = bound + N * 2.0 ** -24 * ((w * torch.where(seen, w_d[None], 0.0)).amax(1, keepdim=True) + 2.0 ** -40)
            o[:, h], e[:, h] = wv, bound
        outs.append(o)
        bounds.append(e)
    return torch.cat(outs), torch.cat(bounds)


def check(bt, out, scale=None, window=0, table=None):
    want, bound = reference(bt, bt.D ** -0.5 if scale is None else scale, window, table)
    got = out[:want.shape[0]].double()
    h = torch.finfo(out.dtype).eps / 2
    bound = bound * (1 + 2 * h) + h * want.abs() + (2.0 ** -25 if out.dtype == F16 else 0.0)
    off = (got - want).abs()
    assert bool(torch.isfinite(got).all())
    assert bool((off <= bound).all()), (float((off - bound).max()), float((off / bound.clamp_min(1e-30)).max()))


# (new, lens): one token, few, the bounds of a row block (16, 32 rows), of a
# tile of keys (16), of a unit (32), of a step (64) and of a share; chunks from
# the first token and after a prefix; batches that mix all of it
DECODE = [([1], [1]), ([1], [2]), ([1], [16]), ([1], [17]), ([1], [31]), ([1], [33]), ([1], [64]), ([1], [127]), ([1], [129]),
          ([1], [511]), ([1], [1000]), ([1], [4133]), ([1, 1, 1], [5, 700, 64]), ([1] * 9, [1, 900, 33, 2, 128, 48, 257, 16, 15])]
CHUNKS = [([2], [2]), ([3], [40]), ([4], [300]), ([5], [5]), ([9], [100]), ([17], [17]), ([33], [33]), ([40], [1000]), ([64], [64]),
          ([65], [130]), ([130], [131]), ([300], [300]), ([77], [2111]), ([1, 60, 1, 5], [513, 60, 7, 300]),
          ([2, 1, 290, 33, 0, 1], [2, 1025, 300, 700, 50, 1])]


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("D,Hq,Hkv,page", [(64, 8, 2, 16), (128, 7, 1, 32), (128, 28, 4, 64), (256, 2, 1, 128), (64, 3, 3, 256)])
@pytest.mark.parametrize("new,lens", DECODE + CHUNKS)
def test_attention(new, lens, D, Hq, Hkv, page, t):
    print(new, lens, D, Hq, Hkv, page, t, flush=True)
    bt = Batch(new, lens, Hq, Hkv, D, page, t, seed=sum(lens) + D)
    check(bt, bt.run(max_q=max(new)))


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 40, 1), (64, 33, 1), (256, 32, 1), (128, 48, 3), (128, 16, 1), (64, 17, 1)])
@pytest.mark.parametrize("new,lens", [([1], [700]), ([1, 2, 1], [65, 300, 16]), ([30, 1], [400, 90])])
def test_group_sizes(new, lens, D, Hq, Hkv, t):
    print(new, lens, D, Hq, Hkv, t, flush=True)
    bt = Batch(new, lens, Hq, Hkv, D, 16, t, seed=3)
    check(bt, bt.run())


@pytest.mark.parametrize("t,out", [(BF16, F32), (F16, F32), (BF16, BF16), (F16, F16)])
@pytest.mark.parametrize("new,lens", [([1, 1], [300, 2000]), ([100], [350])])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_output_types_and_strides(new, lens, D, t, out):
    """Queries as a slice of a fused product's rows, outputs into a slice and into a [H, T, D] tensor; what lies
    between is not touched.  Rows start at any multiple of the type's size."""
    Hq, Hkv = 8, 2
    bt = Batch(new, lens, Hq, Hkv, D, 32, t, seed=5)
    T = sum(new)
    fused = torch.full((T, Hq * D + 3 * D + 1), 9.0, dtype=t, device=DEV)
    q = fused[:, 1:1 + Hq * D].view(T, Hq, D)
    q.copy_(bt.q)
    wide = torch.full((T, Hq + 3, D + 1), -5.0, dtype=out, device=DEV)
    o = wide[:, 1:1 + Hq, 1:]
    got = mmq.attention_i8(q, bt.cache, bt.table, bt.lens, bt.offsets, out=o)
    assert got is o
    check(bt, o)
    rest = torch.ones(wide.shape, dtype=torch.bool, device=DEV)
    rest[:, 1:1 + Hq, 1:] = False
    assert bool((wide[rest] == -5.0).all())
    turned = torch.full((Hq, T, D), -5.0, dtype=out, device=DEV)
    mmq.attention_i8(q, bt.cache, bt.table, bt.lens, bt.offsets, out=turned.transpose(0, 1))
    assert torch.equal(turned.transpose(0, 1), o)


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 513, 5000])
@pytest.mark.parametrize("new,lens", [([1], [800]), ([1, 1, 1], [3, 90, 2500]), ([200], [200]), ([150, 1, 20], [900, 900, 20])])
def test_window(new, lens, window, t):
    bt = Batch(new, lens, 8, 2, 64 if window % 2 else 128, 16, t, seed=window)
    check(bt, bt.run(window=window), window=window)


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("new,lens", [([3, 1, 70, 2], [0, 0, 40, 1]), ([90], [60]), ([1], [0]), ([0, 0], [5, 9])])
def test_rows_that_see_nothing_are_zero(new, lens, t):
    """More new tokens than the cache holds, or none at all: rows before the first key give zeros."""
    bt = Batch(new, lens, 4, 2, 128, 16, t, behind=2)
    out = torch.full_like(bt.q, 7.0)
    bt.run(out=out)
    check(bt, out)
    i = 0
    for n, length in zip(new, lens):
        assert bool((out[i:i + max(n - length, 0)] == 0).all())
        i += n
    assert bool((out[i:] == 7.0).all())


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("new,lens", [([1, 1], [300, 700]), ([80, 1], [300, 40])])
def test_pages_outside_the_cache_are_not_seen(new, lens, t):
    bt = Batch(new, lens, 8, 2, 128, 32, t)
    table = bt.table.clone()
    n_pages = bt.cache.shape[0]
    table[0, 1], table[0, 4], table[1, 0] = n_pages, -1, 2 ** 31 - 1
    out = mmq.attention_i8(bt.q, bt.cache, table, bt.lens, bt.offsets)
    check(bt, out, table=table)
    table[:] = -2 ** 31
    out = mmq.attention_i8(bt.q, bt.cache, table, bt.lens, bt.offsets)
    assert bool((out == 0).all())


def test_lengths_beyond_the_table_and_offsets_beyond_the_rows_are_clamped():
    bt = Batch([1, 1], [100, 60], 4, 2, 64, 16, BF16, max_pages=3)
    bt.new, bt.lens_h = [1, 1], [100, 60]
    out = bt.run()
    check(bt, out)                                                   # the reference clamps to 48 keys too
    bt = Batch([2, 3], [50, 60], 4, 2, 64, 16, BF16)
    out = torch.full_like(bt.q, 7.0)
    mmq.attention_i8(bt.q, bt.cache, bt.table, bt.lens, torch.tensor([0, 2, 1000], dtype=torch.int32, device=DEV), out=out)
    check(bt, out)
    lens = torch.tensor([-5, -2 ** 31], dtype=torch.int32, device=DEV)
    mmq.attention_i8(bt.q, bt.cache, bt.table, lens, bt.offsets, out=out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("Hq", [4, 40])
def test_rows_behind_the_sequences_and_past_max_q_are_left(Hq):
    for new, lens, max_q in [([5, 9], [30, 200], 3), ([40, 1], [100, 100], 17)]:
        bt = Batch(new, lens, Hq, 1, 64, 16, F16, behind=6)
        out = torch.full_like(bt.q, 3.0)
        bt.run(out=out, max_q=max_q)
        full = bt.run()
        keep = torch.zeros(out.shape[0], dtype=torch.bool, device=DEV)
        i = 0
        for n in new:
            keep[i:i + min(n, max_q)] = True
            i += n
        assert bool((out[~keep] == 3.0).all())
        want, bound = reference(bt, 64 ** -0.5)
        err = (out[:i][keep[:i]].double() - want[keep[:i]]).abs()
        assert bool((err <= bound[keep[:i]] * 1.01 + 2.0 ** -11 * want[keep[:i]].abs() + 2.0 ** -25).all())
        assert bool(full[:i].isfinite().all())


@pytest.mark.parametrize("t", [BF16, F16])
def test_nan_and_infinity_reach_their_rows_only(t):
    """A token whose key or value is infinite: rows that see it are NaN, rows before it, other heads and other
    sequences are not."""
    new, lens = [50, 1, 40], [200, 400, 40]
    clean = Batch(new, lens, 4, 2, 128, 16, t, seed=4)
    want = clean.run()
    for what in "kv":
        bt = Batch(new, lens, 4, 2, 128, 16, t, seed=4)
        x = (bt.k, bt.v)[what == "v"].clone()
        x[170, 1, 5] = float("inf")                                  # sequence 0, position 170: new token 20 on
        x[200 + 399, 0, 7] = float("nan")                            # sequence 1, its last token
        mmq.kv_write(x if what == "k" else bt.k, x if what == "v" else bt.v, bt.cache, torch.cat(bt.slots).to(torch.int32).to(DEV))
        got = bt.run()
        bad = torch.zeros(got.shape[:2], dtype=torch.bool, device=DEV)
        bad[20:50, 2:] = True
        bad[50, :2] = True
        assert bool(got[bad].isnan().all())
        assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("qscale", [0.0, 1e-3, 6.0, 60.0])
def test_flat_and_sharp_softmax(qscale, t):
    """All weights equal, and one weight all there is; scores to hundreds."""
    for new, lens in [([1], [3000]), ([70], [600])]:
        bt = Batch(new, lens, 8, 2, 128, 64, t, seed=7, qscale=qscale)
        check(bt, bt.run())


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("rising", [True, False])
def test_values_of_very_different_size(t, rising):
    """Values from 2^-14 to 2^14 along the keys, and keys whose scores grow along them: the running reference moves
    many times, and small values before or after large ones keep their digits where they are all that is seen."""
    def v(total):
        e = torch.linspace(-14, 14, total, device=DEV)
        return torch.exp2(e if rising else -e)[:, None, None] * heads(total, 2, 64, F32, 21)

    def k(total):
        return torch.linspace(-3, 3, total, device=DEV)[:, None, None] * heads(total, 2, 64, F32, 22).abs()
    for new, lens in [([1], [900]), ([300], [300]), ([60], [900])]:
        bt = Batch(new, lens, 4, 2, 64, 16, t, k=k, v=v)             # in fp32: fp16 ends at 65504
        check(bt, bt.run(dtype=F32))


def test_zero_keys_and_values():
    zero = lambda total: torch.zeros((total, 2, 64), device=DEV)
    for t in (BF16, F16):
        bt = Batch([40, 1], [100, 300], 4, 2, 64, 16, t, v=zero)
        assert bool((bt.run() == 0).all())
        bt = Batch([40, 1], [100, 300], 4, 2, 64, 16, t, k=zero)
        check(bt, bt.run())


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("small", [0.0, 1e-37, 1e-30, 1e-6])
@pytest.mark.parametrize("new,lens", [([1], [700]), ([100], [700]), ([200, 1], [200, 90])])
def test_rows_of_zeros_and_tiny_values_keep_their_weight(new, lens, small, t):
    """Values that are zero, or next to nothing, at every third key, at runs of 64 keys and at the keys that weigh most:
    they add nothing to the output and all of their weight to the sum."""
    def v(total):
        x = heads(total, 2, 64, F32, 31)
        i = torch.arange(total, device=DEV)
        x[(i % 3 == 1) | (i // 64 % 4 == 2)] *= small
        return x

    def k(total):
        x = heads(total, 2, 64, F32, 32)
        x[torch.arange(total, device=DEV) % 3 == 1] *= 3.0
        return x
    bt = Batch(new, lens, 8, 2, 64, 16, t, k=k, v=v)
    check(bt, bt.run(dtype=F32))
    check(bt, bt.run())
    bt = Batch(new, lens, 8, 2, 64, 16, t, k=k, v=lambda total: heads(total, 2, 64, F32, 33) * small)
    check(bt, bt.run(dtype=F32))


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,lens,window", [([2500], [2500], 0), ([1300, 900], [3300, 900], 0), ([2100], [4000], 1500)])
def test_long_chunks(new, lens, window, D, t):
    """Workgroups that walk more steps than they look up pages for at once."""
    bt = Batch(new, lens, 16, 8, D, 16 if D == 64 else 32, t, seed=13)
    check(bt, bt.run(window=window), window=window)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 5.0])
def test_scale(scale):
    bt = Batch([1, 66], [200, 300], 8, 2, 64, 16, BF16)
    check(bt, bt.run(scale=scale), scale=scale)


def test_cache_beyond_32_bit_offsets():
    """A cache of 5.4 GB: pages at its end, keys, values and queries at their own far strides."""
    page, H, D = 256, 4, 128
    n_pages = (5 << 30) // (page * H * (2 * D + 8))
    cache = mmq.kv_cache(n_pages, page, H, D, device=DEV)
    bt = Batch([1, 50], [600, 300], 8, H, D, page, BF16, spare=2)
    small = bt.cache.shape[0]
    cache[n_pages - small:] = bt.cache
    table = torch.where(bt.table >= 0, bt.table + (n_pages - small), bt.table)
    assert torch.equal(mmq.attention_i8(bt.q, cache, table, bt.lens, bt.offsets), bt.run())
    slots = (torch.cat(bt.slots) + (n_pages - small) * page).to(torch.int32).to(DEV)
    k, v = mmq.kv_read(cache, slots, D)
    k2, v2 = mmq.kv_read(bt.cache, torch.cat(bt.slots).to(torch.int32).to(DEV), D)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    far = torch.empty((3, 2 ** 30), dtype=BF16, device=DEV)
    q = far[:2, -8 * D:].view(2, 8, D)
    q.copy_(bt.q[:2])
    out = far[:, :8 * D].view(3, 8, D)[1:]
    offsets = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    mmq.attention_i8(q, cache, table, bt.lens, offsets, out=out)
    assert torch.equal(out, mmq.attention_i8(bt.q[:2].contiguous(), cache, table, bt.lens, offsets))


@pytest.mark.parametrize("new,lens", [([1] * 5, [700, 3, 90, 2000, 16]), ([1, 200, 40], [800, 300, 1200])])
def test_graph_replays_streams_and_repeats(new, lens):
    """The same bits on every run; a captured call reads lengths, tables and queries anew at each replay."""
    bt = Batch(new, lens, 28, 4, 128, 16, BF16, seed=9)
    want = bt.run()
    for _ in range(3):
        assert torch.equal(bt.run(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bt.run(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    need = mmq.attention_workspace_bytes(sum(new), len(new), max(new), 28, 4, 128, bt.table.shape[1], 16)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(bt.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bt.run(out=out, workspace=ws, max_q=max(new))
    again = Batch(new, [max(n, length - 1 - i) for i, (n, length) in enumerate(zip(new, lens))], 28, 4, 128, 16, BF16, seed=9,
                  max_pages=bt.table.shape[1])
    for other in (False, True, False):
        src = again if other else bt
        if other:
            keep = bt.lens.clone(), bt.table.clone(), bt.cache.clone()
            bt.lens.copy_(again.lens)
            pages = again.cache.shape[0]
            assert pages <= bt.cache.shape[0]
            bt.cache[:pages] = again.cache
            bt.table.copy_(again.table)
        eager = src.run(max_q=max(new))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        ws.fill_(0xff)
        if other:
            bt.lens.copy_(keep[0])
            bt.table.copy_(keep[1])
            bt.cache.copy_(keep[2])


def test_many_sequences():
    """More sequences than a wave scans at once, of both kinds."""
    g = torch.Generator().manual_seed(3)
    new = [int(torch.randint(0, 4, (1,), generator=g)) if i % 7 else 40 for i in range(200)]
    lens = [n + int(torch.randint(0, 200, (1,), generator=g)) for n in new]
    bt = Batch(new, lens, 8, 2, 64, 16, BF16, seed=11)
    check(bt, bt.run())
    check(bt, bt.run(max_q=40, window=50), window=50)


def test_a_short_sequence_does_not_depend_on_its_neighbours_values():
    a = Batch([1, 1], [100, 500], 8, 2, 128, 16, BF16, seed=2)
    want = a.run()
    slots = a.slots[1].to(torch.int32).to(DEV)
    big = heads(500, 2, 128, F32, 77) * 100
    mmq.kv_write(big, big, a.cache, slots)
    assert torch.equal(a.run()[0], want[0])


def test_two_calls_at_once():
    """Two streams, each with its own batch and workspace, many times over: the results of either alone."""
    a = Batch([1] * 6, [900, 3, 77, 2000, 16, 500], 28, 4, 128, 16, BF16, seed=21)
    b = Batch([300, 1, 40], [700, 400, 1200], 8, 2, 64, 32, F16, seed=22)
    want = [a.run(), b.run()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        outs.append([x.run(stream=s) for x, s in zip((a, b), streams)])
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for got in outs for g, w in zip(got, want))


def test_decode_step_by_step_equals_the_prompt():
    """A prompt in one chunk and token by token: the same cache, rows within both calls' bounds of the exact ones."""
    n = 90
    whole = Batch([n], [n], 8, 2, 128, 16, BF16, seed=23)
    check(whole, whole.run())
    for i in (0, 1, 15, 16, 31, 32, 63, 64, 89):
        one = torch.tensor([i + 1], dtype=torch.int32, device=DEV)
        step = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
        got = mmq.attention_i8(whole.q[i:i + 1], whole.cache, whole.table, one, step)
        want, bound = reference(whole, 128 ** -0.5)
        off = (got[0].double() - want[i]).abs()
        assert bool((off <= bound[i] * 1.01 + 2.0 ** -8 * want[i].abs() * 1.01).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,lens", [([1] * 5, [900, 3, 77, 2000, 16]), ([300, 1], [700, 400]), ([4, 70], [3000, 70]), ([2500], [2500])])
def test_output_over_the_queries(new, lens, D):
    bt = Batch(new, lens, 16, 4, D, 16, F16, seed=24)
    want = bt.run()
    assert bt.run(out=bt.q) is bt.q
    assert torch.equal(bt.q, want)


@pytest.mark.parametrize("Hq", [4, 40])
@pytest.mark.parametrize("offsets", [[0, 5, 2, 8], [3, 3, -7, 9], [9, 4, 1, 0], [-100, 2 ** 31 - 1, 0, 5]])
def test_offsets_that_decrease_stay_within_the_rows(offsets, Hq):
    """What rows between decreasing offsets hold is not said; rows past the last offset anyone names are left."""
    bt = Batch([3, 3, 3], [100, 40, 300], Hq, 1, 64, 16, F16, behind=0)
    store = torch.full((20, Hq, 64), 3.0, dtype=F16, device=DEV)
    mmq.attention_i8(bt.q, bt.cache, bt.table, bt.lens, torch.tensor(offsets, dtype=torch.int32, device=DEV), out=store[5:14])
    assert bool((store[:5] == 3.0).all()) and bool((store[14:] == 3.0).all())
    assert bool(store.isfinite().all())
