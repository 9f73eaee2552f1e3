"""Rotary positions and the int8 paged cache on the GPU against plain
implementations in 64 bits.

Tolerance of a rotated value y of the pair (a, b), u = 2^-53: the kernel's
angle has three roundings and the reference's one, the sines and cosines of
both an ulp or two, the products and the sum one each:
|dy| <= 8 u (|phi| + 2) m (|a| + |b|).  It is rounded to fp32 (2^-24) and to the
type (half a step h), and in fp16 to steps of 2^-24 below 2^-14.
A stored row's scale is amax / 127 to fp32, so within 2^-24 of the rounded
values' own; its codes are within 1/2 + 127 * 2^-22 of y / d (the reciprocal and
the product round once each), and code * d rounds once more."""
import math

import pytest
import torch

import block_quantized_int8_q8_amd as mmq
from tests import kvcache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(shape, t, seed):
    return (torch.randn(shape, generator=gen(seed)) * torch.exp(0.5 * torch.randn(shape[-1], generator=gen(seed + 1)))).to(t)


def turned(x, positions, freqs, layout, mscale, inverse=False):
    """Exact rotation of x (CPU) and the bound on the kernel's value before its roundings."""
    rot = 2 * freqs.numel()
    phi = positions.double()[:, None, None] * freqs
    y = x.double().clone()
    bound = torch.zeros_like(y)
    A, B = ((slice(0, rot // 2), slice(rot // 2, rot)) if layout == mmq.ROPE_HALF else (slice(0, rot, 2), slice(1, rot, 2)))
    a, b = y[..., A].clone(), y[..., B].clone()
    s = -torch.sin(phi) if inverse else torch.sin(phi)
    y[..., A] = mscale * (a * torch.cos(phi) - b * s)
    y[..., B] = mscale * (b * torch.cos(phi) + a * s)
    e = 8 * 2.0 ** -53 * (phi.abs() + 2) * abs(mscale) * (a.abs() + b.abs())
    bound[..., A], bound[..., B] = e, e
    return y, bound


def close(got, y, bound):
    t = got.dtype
    h = 2.0 ** -24 + (0 if t == F32 else torch.finfo(t).eps / 2)
    tol = bound + h * (y.abs() + bound) * (1 + 2.0 ** -8) + (2.0 ** -25 if t == F16 else 2.0 ** -149)
    fits = y.abs() < torch.finfo(t).max
    return bool(((got.cpu().double() - y).abs() <= tol)[fits].all())


ROPES = [(1, 1, 64, 64), (1, 28, 128, 128), (3, 5, 128, 32), (7, 4, 256, 256), (64, 28, 128, 128), (65, 3, 96, 96), (33, 2, 80, 40),
         (1025, 4, 128, 128), (1030, 3, 64, 20), (1027, 1, 8, 6), (5, 9, 512, 512), (17, 6, 40, 2), (1100, 2, 256, 64), (9, 1, 16, 16),
         # four tokens a workgroup
         (4100, 3, 128, 128), (4097, 2, 64, 20), (4099, 1, 80, 40), (4111, 5, 64, 32), (5000, 2, 256, 256), (4098, 2, 8, 8)]


@pytest.mark.parametrize("layout", [mmq.ROPE_HALF, mmq.ROPE_INTERLEAVED])
@pytest.mark.parametrize("T,H,D,rot", ROPES)
def test_rope(T, H, D, rot, layout):
    i = T + H + D
    ti, to = TYPES[i % 3], TYPES[(i // 3) % 3]
    freqs, m = mmq.rope_frequencies(rot, base=500000.0, scaling=[None, "linear", "bands", "yarn"][i % 4], factor=4.0, original=8192)
    positions = torch.randint(-5, 1 << 24, (T,), generator=gen(i), dtype=torch.int32)
    x = rand((T, H, D), ti, i)
    for inverse in (False, True):
        got = mmq.rope(x.to(DEV), positions.to(DEV), freqs.to(DEV), layout=layout, mscale=m, inverse=inverse, dtype=to)
        assert got.dtype == to and got.shape == x.shape
        y, bound = turned(x, positions, freqs, layout, m, inverse)
        assert close(got, y, bound)
        assert torch.equal(got.cpu()[..., rot:], x[..., rot:].float().to(to))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("layout", [mmq.ROPE_HALF, mmq.ROPE_INTERLEAVED])
def test_rope_strides_and_in_place(t, layout):
    """A slice of a fused product's rows turned in place, [H, T, D] in memory, and one head for all: what lies between
    is not touched, and all give the same bits."""
    for T in (6, 1300, 4203):
        H, D = 5, 64
        freqs, _ = mmq.rope_frequencies(48)
        freqs, positions = freqs.to(DEV), torch.arange(T, dtype=torch.int32, device=DEV) * 3
        x = rand((T, H, D), t, T).to(DEV)
        want = mmq.rope(x, positions, freqs, layout=layout)
        fused = torch.full((T, H * D + 131), 5.0, dtype=t, device=DEV)
        part = fused[:, 1:1 + H * D].view(T, H, D)
        part.copy_(x)
        assert mmq.rope(part, positions, freqs, layout=layout, out=part) is part
        assert torch.equal(part, want)
        assert bool((fused[:, 0] == 5.0).all()) and bool((fused[:, 1 + H * D:] == 5.0).all())
        ht = x.transpose(0, 1).contiguous().transpose(0, 1)
        out = torch.empty((H, T, D), dtype=t, device=DEV).transpose(0, 1)
        assert torch.equal(mmq.rope(ht, positions, freqs, layout=layout, out=out), want)
        assert torch.equal(mmq.rope(x[:, :1].expand(T, H, D), positions, freqs, layout=layout)[:, 3], want[:, 0])


def test_rope_is_its_own_gradient_by_differences():
    """<rope(x), g> changes with x as its gradient, rope(g, inverse), says: the map is linear, so a difference of any
    size gives the slope; each inner product of fp32 values carries n 2^-24 of its magnitudes at most."""
    T, H, D = 5, 3, 64
    freqs, m = mmq.rope_frequencies(32, scaling="yarn", factor=8.0, original=4096)
    positions = torch.tensor([0, 7, 100, 4096, 1000000], dtype=torch.int32, device=DEV)
    x, g, dx = (rand((T, H, D), F32, s).to(DEV) for s in (1, 2, 3))
    for layout in (mmq.ROPE_HALF, mmq.ROPE_INTERLEAVED):
        f = lambda z: mmq.rope(z, positions, freqs.to(DEV), layout=layout, mscale=m).double()
        grad = mmq.rope(g, positions, freqs.to(DEV), layout=layout, mscale=m, inverse=True).double()
        slope = ((f(x + dx) - f(x - dx)) * g.double()).sum() / 2
        want = (grad * dx.double()).sum()
        mags = 2 * m * ((x.abs() + dx.abs()).double().sum() * g.abs().max() * 2)
        assert abs(float(slope - want)) <= 4 * 2.0 ** -24 * float(mags)


def test_frequencies_against_the_formulas():
    for rot, base, factor, original in [(128, 1e6, 8.0, 32768), (64, 1e4, 4.0, 4096), (2, 1e4, 2.0, 128), (256, 5e5, 40.0, 8192)]:
        i = torch.arange(rot // 2, dtype=torch.float64)
        f = base ** (-2 * i / rot)
        turns = f * original / (2 * math.pi)
        assert torch.allclose(mmq.rope_frequencies(rot, base)[0], f, rtol=1e-14, atol=0)
        assert torch.allclose(mmq.rope_frequencies(rot, base, "linear", factor)[0], f / factor, rtol=1e-14, atol=0)
        keep = ((turns - 1) / 3).clamp(0, 1)
        got, m = mmq.rope_frequencies(rot, base, "bands", factor, original=original)
        assert m == 1.0 and torch.allclose(got, f / factor * (1 - keep) + f * keep, rtol=1e-13, atol=0)
        pair = lambda n: rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))
        a, b = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), rot - 1)
        keep = (1 - (i - a) / max(b - a, 0.001)).clamp(0, 1)
        got, m = mmq.rope_frequencies(rot, base, "yarn", factor, original=original)
        assert math.isclose(m, 0.1 * math.log(factor) + 1, rel_tol=1e-15)
        assert torch.allclose(got, f / factor * (1 - keep) + f * keep, rtol=1e-13, atol=0)


# ---------------------------------------------------------------------------
# cache
# ---------------------------------------------------------------------------
CACHES = [(1, 1, 64, 16), (1, 4, 128, 16), (5, 3, 256, 32), (64, 4, 128, 64), (70, 8, 64, 128), (1024, 2, 128, 16), (1111, 1, 64, 256),
          (1030, 5, 256, 64),
          # sixteen tokens a workgroup
          (4099, 2, 64, 16), (2061, 5, 128, 64), (1501, 8, 256, 32), (4100, 1, 128, 16), (2050, 7, 64, 256), (5000, 3, 256, 16)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("T,H,D,page", CACHES)
def test_write_and_read(T, H, D, page, t):
    """Codes and scales bit for bit where nothing is turned; every other byte of the cache as it was; values back."""
    n_pages = -(-T // page) + 2
    cache = mmq.kv_cache(n_pages, page, H, D, device=DEV)
    cache.fill_(0xa5)
    slots = torch.randperm(n_pages * page, generator=gen(T))[:T].to(torch.int32)
    if T % 2:
        slots = slots.sort().values                                  # in order, as a prompt's are
    k, v = rand((T, H, D), t, 1), rand((T, H, D), t, 2)
    k[0, 0], v[-1, -1] = 0.0, 0.0
    mmq.kv_write(k.to(DEV), v.to(DEV), cache, slots.to(DEV))
    before = kvcache.unpack(torch.full_like(cache, 0xa5).cpu(), D)
    got = kvcache.unpack(cache.cpu(), D)
    out = mmq.kv_read(cache, slots.to(DEV), D, dtype=t)
    for x, (codes, d), (codes0, d0), read in zip((k, v), got, before, out):
        want, scale = kvcache.quantize_rows(x)
        codes0[slots.long()], d0[slots.long()] = want, scale
        assert torch.equal(codes, codes0) and torch.equal(d.view(torch.int32), d0.view(torch.int32))
        assert read.dtype == t and torch.equal(read.cpu(), (want.float() * scale[..., None]).to(t))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("first", [0, 1, 2, 3, 7])
@pytest.mark.parametrize("H,D", [(4, 128), (8, 64), (3, 256)])
def test_write_consecutive_slots_from_any_place(H, D, first, t):
    """A prompt's slots in a row, from any place of a page, with a jump and a token that is passed over among them, and
    a batch whose sequences begin at their own places."""
    T = 4099
    n_pages = (T + 200) // 32 + 1
    slots = torch.arange(first, first + T, dtype=torch.int32)
    slots[1000:] += 5
    slots[2000:] += 50
    slots[77] = -1
    slots[3001:3400] = slots[3001:3400].flip(0)
    cache = mmq.kv_cache(n_pages, 32, H, D, device=DEV)
    cache.fill_(0x11)
    before = kvcache.unpack(cache.cpu(), D)
    k, v = rand((T, H, D), t, 1), rand((T, H, D), t, 2)
    mmq.kv_write(k.to(DEV), v.to(DEV), cache, slots.to(DEV))
    kept = slots >= 0
    for x, (codes, d), (codes0, d0) in zip((k, v), kvcache.unpack(cache.cpu(), D), before):
        want, scale = kvcache.quantize_rows(x)
        codes0[slots[kept].long()], d0[slots[kept].long()] = want[kept], scale[kept]
        assert torch.equal(codes, codes0) and torch.equal(d.view(torch.int32), d0.view(torch.int32))


@pytest.mark.parametrize("layout", [mmq.ROPE_HALF, mmq.ROPE_INTERLEAVED])
@pytest.mark.parametrize("T,H,D,rot,t", [(1, 4, 128, 128, BF16), (9, 2, 64, 20, F32), (1031, 3, 128, 32, F16), (1050, 1, 256, 256, F32),
                                         (40, 8, 256, 128, BF16), (4101, 2, 128, 128, BF16), (1503, 7, 64, 20, F32),
                                         (1499, 8, 256, 64, F16), (4100, 1, 128, 6, BF16)])
def test_write_turns_keys(T, H, D, rot, t, layout):
    freqs, m = mmq.rope_frequencies(rot, base=1e6, scaling="yarn", factor=8.0, original=32768)
    positions = torch.arange(900000, 900000 + T, dtype=torch.int32)
    n_pages = T // 16 + 1
    cache = mmq.kv_cache(n_pages, 16, H, D, device=DEV)
    slots = torch.arange(T, dtype=torch.int32)
    kv = rand((T, 2 * H, D), t, T).to(DEV)
    k, v = kv[:, :H], kv[:, H:]
    mmq.kv_write(k, v, cache, slots.to(DEV), positions=positions.to(DEV), freqs=freqs.to(DEV), layout=layout, mscale=m)
    (kc, kd), (vc, vd) = kvcache.unpack(cache.cpu(), D)
    y, bound = turned(k.cpu(), positions, freqs, layout, m)
    bound = bound + 2.0 ** -24 * y.abs()
    kc, kd = kc[:T].double(), kd[:T].double()
    amax = y.abs().amax(-1)
    assert bool(((kd * 127 - amax).abs() <= bound.amax(-1) + 2.0 ** -24 * amax).all())
    assert bool(((kc * kd[..., None] - y).abs() <= kd[..., None] * (0.5 + 127 * 2.0 ** -22) + bound).all())
    want, scale = kvcache.quantize_rows(v.cpu())
    assert torch.equal(vc[:T], want) and torch.equal(vd[:T], scale)


def test_write_passes_over_slots_outside_and_read_leaves_their_rows():
    H, D, page = 2, 64, 16
    for T in (9, 1500, 4503):
        n_pages = T // 16 + 1
        cache = mmq.kv_cache(n_pages, page, H, D, device=DEV)
        cache.fill_(0x5a)
        k, v = rand((T, H, D), BF16, 1).to(DEV), rand((T, H, D), BF16, 2).to(DEV)
        slots = torch.arange(T, dtype=torch.int32)
        slots[1], slots[4], slots[7] = -1, n_pages * page, -2 ** 31
        kept = torch.ones(T, dtype=torch.bool)
        kept[[1, 4, 7]] = False
        mmq.kv_write(k, v, cache, slots.to(DEV))
        (kc, kd), (vc, vd) = kvcache.unpack(cache.cpu(), D)
        free = torch.ones(n_pages * page, dtype=torch.bool)
        free[slots[kept].long()] = False
        assert bool((kc[free] == 0x5a).all()) and bool((vc[free] == 0x5a).all())
        assert torch.equal(kc[slots[kept].long()], kvcache.quantize_rows(k.cpu()[kept])[0])
        ko, vo = torch.full((T, H, D), 4.0, device=DEV), torch.full((H, T, D), 4.0, device=DEV).transpose(0, 1)
        mmq.kv_read(cache, slots.to(DEV), D, k=ko, v=vo)
        assert bool((ko.cpu()[~kept] == 4.0).all()) and bool((vo.cpu()[~kept] == 4.0).all())
        for x, o in ((k, ko), (v, vo)):
            c, d = kvcache.quantize_rows(x.cpu())
            assert torch.equal(o.cpu()[kept], (c.float() * d[..., None])[kept])
        again = torch.tensor([3, 3, 0, 3], dtype=torch.int32, device=DEV)
        assert torch.equal(mmq.kv_read(cache, again, D, dtype=F32)[0], ko[[3, 3, 0, 3]])


@pytest.mark.parametrize("t", TYPES)
def test_rows_with_infinities_nan_and_tiny_values(t):
    T, H, D = 6, 2, 64
    k, v = rand((T, H, D), t, 1), rand((T, H, D), t, 2)
    k[0, 0, 3], k[1, 1, 0], v[2, 0, 63], v[3, 1, 1] = float("inf"), float("nan"), float("-inf"), float("nan")
    k[4], v[4] = torch.finfo(t).max, -torch.finfo(t).max
    tiny = torch.finfo(t).smallest_normal if t == F16 else 1e-40
    k[5], v[5] = tiny, -tiny
    cache = mmq.kv_cache(1, 16, H, D, device=DEV)
    mmq.kv_write(k.to(DEV), v.to(DEV), cache, torch.arange(T, dtype=torch.int32, device=DEV))
    for x, (c, d) in zip((k, v), kvcache.unpack(cache.cpu(), D)):
        want, scale = kvcache.quantize_rows(x)
        assert torch.equal(c[:T], want)
        assert torch.equal(d[:T].isnan(), scale.isnan()) and torch.equal(d[:T].nan_to_num(7.0), scale.nan_to_num(7.0))
    ko, _ = mmq.kv_read(cache, torch.arange(T, dtype=torch.int32, device=DEV), D, dtype=F32)
    assert bool(ko[0, 0].isnan().all()) and bool(ko[0, 1].isfinite().all()) and bool(ko[1, 1].isnan().all())


def test_layer_from_the_product_to_the_product():
    """As they are used: one int8 product gives q, k and v of new tokens; q is turned in place, k and v go to the cache
    (k turned there), attention reads it, and its rows are quantized for the output product.  Two steps: a prompt in one
    chunk, then a token; the cache carries over, the second as a captured graph replayed."""
    hidden, Hq, Hkv, D, page = 512, 14, 2, 64, 16
    wide = (Hq + 2 * Hkv) * D
    w, ws = mmq.quantize_i8(torch.randn((wide, hidden), generator=gen(1)).to(DEV) / hidden ** 0.5)
    wo, wos = mmq.quantize_i8(torch.randn((hidden, Hq * D), generator=gen(2)).to(DEV) / hidden ** 0.5)
    freqs, m = mmq.rope_frequencies(D, base=1e6)
    freqs = freqs.to(DEV)
    n_pages = 12
    cache = mmq.kv_cache(n_pages, page, Hkv, D, device=DEV)
    cache.fill_(0xff)
    pages = torch.randperm(n_pages, generator=gen(3)).to(torch.int32).to(DEV)
    table = pages[None].contiguous()

    def step(x, positions, slots, lens, offsets):
        qkv = mmq.gemm_i8(*mmq.quantize_i8(x), w, ws, dtype=BF16).view(x.shape[0], Hq + 2 * Hkv, D)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        mmq.rope(q, positions, freqs, mscale=m, out=q)
        mmq.kv_write(k, v, cache, slots, positions=positions, freqs=freqs, mscale=m)
        o = mmq.attention_i8(q, cache, table, lens, offsets)
        return q, k, v, o, mmq.gemm_i8(*mmq.quantize_i8(o.view(x.shape[0], Hq * D)), wo, wos, dtype=BF16)

    def inputs(first, n, seed):
        pos = torch.arange(first, first + n, dtype=torch.int32, device=DEV)
        slots = pages[(pos // page).long()] * page + pos % page
        return (torch.randn((n, hidden), generator=gen(seed)).to(DEV, BF16), pos, slots.to(torch.int32),
                torch.tensor([first + n], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV))

    keys, values = [], []

    def expect(got, args):
        q, k, v, o, y = got
        n = q.shape[0]
        keys.append(turned(k.cpu(), args[1].cpu(), freqs.cpu(), mmq.ROPE_HALF, m)[0])
        values.append(v.cpu().double())
        K, V = torch.cat(keys), torch.cat(values)
        L = K.shape[0]
        want = torch.empty((n, Hq, D), dtype=torch.float64)
        for h in range(Hq):
            s = q[:, h].cpu().double() @ K[:, h // 7].t() / math.sqrt(D)
            s = s.masked_fill(torch.arange(L)[None] > torch.arange(L - n, L)[:, None], -math.inf)
            want[:, h] = torch.softmax(s, 1) @ V[:, h // 7]
        # codes are within half a step of 1/127 of a row's largest value: values and scores move by that much at most
        dk, dv = K.abs().amax(-1) / 254, V.abs().amax(-1) / 254
        ds = (q.cpu().double().abs().sum(-1).amax() * dk.amax() / math.sqrt(D))
        bound = dv.amax() + (torch.exp(2 * ds) - 1) * V.abs().amax() + 2.0 ** -7 * V.abs().amax()
        assert float((o.cpu().double() - want).abs().max()) <= float(bound)
        # the typical element is far nearer: the steps' errors are independent and average out
        assert float((o.cpu().double() - want).norm() / want.norm()) < 0.05
        full = torch.matmul(o.cpu().double().reshape(n, Hq * D), (wo.cpu().double() * wos.cpu().double()[:, None]).t())
        assert float((y.cpu().double() - full).norm() / full.norm()) < 0.02

    first = inputs(0, 150, 5)
    expect(step(*first), first)
    held = inputs(150, 1, 6)
    mmq.attention_i8(torch.zeros((1, Hq, D), dtype=BF16, device=DEV), cache, table, held[3], held[4])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*held)
    for i in range(4):
        for dst, src in zip(held, inputs(150 + i, 1, 6 + i)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        expect(got, held)
        eager = step(*held)
        assert all(torch.equal(a, b) for a, b in zip(eager, got))


def test_streams():
    """On a named stream, results are allocated there and the inputs kept until it is done."""
    x = rand((70, 4, 64), BF16, 1).to(DEV)
    freqs = mmq.rope_frequencies(64)[0].to(DEV)
    pos = torch.arange(70, dtype=torch.int32, device=DEV)
    cache = mmq.kv_cache(5, 16, 4, 64, device=DEV)
    want = mmq.rope(x, pos, freqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mmq.rope(x, pos, freqs, stream=side)
    mmq.kv_write(x, x, cache, pos, stream=side)
    k, v = mmq.kv_read(cache, pos, 64, stream=side)
    side.synchronize()
    c, d = kvcache.quantize_rows(x.cpu())
    back = (c.float() * d[..., None]).to(BF16)
    assert torch.equal(got, want) and torch.equal(k.cpu(), back) and torch.equal(v.cpu(), back)


def test_binding_refuses():
    x = torch.zeros((3, 2, 64), dtype=BF16, device=DEV)
    i3 = torch.zeros(3, dtype=torch.int32, device=DEV)
    f = torch.ones(32, dtype=torch.float64, device=DEV)
    cache = mmq.kv_cache(2, 16, 2, 64, device=DEV)
    table, lens = torch.zeros((1, 2), dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    calls = [
        (lambda: mmq.rope(x[0], i3, f), "tokens, heads"), (lambda: mmq.rope(x, i3.long(), f), "positions"),
        (lambda: mmq.rope(x, i3[:2], f), "positions"), (lambda: mmq.rope(x, i3, f.float()), "freqs"),
        (lambda: mmq.rope(x, i3, f.cpu()), "freqs is on"), (lambda: mmq.rope(x.to(torch.int8), i3, f), "expected"),
        (lambda: mmq.rope(x, i3, f, out=x[:2]), "out"), (lambda: mmq.rope(x, i3, f, dtype=F32, out=x), "out"),
        (lambda: mmq.rope(x.transpose(1, 2), i3, f), "adjacent"), (lambda: mmq.rope(x, i3, f, out=x[:1].expand(3, 2, 64)), "overlap"),
        (lambda: mmq.kv_write(x, x[:2], cache, i3), "v:"), (lambda: mmq.kv_write(x, x.half(), cache, i3), "v:"),
        (lambda: mmq.kv_write(x[:, :1], x[:, :1], cache, i3), "heads"), (lambda: mmq.kv_write(x, x, cache[:, :, :-8], i3), "cache"),
        (lambda: mmq.kv_write(x, x, cache, i3[:1]), "slots"), (lambda: mmq.kv_write(x, x, cache, i3, freqs=f), "positions"),
        (lambda: mmq.kv_write(x, x, cache, i3, positions=i3), "positions"),
        (lambda: mmq.kv_read(cache, i3, 128), "cache"), (lambda: mmq.kv_read(cache, i3, 64, dtype=F32, k=x), "k:"),
        (lambda: mmq.attention_i8(x.float(), cache, table, lens, off), "bf16 or fp16"),
        (lambda: mmq.attention_i8(x, cache, table[0], lens, off), "page_table"),
        (lambda: mmq.attention_i8(x, cache, table.long(), lens, off), "page_table"),
        (lambda: mmq.attention_i8(x, cache, table, lens, off[:1]), "q_offsets"),
        (lambda: mmq.attention_i8(x, cache, table, lens.long(), off), "lens"),
        (lambda: mmq.attention_i8(x[:, :1], cache, table, lens, off), "multiple"),
        (lambda: mmq.attention_i8(x, cache, table, lens, off, dtype=F16), "queries' type"),
        (lambda: mmq.attention_i8(x, cache, table, lens, off, workspace=lens), "workspace"),
    ]
    for call, why in calls:
        with pytest.raises((ValueError, mmq.MMQError), match=why):
            call()
    k, v = mmq.kv_read(cache, i3, 64, k=torch.empty((3, 2, 64), dtype=F16, device=DEV))      # the type of the output given
    assert k.dtype == v.dtype == F16
    need = mmq.attention_workspace_bytes(1, 1, 1, 2, 2, 64, 64, 16)
    assert need > 0
    long = torch.zeros((1, 64), dtype=torch.int32, device=DEV)
    with pytest.raises(mmq.MMQError, match="workspace of"):
        mmq.attention_i8(x[:1], cache, long, lens, off[[0, 1]], workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
