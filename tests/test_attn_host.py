"""The rotary, cache and attention entry points without a GPU: what they refuse
(before any device work), what the plan says, and what the binding refuses.
The pointers handed in are never read: every refusal here is decided from the
arguments, and a call whose arguments are fine ends at the device query."""
import ctypes
import math

import pytest
import torch

import block_quantized_int8_q8_amd as mmq

OK = 1 << 20          # an address that is aligned to anything; never read
p = ctypes.c_void_p
nan = float("nan")


def frequencies(scaling=0, rot=64, base=1e4, factor=2.0, low=1.0, high=4.0, original=4096, null=False):
    f, m = (ctypes.c_double * 256)(), ctypes.c_double()
    return mmq.lib().mmq_rope_frequencies(scaling, rot, base, factor, low, high, original, None if null else f, ctypes.byref(m))


def rope(type=0, x=OK, ldt=512, ldh=64, out_type=0, out=2 * OK, odt=512, odh=64, pos=OK, freqs=OK, rot=64, layout=0, mscale=1.0,
         inverse=0, T=4, H=8, D=64):
    return mmq.lib().mmq_rope(type, p(x), ldt, ldh, out_type, p(out), odt, odh, p(pos), p(freqs), rot, layout, mscale, inverse, T, H,
                              D, None)


def write(type=0, k=OK, kdt=512, kdh=64, v=OK, vdt=512, vdh=64, pos=OK, freqs=OK, rot=64, layout=0, mscale=1.0, slots=OK, T=4,
          cache=OK, n_pages=8, page=16, H=8, D=64):
    return mmq.lib().mmq_kv_write(type, p(k), kdt, kdh, p(v), vdt, vdh, p(pos), p(freqs), rot, layout, mscale, p(slots), T, p(cache),
                                  n_pages, page, H, D, None)


def read(type=0, cache=OK, n_pages=8, page=16, H=8, D=64, slots=OK, T=4, k=OK, kdt=512, kdh=64, v=OK, vdt=512, vdh=64):
    return mmq.lib().mmq_kv_read(type, p(cache), n_pages, page, H, D, p(slots), T, p(k), kdt, kdh, p(v), vdt, vdh, None)


def attention(type=1, q=OK, qdt=512, qdh=64, cache=OK, n_pages=8, page=16, table=OK, max_pages=4, lens=OK, offsets=OK, B=2, T=4,
              max_q=4, Hq=8, Hkv=2, D=64, scale=0.1, window=0, out_type=1, out=2 * OK, odt=512, odh=64, ws=OK, wn=1 << 40):
    return mmq.lib().mmq_attention_i8(type, p(q), qdt, qdh, p(cache), n_pages, page, p(table), max_pages, p(lens), p(offsets), B, T,
                                      max_q, Hq, Hkv, D, scale, window, out_type, p(out), odt, odh, p(ws), wn, None)


CALLS = {
    "frequencies": (frequencies, [
        (dict(scaling=4), "scaling"), (dict(scaling=-1), "scaling"), (dict(rot=3), "even"), (dict(rot=0), "even"),
        (dict(rot=514), "even"), (dict(base=1.0), "base"), (dict(base=nan), "base"), (dict(base=math.inf), "base"),
        (dict(scaling=1, factor=0.0), "factor"), (dict(scaling=1, factor=nan), "factor"), (dict(scaling=2, low=0.0), "low"),
        (dict(scaling=2, low=4.0), "low"), (dict(scaling=3, high=math.inf), "low"), (dict(scaling=3, original=0), "original"),
        (dict(null=True), "null")]),
    "rope": (rope, [
        (dict(type=3), "type"), (dict(out_type=-1), "type"), (dict(T=-1), "tokens"), (dict(T=(1 << 24) + 1), "tokens"),
        (dict(H=0), "heads"), (dict(H=1025), "heads"), (dict(D=60), "multiple of 8"), (dict(D=520), "multiple of 8"),
        (dict(D=0), "multiple of 8"), (dict(rot=66), "even"), (dict(rot=7), "even"), (dict(rot=0), "even"), (dict(layout=2), "layout"),
        (dict(ldt=-1), "strides"), (dict(ldh=1 << 41), "strides"), (dict(odh=63), "overlap"), (dict(odt=511), "overlap"),
        (dict(odt=0), "overlap"), (dict(x=None), "null"), (dict(out=None), "null"), (dict(pos=None), "null"),
        (dict(freqs=None), "null"), (dict(x=OK + 2), "aligned"), (dict(out_type=1, out=OK + 1), "aligned"), (dict(pos=OK + 2), "aligned"),
        (dict(freqs=OK + 4), "aligned"), (dict(mscale=nan), "mscale"), (dict(mscale=math.inf), "mscale"),
        (dict(out=OK, out_type=1), "in place"), (dict(out=OK, odt=1024), "in place")]),
    "write": (write, [
        (dict(type=7), "type"), (dict(D=96), "64, 128 or 256"), (dict(page=48), "16, 32, 64, 128 or 256"), (dict(page=8), "16, 32"),
        (dict(H=0), "heads"), (dict(H=2000), "heads"), (dict(n_pages=0), "tokens"), (dict(n_pages=1 << 27), "tokens"),
        (dict(n_pages=1 << 24, page=64, H=64), "tiles"), (dict(T=-3), "tokens"), (dict(kdt=-1), "strides"), (dict(vdh=-1), "strides"),
        (dict(k=None), "null"), (dict(v=None), "null"), (dict(slots=None), "null"), (dict(cache=None), "null"),
        (dict(pos=None), "null"), (dict(rot=65), "even"), (dict(layout=5), "layout"), (dict(mscale=nan), "mscale"),
        (dict(k=OK + 2), "aligned"), (dict(type=1, v=OK + 1), "aligned"), (dict(slots=OK + 2), "aligned"), (dict(cache=OK + 8), "aligned")]),
    "read": (read, [
        (dict(type=-2), "type"), (dict(D=32), "64, 128 or 256"), (dict(page=512), "16, 32"), (dict(T=1 << 25), "tokens"),
        (dict(kdt=511), "overlap"), (dict(vdh=8), "overlap"), (dict(k=None), "null"), (dict(v=None), "null"), (dict(cache=None), "null"),
        (dict(slots=None), "null"), (dict(v=OK + 2), "aligned"), (dict(cache=OK + 4), "aligned")]),
    "attention": (attention, [
        (dict(type=0), "bf16 or fp16"), (dict(out_type=2), "queries' type"), (dict(T=-1), "tokens"), (dict(T=1 << 24, Hq=128), "2^30"),
        (dict(Hq=7), "multiple"), (dict(Hkv=0), "multiple"), (dict(Hq=0), "heads"), (dict(D=80), "64, 128 or 256"),
        (dict(page=24), "16, 32"), (dict(B=-1), "sequences"), (dict(B=1 << 21), "sequences"), (dict(max_pages=-1), "2^30"),
        (dict(max_pages=1 << 27), "2^30"), (dict(max_q=0), "max_q"), (dict(n_pages=0), "tokens"), (dict(qdt=-4), "strides"),
        (dict(odt=500), "overlap"), (dict(scale=nan), "scale"), (dict(scale=math.inf), "scale"), (dict(window=-1), "window"),
        (dict(q=None), "null"), (dict(cache=None), "null"), (dict(table=None), "null"), (dict(lens=None), "null"),
        (dict(offsets=None), "null"), (dict(out=None), "null"), (dict(q=OK + 1), "aligned"), (dict(out_type=0, out=OK + 2), "aligned"),
        (dict(cache=OK + 8), "aligned"), (dict(lens=OK + 2), "aligned"), (dict(table=OK + 1), "aligned"), (dict(offsets=OK + 3), "aligned"),
        (dict(out=OK, out_type=0), "in place"), (dict(out=OK, odt=1024), "in place"), (dict(out=OK, odh=64, odt=640), "in place")]),
}
REFUSALS = [(n, kw, why) for n, (_, cases) in CALLS.items() for kw, why in cases]


@pytest.mark.parametrize("name,kw,why", REFUSALS, ids=[f"{n}-{'-'.join(k)}-{i}" for i, (n, k, _) in enumerate(REFUSALS)])
def test_refused_before_any_device_work(name, kw, why):
    assert CALLS[name][0](**kw) == 0
    assert why in mmq.last_error(), mmq.last_error()


@pytest.mark.parametrize("name,kw", [("rope", dict(T=0, x=None, out=None)), ("write", dict(T=0, k=None, slots=None)),
                                     ("read", dict(T=0, k=None)), ("attention", dict(T=0, q=None, out=None)),
                                     ("attention", dict(B=0, lens=None, table=None))])
def test_nothing_to_do(name, kw):
    assert CALLS[name][0](**kw) == 1
    assert mmq.last_error() == ""


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on the dummy pointers")
@pytest.mark.parametrize("name", ["rope", "write", "read", "attention"])
def test_good_arguments_reach_the_device_query(name):
    assert CALLS[name][0]() == 0
    assert "device" in mmq.last_error()


def test_transposed_outputs_are_taken_and_overlapping_ones_are_not():
    for kw in (dict(odt=64, odh=256), dict(odt=70, odh=280), dict(T=1, odt=0, odh=64), dict(H=1, odt=64, odh=0)):
        assert rope(x=None, **kw) == 0 and "null" in mmq.last_error()          # the check after the strides'
    for kw in (dict(odt=64, odh=255), dict(odt=64, odh=64), dict(odt=63, odh=512)):
        assert rope(**kw) == 0 and "overlap" in mmq.last_error()


def test_cache_bytes():
    assert mmq.kv_cache_bytes(10, 64, 4, 128) == 10 * 64 * 4 * 264
    assert mmq.kv_cache_bytes(3, 16, 1, 64) == 3 * 16 * 136
    for bad in ((0, 16, 1, 64), (1, 17, 1, 64), (1, 16, 0, 64), (1, 16, 1, 100)):
        with pytest.raises(mmq.MMQError):
            mmq.kv_cache_bytes(*bad)
    c = mmq.kv_cache(3, 32, 2, 64, device="cpu")
    assert c.shape == (3, 2, 32 * 136) and c.numel() == mmq.kv_cache_bytes(3, 32, 2, 64)


def test_frequencies_need_no_device():
    f, m = mmq.rope_frequencies(8, base=16.0)
    assert m == 1.0 and torch.allclose(f, torch.tensor([1.0, 0.5, 0.25, 0.125], dtype=torch.float64), rtol=1e-15, atol=0)
    f, m = mmq.rope_frequencies(8, base=16.0, scaling="linear", factor=4.0)
    assert torch.allclose(f, torch.tensor([0.25, 0.125, 0.0625, 0.03125], dtype=torch.float64), rtol=1e-15, atol=0)
    # one turn or fewer within 64 positions: divided; four or more: kept
    f, m = mmq.rope_frequencies(4, base=1e4, scaling="bands", factor=8.0, original=64)
    assert math.isclose(f[0], 1.0, rel_tol=1e-15) and math.isclose(f[1], 0.01 / 8, rel_tol=1e-14)
    with pytest.raises(ValueError):
        mmq.rope_frequencies(8, scaling="other")
    with pytest.raises(mmq.MMQError):
        mmq.rope_frequencies(8, scaling="yarn", factor=2.0)          # no original length


def test_binding_wants_gpu_tensors():
    x, i = torch.zeros(2, 2, 64), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: mmq.rope(x, i, torch.ones(32, dtype=torch.float64)), lambda: mmq.kv_write(x, x, x, i),
                 lambda: mmq.kv_read(torch.zeros(1, 1, 16 * 136, dtype=torch.uint8), i, 64),
                 lambda: mmq.attention_i8(x.half(), x, x, i, i)):
        with pytest.raises(ValueError, match="GPU"):
            call()
