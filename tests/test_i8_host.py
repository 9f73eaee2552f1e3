"""The per-token / per-channel int8 operators without a GPU: what their entry
points refuse (before any device work) and what the planner picks.  The
pointers handed in are never read: every refusal here is decided from the
arguments, and a call whose arguments are fine ends at the device query."""
import ctypes
import re

import pytest
import torch

import block_quantized_int8_q8_amd as mmq

OK = 1 << 20          # an address that is aligned to anything; never read
p = ctypes.c_void_p


def quantize(type=0, x=OK, ldx=64, q=OK, ldq=64, scale=OK, M=4, K=64):
    return mmq.lib().mmq_quantize_i8(type, p(x), ldx, p(q), ldq, p(scale), M, K, None)


def silu(type=0, gate=OK, up=OK, ld=64, q=OK, ldq=64, scale=OK, M=4, K=64):
    return mmq.lib().mmq_silu_mul_quantize_i8(type, p(gate), p(up), ld, p(q), ldq, p(scale), M, K, None)


def gemm(type=0, x=OK, ldx=64, xs=OK, w=OK, ldw=64, ws=OK, bias=None, out=OK, ldo=32, M=4, N=32, K=64):
    return mmq.lib().mmq_gemm_i8(type, p(x), ldx, p(xs), p(w), ldw, p(ws), p(bias), p(out), ldo, M, N, K, None)


def grouped(type=0, x=OK, ldx=64, xs=OK, T=4, rows=None, offsets=OK, E=3, w=OK, ldw=64, ws=OK, out=OK, ldo=32, R=4,
            N=32, K=64):
    return mmq.lib().mmq_grouped_gemm_i8(type, p(x), ldx, p(xs), T, p(rows), p(offsets), E, p(w), ldw, p(ws), p(out),
                                         ldo, R, N, K, None)


CALLS = {
    "quantize": (quantize, [
        (dict(type=3), "type"), (dict(M=-1), "M must"), (dict(K=0), "K >= 1"), (dict(K=131057, ldx=1 << 18, ldq=1 << 18), "131056"),
        (dict(ldx=63), "shorter"), (dict(ldq=48), "pitch"), (dict(ldq=72), "pitch"), (dict(K=65, ldx=65, ldq=64), "pitch"),
        (dict(ldq=(1 << 22) + 16), "2^22"), (dict(M=1 << 31), "2^31"), (dict(x=None), "null"), (dict(q=None), "null"),
        (dict(scale=None), "null"), (dict(x=OK + 2), "aligned"), (dict(type=1, x=OK + 1), "aligned"),
        (dict(q=OK + 8), "16-byte"), (dict(scale=OK + 2), "4-byte")]),
    "silu": (silu, [
        (dict(type=-1), "type"), (dict(K=0), "K >= 1"), (dict(up=None), "null"), (dict(gate=None), "null"),
        (dict(up=OK + 2), "aligned"), (dict(ld=10), "shorter"), (dict(q=OK + 4), "16-byte")]),
    "gemm": (gemm, [
        (dict(type=9), "type"), (dict(M=-2), "M must"), (dict(N=0), "N and K"), (dict(K=0), "N and K"),
        (dict(K=56), "multiple of 16"), (dict(K=131072, ldx=131072, ldw=131072), "131056"), (dict(ldx=48), "pitch"),
        (dict(ldw=48), "pitch"), (dict(ldx=72), "pitch"), (dict(ldw=72), "pitch"), (dict(ldx=1 << 23), "2^22"),
        (dict(ldo=31), "shorter"), (dict(x=None), "null"), (dict(xs=None), "null"), (dict(w=None), "null"),
        (dict(ws=None), "null"), (dict(out=None), "null"), (dict(x=OK + 8), "16-byte"), (dict(w=OK + 4), "16-byte"),
        (dict(xs=OK + 1), "4-byte"), (dict(bias=OK + 2), "4-byte"), (dict(out=OK + 2), "output"),
        (dict(type=1, out=OK + 1), "output"), (dict(M=1 << 31), "2^31"), (dict(N=1 << 31, ldo=1 << 31), "2^31")]),
    "grouped": (grouped, [
        (dict(E=0), "n_experts"), (dict(E=2049), "n_experts"), (dict(T=-1), "T must"), (dict(T=3), "no row index"),
        (dict(T=0, rows=OK), "gather"), (dict(offsets=None), "null"), (dict(offsets=OK + 2), "4-byte"),
        (dict(rows=OK + 1), "4-byte"), (dict(K=40), "multiple of 16"), (dict(R=-1), "M must"), (dict(w=None), "null"),
        (dict(type=3), "type"), (dict(ldo=8), "shorter"), (dict(T=1 << 20, ldx=1 << 16, rows=OK), "4 GiB")]),
}
REFUSALS = [(n, kw, why) for n, (_, cases) in CALLS.items() for kw, why in cases]


@pytest.mark.parametrize("name,kw,why", REFUSALS, ids=[f"{n}-{'-'.join(k)}-{i}" for i, (n, k, _) in enumerate(REFUSALS)])
def test_refused_before_any_device_work(name, kw, why):
    assert CALLS[name][0](**kw) == 0
    assert why in mmq.last_error(), mmq.last_error()


@pytest.mark.parametrize("name,kw", [("quantize", dict(M=0, x=None, q=None, scale=None)), ("silu", dict(M=0)),
                                     ("gemm", dict(M=0, x=None, out=None)),
                                     ("grouped", dict(R=0, T=0, rows=None)), ("grouped", dict(R=0, T=5, rows=OK))])
def test_no_rows_is_nothing_to_do(name, kw):
    assert CALLS[name][0](**kw) == 1
    assert mmq.last_error() == ""


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on the dummy pointers")
@pytest.mark.parametrize("name", list(CALLS))
def test_good_arguments_reach_the_device_query(name):
    assert CALLS[name][0]() == 0
    assert "device" in mmq.last_error()


def plan(M, N, K, E=0, cus=256):
    ok, desc = mmq.plan_i8(M, N, K, E, cus)
    assert ok, desc
    return desc


@pytest.mark.parametrize("M,N,K,E,why", [(1, 1, 24, 0, "multiple of 16"), (-1, 1, 16, 0, "M must"), (1, 0, 16, 0, "N and K"),
                                         (1, 1, 131072, 0, "131056"), (1, 1, 16, 2049, "n_experts"),
                                         (1, 1, 16, -1, "n_experts"), ((1 << 31) - 1, (1 << 31) - 1, 16, 0, "tiles")])
def test_plan_refusals(M, N, K, E, why):
    ok, desc = mmq.plan_i8(M, N, K, E, 256)
    assert not ok and why in desc
    assert not mmq.plan_i8(64, 64, 64, 0, 0)[0]


@pytest.mark.parametrize("M,N,why", [((1 << 31) - 100, 8, "2^31 rows"), (16, (1 << 31) - 100, "2^32"), (16, 1 << 30, "2^32")])
def test_plan_refuses_what_a_launch_cannot_hold(M, N, why):
    ok, desc = mmq.plan_i8(M, N, 16, 0, 256)
    assert not ok and why in desc, desc


@pytest.mark.parametrize("E", [0, 1, 5, 128, 2048])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 3584), (8, 1536), (13, 18944), (64, 512), (65, 65), (509, 4608), (2048, 3584),
                                 (8192, 18944), (12008, 2048), (16384, 1536)])
def test_plan_grid_covers_every_grouping(M, N, E):
    """The grid holds a tile for every row and column however the rows are
    grouped: with E experts at most min(E, M) groups have a partial tile, and
    a grouping into full tiles plus such remainders needs no more than
    M / tile_m + min(E, M) (rounded down) of them."""
    d = plan(M, N, 3584, E)
    tile_m, tile_n = map(int, re.search(r"tile=(\d+)x(\d+)", d).groups())
    tiles_m, tiles_n = map(int, re.search(r"tiles=(\d+)x(\d+)", d).groups())
    assert tiles_n * tile_n >= N > (tiles_n - 1) * tile_n
    if E == 0:
        assert tiles_m * tile_m >= M > (tiles_m - 1) * tile_m
    else:
        worst = max(sum(-(-n // tile_m) for n in split) for split in _groupings(M, E, tile_m))
        assert worst <= tiles_m <= M // tile_m + min(E, M)


def _groupings(M, E, tile):
    yield [M]
    g = min(E, M)
    yield [M - (g - 1)] + [1] * (g - 1)
    yield [M // g + (i < M % g) for i in range(g)]
    one, rest = (tile + 1, M) if M > tile else (1, M)
    s = []
    while rest > 0 and len(s) < E - 1:
        s.append(min(one, rest))
        rest -= s[-1]
    yield s + ([rest] if rest else [])
