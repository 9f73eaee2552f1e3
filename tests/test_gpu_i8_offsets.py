"""Grouped int8 products whose offsets decrease: a group starts where the
furthest group before it ended, on every kernel alike, so that a row belongs
to one group at most.  Results are compared bit for bit with the groups of
that rule, rows of no group with what was there."""
import pytest
import torch

import block_quantized_int8_q8_amd as mmq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# rows, columns, experts, and the kernel that multiplies them
SHAPES = [(60, 70, 5, "rows tile=16x16"), (60, 1100, 130, "rows tile=16x32"), (3000, 70, 5, "rows tile=32x32"),
          (3000, 70, 130, "rows tile=32x64"), (3400, 197, 3, "rows tile=64x64"), (1500, 1100, 5, "tile tile=64x128"),
          (400, 1100, 40, "tile tile=64x128"), (3000, 2100, 40, "tile tile=128x128"), (5000, 4100, 5, "tile tile=128x256"),
          (3000, 1100, 40, "tile tile=128x256"), (5000, 2100, 5, "tile tile=256x256"), (12000, 2100, 700, "tile tile=")]


def groups_of(offsets, R):
    """(expert, first row, end) by the rule."""
    at = min(max(offsets[0], 0), R)
    for e, o in enumerate(offsets[1:]):
        o = min(max(o, 0), R)
        if o > at:
            yield e, at, o
            at = o


def offsets_of(kind, E, R, gen):
    off = torch.cat([torch.zeros(1), torch.rand(E, generator=gen).sort().values * R]).long()
    off[-1] = R
    if kind == "dip":                      # the last groups start again near the front
        off[-2] = R // 5
        off[1] = R // 2
    elif kind == "swapped":
        for i in torch.randint(1, E, (max(1, E // 8),), generator=gen).tolist():
            off[i], off[i + 1] = off[i + 1].item(), off[i].item()
    elif kind == "random":
        off = torch.randint(-R // 4, R + R // 4, (E + 1,), generator=gen)
    elif kind == "falling":
        off = off.flip(0)
    return off


@pytest.mark.parametrize("gather", [False, True], ids=["inplace", "gather"])
@pytest.mark.parametrize("kind", ["dip", "swapped", "random", "falling"])
@pytest.mark.parametrize("R,N,E,kernel", SHAPES)
def test_decreasing_offsets_keep_groups_disjoint(R, N, E, kernel, kind, gather):
    K = 208
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert f"kernel={kernel}" in mmq.plan_i8(R, N, K, E, cus)[1]
    gen = torch.Generator().manual_seed(R + N + E)
    off = offsets_of(kind, E, R, gen)
    T = max(1, R // 3) if gather else R
    xq = torch.randint(-128, 128, (T, K), generator=gen, dtype=torch.int8).to(DEV)
    wq = torch.randint(-128, 128, (E, N, K), generator=gen, dtype=torch.int8).to(DEV)
    xs, ws = (torch.rand(T, generator=gen) + 0.5).to(DEV), (torch.rand((E, N), generator=gen) + 0.5).to(DEV)
    rows = torch.randint(0, T, (R,), generator=gen, dtype=torch.int32).to(DEV) if gather else None
    out = torch.full((R, N), -5.0, device=DEV)
    mmq.grouped_gemm_i8(xq, xs, wq, ws, off.to(torch.int32).to(DEV), rows=rows, out=out)
    src = torch.arange(R, device=DEV) if rows is None else rows.long()
    want = torch.full((R, N), -5.0, device=DEV)
    for e, a, b in groups_of(off.tolist(), R):
        t = src[a:b]
        acc = torch.matmul(xq[t].double(), wq[e].double().t())            # integers below 2^53: exact
        want[a:b] = acc.float() * xs[t][:, None] * ws[e]
    assert torch.equal(out, want)
