"""How many bits attention's weights keep, against the definition in 64 bits:
two parts of q's type for fp32 outputs and for sequences of few rows, one for
16-bit outputs of longer ones.  The bound is derived in
tests/test_gpu_attention_scales.py."""
import pytest
import torch

from tests.test_gpu_attention import BF16, F16, F32, Batch
from tests.test_gpu_attention_scales import check

pytestmark = pytest.mark.gpu

FEW = [([1], [2]), ([1], [5]), ([1], [700]), ([1, 1, 2], [33, 4000, 3])]
MANY = [([40], [41]), ([70], [300]), ([5, 1, 40], [900, 3, 2500])]


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 28, 4), (256, 16, 1)])
@pytest.mark.parametrize("new,lens", FEW + MANY)
def test_fp32_outputs(new, lens, D, Hq, Hkv, t):
    bt = Batch(new, lens, Hq, Hkv, D, 16, t, seed=51)
    check(bt, bt.run(dtype=F32), parts=2)


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 28, 4), (256, 16, 1)])
@pytest.mark.parametrize("new,lens", FEW)
def test_outputs_of_few_rows(new, lens, D, Hq, Hkv, t):
    bt = Batch(new, lens, Hq, Hkv, D, 16, t, seed=52)
    check(bt, bt.run(max_q=max(new)), parts=2)


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
def test_a_wider_output_rounds_to_the_narrow_one_where_rows_are_few(D, t):
    bt = Batch([1, 1], [900, 40], 8, 2, D, 16, t, seed=53)
    assert torch.equal(bt.run(dtype=F32).to(t), bt.run())
