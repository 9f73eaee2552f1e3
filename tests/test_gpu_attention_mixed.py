"""Decoding sequences of long contexts beside prompts, against 64 bits."""
import pytest

from tests.test_gpu_attention import BF16, F16, Batch
from tests.test_gpu_attention_scales import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D", [([300, 1], [300, 70001], 8, 2, 128), ([1, 260, 1, 2], [8192, 260, 33000, 500], 8, 2, 64),
                                               ([600, 1, 1], [600, 12345, 20], 4, 2, 256)])
def test_long_decodes_beside_a_prompt(new, lens, Hq, Hkv, D, t):
    bt = Batch(new, lens, Hq, Hkv, D, 128, t, seed=61)
    out = bt.run()
    check(bt, out)
    assert bool((bt.run(max_q=max(new)) == out).all())
