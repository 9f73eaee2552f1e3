"""What the bits of an attention row may depend on: its own query, what it sees
of the cache, and the batch's lengths; not on when other workgroups run."""
import pytest
import torch

from tests.test_gpu_attention import BF16, F16, Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D", [([1500], [1500], 28, 4, 128), ([1203], [1203], 24, 4, 64), ([777], [777], 12, 2, 256),
                                               ([900, 1, 333], [900, 700, 4000], 28, 4, 128)])
def test_output_over_the_queries_whenever_its_workgroups_run(new, lens, Hq, Hkv, D, t):
    """A last tile of rows that is not full, in several shares that start when the sequence's first rows may have their
    outputs already; scores to hundreds, so that references move in most steps."""
    bt = Batch(new, lens, Hq, Hkv, D, 16, t, seed=31, qscale=40.0)
    q = bt.q.clone()
    want = bt.run()
    for _ in range(20):
        bt.q.copy_(q)
        bt.run(out=bt.q)
        assert torch.equal(bt.q, want)


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D", [([1], [3000], 8, 1, 128), ([1] * 220, [400] * 220, 28, 4, 64),
                                               ([3, 1], [900, 2500], 8, 1, 64), ([1], [700], 32, 1, 256),
                                               ([150], [900], 4, 1, 128), ([200], [200], 8, 2, 64), ([90], [700], 4, 1, 256)])
def test_a_row_does_not_depend_on_the_other_rows_queries(new, lens, Hq, Hkv, D, t):
    """Rows of a wave share its products, and one whose scores rise makes the wave rescale: every third row's query is
    made forty times as large, and the others keep their bits."""
    bt = Batch(new, lens, Hq, Hkv, D, 16, t, seed=32)
    want = bt.run().clone()
    rows = torch.arange(bt.q.shape[0] * Hq, device=bt.q.device).view(bt.q.shape[:2])
    loud = rows % 3 == 1
    bt.q[loud] *= 40.0
    assert torch.equal(bt.run()[~loud], want[~loud])
