"""The token side (include/tbe_tokens.h) where it once went wrong, or where no test had looked."""
import pytest
import torch

from bwd_tbe_fwd_gb300 import SoftmaxLoss
from test_gpu_tokens import check_loss, loss_inputs

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------
# The end of a product
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dim", [8, 64, 72, 200, 328, 384, 392, 520, 776])
@pytest.mark.parametrize("tokens", [20, 100, 300])
def test_products_that_end_anywhere_in_the_ring(tokens, dim):
    """1 to 13 stages to a tile, tiles in one and several turns: the waits at a product's end are for phases that come."""
    check_loss(tokens, 500, dim, "bf16", seed=dim)


def test_products_one_after_the_other():
    """Short products back to back, each of whose CTAs starts as those of the one before end."""
    h, w, t, _ = loss_inputs(140, 700, 72, "bf16", seed=1)
    op = SoftmaxLoss(700, 72, 140)
    want = None
    for _ in range(200):
        loss, lse, mean = op.forward(h, w, t)
        got = [loss, *op.backward(h, w, t, lse, mean=mean)]
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not op.stats.any()
