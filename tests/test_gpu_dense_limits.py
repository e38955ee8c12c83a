"""Where the dense side's arithmetic ends, as include/tbe_dense.h states it."""
import math

import pytest
import torch

from bwd_tbe_fwd_gb300 import GradNorm
from test_gpu_dense import DT, host

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------
# Gradient norm: squares in fp32
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grad_norm_of_gradients_at_fp32s_ends(dtype):
    def norm(value):
        t = torch.zeros(3000, dtype=DT[dtype], device="cuda")
        t[1234] = value
        return host(GradNorm([t]).compute(1.0))

    assert math.isinf(norm(2.0 ** 64)[0])
    assert norm(2.0 ** 63)[0] == 2.0 ** 63
    assert norm(2.0 ** -74)[0] == 2.0 ** -74  # its square is an fp32 value still
    assert norm(2.0 ** -76).tolist() == [0.0, 1.0]
