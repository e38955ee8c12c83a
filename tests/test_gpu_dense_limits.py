"""Where the dense side's arithmetic ends, as include/tbe_dense.h states it."""
import math

import pytest
import torch

from bwd_tbe_fwd_gb300 import DenseAdamW, GradNorm
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


# ------------------------------------------------------------------------------------------
# 8-bit states: betas of 0 make the moments the gradient and its square
# ------------------------------------------------------------------------------------------
def q8_of(gradients):
    g = torch.tensor(gradients, device="cuda")
    opt = DenseAdamW([torch.zeros_like(g)], [g], "q8", weight_decay=0.0, betas=(0.0, 0.0))
    opt.step(1e-3)
    return [t[0].tolist() for t in (opt.exp_avg, opt.exp_avg_scale, opt.exp_avg_sq, opt.exp_avg_sq_scale)]


def test_q8_a_positive_second_moment_has_a_code():
    """Also one whose quotient by the block's scale is below fp32."""
    _, _, v, scale = q8_of([2.0 ** 10, 2.0 ** -20, 2.0 ** -60, 2.0 ** -65, 2.0 ** -74, 0.0])
    assert scale == [2.0 ** 20] and v == [255, 1, 1, 1, 1, 0]
