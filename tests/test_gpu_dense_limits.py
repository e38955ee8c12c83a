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


def test_q8_first_moment_next_to_zero():
    """Code 1 stands for 2^-18 of the scale and begins at 0.5625 of that."""
    one = 2.0 ** -18
    m, scale, _, _ = q8_of([1.0, 0.5 * one, 0.56 * one, 0.565 * one, one, -0.56 * one, -0.565 * one, -one])
    assert scale == [1.0] and [c & 127 for c in m] == [127, 0, 0, 1, 1, 0, 1, 1]
    assert [c >> 7 for c in m[6:]] == [1, 1]


def test_q8_blocks_below_the_least_scale_are_zeros():
    least = 2.0 ** -60  # its square is 2^-120
    for g, want in ((least, [255, least ** 2]), (-least, [255, least ** 2]), (0.99 * least, [0, 0.0])):
        m, m_scale, v, v_scale = q8_of([g] + [0.0] * 300)
        assert [v[0], v_scale[0]] == want and v[1:] == [0] * 300 and v_scale[1] == 0.0
        assert m[0] & 127 == 127 and m_scale == [abs(torch.tensor(g).item()), 0.0]


def test_adamw_second_moments_below_the_least_root():
    """eps = 0 and a second moment that fp32 has lost: its root counts as 2^-63, and the step is finite."""
    g = torch.tensor([2.0 ** -80, 2.0 ** -70, 0.0], device="cuda")
    p = torch.zeros(3, device="cuda")
    DenseAdamW([p], [g], weight_decay=0.0, betas=(0.0, 0.0), eps=0.0).step(1.0)
    assert p.tolist() == pytest.approx([-2.0 ** -17, -2.0 ** -7, 0.0], rel=2.0 ** -19, abs=0)
