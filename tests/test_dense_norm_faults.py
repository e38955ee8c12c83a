"""Layer norm where it once went wrong: column offsets that are not the widths', rows of equal values."""
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import dense_reference as ref
from bwd_tbe_fwd_gb300 import LayerNorm
from bwd_tbe_fwd_gb300 import build as tbe_build
from test_gpu_dense import within

HERE = os.path.dirname(os.path.abspath(__file__))
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def test_columns_and_weights_stay_in_the_row_for_any_offsets(tmp_path):
    """The kernels' own index arithmetic, run on the host: no offsets make a segment's columns, or the weights that
    its threads read (those without a column included), leave the row."""
    exe = tmp_path / "norm_spans"
    subprocess.run([tbe_build._nvcc(), *tbe_build.ARCH, "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-I",
                    tbe_build.INCLUDE, "-I", tbe_build.CSRC, os.path.join(HERE, "sanitize", "norm_spans.cu"), "-o", str(exe),
                    "-cudart", "shared"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "spans ok\n", r.stdout[-2000:] + r.stderr[-2000:]


@pytest.mark.gpu
@pytest.mark.parametrize("x,y", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("offsets", [[0, 96, 96, 96], [96, 96, 96, 96], [0, 1 << 30, 1 << 30, -1], [95, 96, 97, 98]])
def test_disagreeing_offsets_with_weights(offsets, x, y):
    """Segments of no columns at the row's end, with weights: the call ends and writes nothing beside the rows."""
    ln = LayerNorm([32, 56, 8], DT[x], DT[y])
    ln.col_offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
    w, b = torch.randn(2, 96, device="cuda").unbind(0)
    rows = torch.randn(50, 96, device="cuda")
    out = torch.full((50, 128), 7.0, device="cuda", dtype=DT[y])
    _, mean, rstd = ln.forward(rows.to(DT[x]), w, b, y=out[:, 16:112])
    assert bool((out[:, :16] == 7).all()) and bool((out[:, 112:] == 7).all())
    dx = torch.full((50, 128), 7.0, device="cuda", dtype=DT[x])
    ln.backward(rows.to(DT[y]), rows.to(DT[x]), mean, rstd, w, dx=dx[:, 16:112])
    torch.cuda.synchronize()
    assert bool((dx[:, :16] == 7).all()) and bool((dx[:, 112:] == 7).all())


# ------------------------------------------------------------------------------------------
# Rows of equal values
# ------------------------------------------------------------------------------------------
VALUES = [0.1, 1000.1, -7.3, 1e-3, 3.0, 0.0, -1e-12, 123456.7, 3e30]  # whose sums of 40007 stay in fp32
TINY = [1e-17, -1e-30, 1e-40]
WIDTHS = [1, 2, 3, 37, 100, 260, 520, 1000, 1001, 3001, 4096, 5001, 8192, 8195, 12001, 16383, 16384, 20000, 40007]
NORM_TYPES = [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16")]


def rows_of(values, width, dtype):
    return torch.tensor(values)[:, None].expand(-1, width).contiguous().to(DT[dtype]).cuda()


def affine(width):
    return torch.randn(2, width, generator=torch.Generator().manual_seed(width)).cuda().unbind(0)


@pytest.mark.gpu
@pytest.mark.parametrize("eps", [1e-5, 0.0])
@pytest.mark.parametrize("x,y", NORM_TYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_equal_values_have_no_xhat(width, x, y, eps):
    """mean is the value, xhat exactly 0 and y the bias, forward and backward, whatever the sum's rounding; eps counts as
    2^-126 at least."""
    values = [v for v in VALUES if x != "f16" or 1e-4 < abs(v) < 60_000 or v == 0]
    rows = rows_of(values, width, x)
    ln = LayerNorm([width], DT[x], DT[y], eps=eps)
    w, b = affine(width)
    out, mean, rstd = ln.forward(rows, w, b)
    assert torch.equal(mean[:, 0], rows[:, 0].float())
    assert torch.equal(out, b.to(DT[y]).expand_as(out))
    want = 1 / math.sqrt(max(float(np.float32(eps)), 2.0 ** -126))
    assert bool(((rstd.double() - want).abs() <= 2 * ref.U * want).all())
    dy = torch.randn(len(values), width, generator=torch.Generator().manual_seed(width)).to(DT[y]).cuda()
    dx, dw, db = ln.backward(dy, rows, mean, rstd, w)
    assert bool((dw == 0).all())
    h = lambda t: t.double().cpu().numpy()  # noqa: E731
    want, bound = ref.layer_norm_gradients(h(dy), h(rows), h(mean), h(rstd), [width], h(w), x)
    within(db[None], want[2][None], bound[2][None], "dbias")
    fits = [k for k, v in enumerate(values) if eps > 0 or (x != "f16" and abs(v) < 2 ** 60)]  # |mean| 2^63 is to stay in fp32
    within(dx[fits], want[0][fits], bound[0][fits], "dx")


@pytest.mark.gpu
@pytest.mark.parametrize("x,y", NORM_TYPES[:3])
@pytest.mark.parametrize("width", WIDTHS)
def test_equal_values_whose_squares_leave_fp32(width, x, y):
    """mean to 2^-18 of the value, and xhat to as much of it times rstd: nothing beside the bias."""
    rows = rows_of(TINY, width, x)
    w, b = affine(width)
    out, mean, rstd = LayerNorm([width], DT[x], DT[y]).forward(rows, w, b)
    v = rows[:, :1].double()
    assert bool(((mean.double() - v).abs() <= 2.0 ** -18 * v.abs() + 2.0 ** -149).all())
    off = 2.0 ** -18 * v.abs() * rstd.double() * w.double().abs()
    assert bool(((out.double() - b.to(DT[y]).double()).abs() <= off + 2.0 ** -24 * b.double().abs() * (y == "f32")).all())


@pytest.mark.gpu
@pytest.mark.parametrize("widths", [[64], [260], [37], [1001], [1, 37, 128], [1024], [3001], [4096], [5001], [20000], [40007]])
@pytest.mark.parametrize("x", ["f32", "f16"])
def test_equal_values_beside_other_rows(widths, x):
    """Rows of equal values between others, more of each than a CTA takes at once: the others keep their bits, and equal
    values in one segment of a row leave its other segments alone."""
    n = sum(widths)
    rows = 3000 if n < 5000 else 700
    g = torch.Generator().manual_seed(n)
    data = torch.randn(rows, n, generator=g).to(DT[x]).cuda()
    w, b = affine(n)
    ln = LayerNorm(widths, DT[x])
    want = ln.forward(data, w, b)
    flat = (torch.rand(rows, len(widths), generator=g) < 0.3).cuda()
    value = torch.randn(rows, len(widths), generator=g).mul_(10).to(DT[x]).cuda()
    spread = lambda t: t.repeat_interleave(torch.tensor(widths, device="cuda"), 1)  # noqa: E731
    mixed = torch.where(spread(flat), spread(value), data)
    y, mean, rstd = ln.forward(mixed, w, b)
    assert torch.equal(y, torch.where(spread(flat), b.to(DT[x]).expand_as(y), want[0]))
    assert torch.equal(mean, torch.where(flat, value.float(), want[1]))
    assert torch.equal(rstd[~flat], want[2][~flat])
    assert torch.equal(ln.forward(mixed, w, b, y=mixed)[0], y)  # in place


@pytest.mark.gpu
@pytest.mark.parametrize("width", [64, 260, 1001, 4096, 20000, 40007])
def test_values_nearly_equal(width):
    """One element a unit in the last place off the others: its deviation is kept, against the formula with eps = 0, where
    the spread alone is the scale.  mean is an fp32 value, at most half a unit (2^-15) off, and the deviations are from it:
    multiples of a unit, whose squares' mean is within 50 roundings and 1 / rstd within 25 and two more."""
    x = torch.full((4, width), 1000.1, device="cuda")
    x[:, width // 2] = torch.nextafter(x[0, 0], torch.tensor(math.inf, device="cuda"))
    y, mean, rstd = LayerNorm([width], eps=0.0).forward(x)
    v = x[0].double().cpu().numpy()
    assert abs(float(mean[0]) - v.mean()) <= 2.0 ** -15
    off = v - float(mean[0])
    rs = 1 / np.sqrt((off * off).mean())
    np.testing.assert_allclose(y.double().cpu().numpy()[0], off * rs, rtol=(25 + width // 2048 + 4) * ref.U, atol=0)
    assert torch.equal(y[0], y[3])
