"""Layer norm where it once went wrong: column offsets that are not the widths'."""
import os
import subprocess

import pytest
import torch

from bwd_tbe_fwd_gb300 import LayerNorm
from bwd_tbe_fwd_gb300 import build as tbe_build

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
