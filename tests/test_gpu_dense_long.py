"""The dense side's longer walks, against the formulas in 64 bits: chunks of several passes of AdamW and of the gradients'
norm, and layer norm backward with more rows to a CTA than one batch of statistics holds.  Sizes follow from the device's
number of SMs, as the kernels' rules do."""
import math

import numpy as np
import pytest
import torch

import dense_reference as ref
from bwd_tbe_fwd_gb300 import DenseAdamW, GradNorm, LayerNorm
from test_gpu_dense import B1, B2, DT, EPS, check_steps, gen, host, within

pytestmark = pytest.mark.gpu

PASS = 2048  # elements of a CTA's pass over its chunk


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def cuda_gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------------------------------
# Chunks of several passes: of k passes (a power of two, at most 4 or 16) from 16 chunks to an SM on
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("passes", [2, 4])
@pytest.mark.parametrize("p,g,master", [("f32", "f32", False), ("bf16", "bf16", True)])
def test_adamw_chunks_of_several_passes(p, g, master, passes):
    """Tensors that follow one another in flat buffers, each starting off a vector's boundary, some shorter than a pass or
    than a chunk, the last one ragged; two steps."""
    small = [3, 2047, 2049, 4095, 8193, 5 * PASS + 1]
    long = 16 * passes * PASS * sms() + 11
    sizes = [1] + small[:3] + [long // 3] + small[3:] + [long - long // 3, 8 * PASS - 5]
    starts = np.concatenate([[0], np.cumsum(sizes)])
    total = int(starts[-1])
    assert 16 * passes * sms() <= total // PASS < 32 * passes * sms()
    r = cuda_gen(passes)
    flat = dict(master=torch.randn(total, generator=r, device="cuda"), m=0.1 * torch.randn(total, generator=r, device="cuda"),
                v=torch.rand(total, generator=r, device="cuda"))
    flat["params"] = flat["master"].to(DT[p])
    flat["grads"] = torch.randn(total, generator=r, device="cuda").to(DT[g])
    cut = lambda t: [t[a:b] for a, b in zip(starts[:-1], starts[1:])]  # noqa: E731
    s = {k: cut(v) for k, v in flat.items()}
    if not master:
        s["master"] = None
    n = len(sizes)
    decay, scale = [0.1 * (i % 2) for i in range(n)], [1.0 - 0.5 * (i % 2) for i in range(n)]
    opt = DenseAdamW(s["params"], s["grads"], "f32", s["master"], state={"exp_avg": s["m"], "exp_avg_sq": s["v"]},
                     weight_decay=decay, lr_scale=scale, betas=(B1, B2), eps=EPS)
    check_steps(opt, s, p, 2, sizes, decay, scale, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("passes", [1, 2, 16])
def test_grad_norm_chunks_of_several_passes(passes, dtype):
    """A thread's share of a chunk of 16 passes is 128 squares and, where the chunk starts off a 16-byte boundary, one before
    and one after: 130 roundings that a square passes through, and half of their sum in the root; 4 units for the
    conversion and the root."""
    total = 16 * passes * PASS * sms() + 12_345 if passes > 1 else 8 * PASS * sms()
    flat = torch.randn(total + 3, generator=cuda_gen(passes), device="cuda").to(DT[dtype])[3:]
    parts = [flat[:1], flat[1:5], flat[5:total // 2], flat[total // 2:]]
    squares = sum(float(t.double().square().sum()) for t in flat.split(1 << 24))
    want = math.sqrt(squares)
    norm = GradNorm(parts)
    for max_norm in (math.inf, 0.5 * want):
        got = host(norm.compute(max_norm))
        assert abs(got[0] - want) <= (130 / 2 + 4) * ref.U * want
        coef = min(1.0, max_norm / (got[0] + 1e-6))
        assert abs(got[1] - coef) <= 4 * ref.U * coef
    assert torch.equal(norm.compute(1.0), norm.compute(1.0))


# ------------------------------------------------------------------------------------------
# Layer norm backward: many rows to a CTA
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("width", [520, 1024, 2048, 4096, 8192])
@pytest.mark.parametrize("slots", [1, 2])
def test_norm_backward_many_rows_to_a_cta(width, dtype, slots):
    """So many segments that `slots` CTAs share a segment's rows, and rows on either side of one, two and three batches of
    32 to a CTA (the last CTA one fewer).  All segments hold the same columns, so one is checked and the others are
    equal to it."""
    threads = 64
    while 16 * threads < width:
        threads *= 2
    resident = sms() * (512 // threads)  # CTAs that the segments share
    segments = resident // (slots + 1) + 1
    assert resident // segments == slots
    ln = LayerNorm([width] * segments, DT[dtype])
    r = gen(width)
    weight = 1 + 0.3 * torch.randn(width, generator=r)
    for k in (31, 32, 33, 63, 64, 65, 96, 97):
        rows = slots * k - (slots - 1)
        x = (torch.randn(rows, width, generator=r) + torch.randn(rows, 1, generator=r)).to(DT[dtype])
        dy = torch.randn(rows, width, generator=r).to(DT[dtype])
        (_, mean, rstd), _ = ref.layer_norm(host(x), [width], None, None, 1e-5)
        mean, rstd = torch.from_numpy(mean).float(), torch.from_numpy(rstd).float()
        wide = lambda t: t.cuda().repeat(1, segments)  # noqa: E731
        dx, dw, db = ln.backward(wide(dy), wide(x), wide(mean), wide(rstd), weight.cuda().repeat(segments))
        want, bound = ref.layer_norm_gradients(host(dy), host(x), host(mean), host(rstd), [width], host(weight), dtype)
        for got, v, b, name in zip((dx, dw[None], db[None]), want, bound, ("dx", "dweight", "dbias")):
            within(got[:, :width], v, b, f"{name}, {rows} rows")
            assert bool((got.view(got.shape[0], segments, width) == got[:, None, :width]).all())
