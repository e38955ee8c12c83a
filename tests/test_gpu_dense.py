"""Layer norm, the gradients' norm and AdamW (include/tbe_dense.h) against their formulas in 64 bits
(tests/dense_reference.py, whose bounds follow from the roundings), at the sizes, strides and values
where they can go wrong."""
import math

import numpy as np
import pytest
import torch

import dense_reference as ref
from bwd_tbe_fwd_gb300 import DenseAdamW, GradNorm, LayerNorm, TableBatchedEmbedding, TBEError

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def host(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what):
    got = host(got)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside; first at {tuple(np.argwhere(bad)[0])}: "
                           f"{got[bad][0]!r} for {want[bad][0]!r} +- {bound[bad][0]!r}")


# ------------------------------------------------------------------------------------------
# Layer norm
# ------------------------------------------------------------------------------------------
def norm_inputs(rows, widths, x, y, w="f32", pad=0, seed=0, shift=0.5):
    g = gen(seed)
    n = sum(widths)
    full = torch.randn(rows, n + pad, generator=g) + shift * torch.randn(rows, 1, generator=g)
    if rows > 2:
        full[1] = 0.0  # the pooled row of an empty bag
    dy = torch.randn(rows, n + pad, generator=g)
    return dict(x=full.to(DT[x]).cuda()[:, :n], dy=dy.to(DT[y]).cuda()[:, :n],
                weight=(1 + 0.3 * torch.randn(n, generator=g)).to(DT[w]).cuda(),
                bias=(0.3 * torch.randn(n, generator=g)).to(DT[w]).cuda())


def check_norm(rows, widths, x="f32", y="f32", w="f32", pad=0, affine=True, eps=1e-5, seed=0, shift=0.5):
    s = norm_inputs(rows, widths, x, y, w, pad, seed, shift)
    weight, bias = (s["weight"], s["bias"]) if affine else (None, None)
    ln = LayerNorm(widths, DT[x], DT[y], DT[w], eps)
    out = ln.forward(s["x"], weight, bias)
    h = lambda t: None if t is None else host(t)  # noqa: E731
    want, bound = ref.layer_norm(h(s["x"]), widths, h(weight), h(bias), float(np.float32(eps)), y)
    for got, v, b, name in zip(out, want, bound, ("y", "mean", "rstd")):
        within(got, v, b, name)
    mean, rstd = out[1], out[2]
    grads = ln.backward(s["dy"], s["x"], mean, rstd, weight)
    want, bound = ref.layer_norm_gradients(h(s["dy"]), h(s["x"]), h(mean), h(rstd), widths, h(weight), x, w)
    for got, v, b, name in zip(grads, want, bound, ("dx", "dweight", "dbias")):
        within(got, v, b, name)
    return ln, s, out, grads


TYPES = [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("x,y", TYPES)
@pytest.mark.parametrize("width", [4, 32, 100, 128, 513, 1024, 2048, 5000])
def test_norm_types_and_widths(width, x, y):
    check_norm(37, [width], x, y, seed=width)


@pytest.mark.parametrize("width", [1, 2, 3, 7, 31, 33, 63, 65, 127, 129, 255, 257, 511, 1001, 1023, 1025, 2047, 2049, 4095,
                                   4096, 4097, 8191, 8192, 8193, 16383, 16384, 16385, 20000, 40007])
def test_norm_every_width_path(width):
    check_norm(19, [width], seed=width)
    check_norm(5, [width], "bf16", "bf16", seed=width + 1)


@pytest.mark.parametrize("rows", [1, 2, 3, 31, 33, 257, 1000, 4099])
@pytest.mark.parametrize("width", [64, 260, 1536])
def test_norm_rows(rows, width):
    check_norm(rows, [width], seed=rows)


@pytest.mark.parametrize("widths", [[64, 64], [32, 64, 128, 256] * 4, [4, 100, 36, 260], [1024, 4, 512], [1, 2, 3, 5, 8, 13],
                                    [8] * 300, [4096, 8, 1000], [20000, 8, 16]])
@pytest.mark.parametrize("x,y", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_norm_segments(widths, x, y):
    check_norm(67, widths, x, y, seed=len(widths))


@pytest.mark.parametrize("pad", [1, 4, 8, 61])
@pytest.mark.parametrize("x,y", [("f32", "bf16"), ("f16", "f16")])
def test_norm_strided_rows(x, y, pad):
    ln, s, out, _ = check_norm(45, [128, 128], x, y, pad=pad, seed=pad)
    # outputs into views of wider buffers leave the rest alone
    wide = torch.full((45, 256 + pad), 7.0, dtype=DT[y], device="cuda")
    ln.forward(s["x"], s["weight"], s["bias"], y=wide[:, :256])
    assert torch.equal(wide[:, :256], out[0]) and bool((wide[:, 256:] == 7).all())


@pytest.mark.parametrize("w", ["f16", "bf16"])
def test_norm_weight_types_and_none(w):
    check_norm(50, [128, 36], "f32", "f32", w)
    check_norm(50, [1500], "bf16", "bf16", w)
    check_norm(50, [128, 36], affine=False)
    check_norm(50, [9000], affine=False)


def test_norm_misaligned_base():
    buf = torch.randn(1 + 33 * 128, device="cuda")
    x = buf[1:].view(33, 128)
    y, mean, rstd = LayerNorm([128]).forward(x)
    y2, mean2, rstd2 = LayerNorm([128]).forward(x.clone())
    want, bound = ref.layer_norm(host(x), [128], None, None, float(np.float32(1e-5)))
    for got in ((y, mean, rstd), (y2, mean2, rstd2)):
        for v, t, b in zip(got, want, bound):
            within(v, t, b, "misaligned")


@pytest.mark.parametrize("width", [3, 37, 300, 1001, 3001])
@pytest.mark.parametrize("offset", [1, 5, 7])
def test_norm_odd_rows_from_anywhere(width, offset):
    """Rows of an odd width that start at any element of a buffer: nothing around them is read into them or written."""
    rows, g = 29, gen(width + offset)
    n = rows * width
    buf = torch.full((n + 64,), math.nan).half()
    buf[offset:offset + n] = torch.randn(n, generator=g).half()
    x = buf.cuda()[offset:offset + n].view(rows, width)
    out = torch.full((n + 64,), 7.0).half().cuda()
    ln = LayerNorm([width], torch.float16)
    y, mean, rstd = ln.forward(x, y=out[offset:offset + n].view(rows, width))
    want, bound = ref.layer_norm(host(x), [width], None, None, float(np.float32(1e-5)), "f16")
    for got, v, b in zip((y, mean, rstd), want, bound):
        within(got, v, b, "odd rows")
    dx, dw, db = ln.backward(x, x, mean, rstd)
    want, bound = ref.layer_norm_gradients(host(x), host(x), host(mean), host(rstd), [width], None, "f16")
    for got, v, b in zip((dx, dw, db), want, bound):
        within(got, v, b, "odd rows' gradients")
    assert bool((out[:offset] == 7).all()) and bool((out[offset + n:] == 7).all())


@pytest.mark.parametrize("width", [37, 64, 1000, 3001, 9000])
def test_norm_results_left_out(width):
    """The C interface's NULLs: no statistics, no dx, no dweight, no dbias; the others are the same bits."""
    s = norm_inputs(300, [width], "f32", "f32")
    ln = LayerNorm([width])
    y, mean, rstd = ln.forward(s["x"], s["weight"], s["bias"])
    dx, dw, db = ln.backward(s["dy"], s["x"], mean, rstd, s["weight"])
    y2 = torch.empty_like(y)
    stream = torch.cuda.current_stream().cuda_stream
    p = lambda v: None if v is None else v.data_ptr()  # noqa: E731
    assert ln.lib.tbe_layer_norm_forward(ln._prob, p(s["x"]), p(s["weight"]), p(s["bias"]), p(y2), None, None, stream) == 0
    assert torch.equal(y, y2)
    for keep in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (1, 1, 0)):
        out = [torch.full_like(v, 3.0) if k else None for v, k in zip((dx, dw, db), keep)]
        assert ln.lib.tbe_layer_norm_backward(ln._prob, p(s["dy"]), p(s["x"]), p(mean), p(rstd), p(s["weight"]), p(out[0]),
                                              p(out[1]), p(out[2]), p(ln.ws), ln.ws.numel(), stream) == 0
        for got, want in zip(out, (dx, dw, db)):
            assert got is None or torch.equal(got, want)


@pytest.mark.parametrize("offsets", [[0, 1 << 30, -5, 96], [90, 10, 5, 0], [1, 3, 95, 97], [0, 96, 96, 96]])
def test_norm_column_offsets_that_disagree_stay_in_the_row(offsets):
    """col_offsets that are not the widths' (a caller's mistake): unspecified values, but nothing outside the row."""
    ln = LayerNorm([32, 60, 4])
    ln.col_offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
    wide = torch.randn(50, 128, device="cuda")
    y = torch.full((50, 128), 7.0, device="cuda")
    _, mean, rstd = ln.forward(wide[:, 16:112], y=y[:, 16:112])
    assert bool((y[:, :16] == 7).all()) and bool((y[:, 112:] == 7).all())
    dx = torch.full((50, 128), 7.0, device="cuda")
    ln.backward(wide[:, 16:112], wide[:, 16:112], mean, rstd, dx=dx[:, 16:112])
    assert bool((dx[:, :16] == 7).all()) and bool((dx[:, 112:] == 7).all())


def test_norm_large_offset_and_constant_rows():
    # a mean 2^8 times the spread: the deviations are taken from the mean, not from E[x^2]
    check_norm(40, [256], shift=256.0, seed=3)
    x = torch.full((5, 96), 3.0, device="cuda")
    y, mean, rstd = LayerNorm([96]).forward(x)
    assert bool((mean == 3).all()) and bool((y == 0).all())
    within(rstd, np.full((5, 1), 1 / math.sqrt(float(np.float32(1e-5)))), np.full((5, 1), 1e-4), "rstd")


@pytest.mark.parametrize("width", [128, 513, 3000, 20000])
def test_norm_non_finite_rows_stay_in_their_row(width):
    x = torch.randn(20, width, device="cuda")
    x[3, 5], x[7, 0] = math.nan, math.inf
    ln = LayerNorm([width])
    y, mean, rstd = ln.forward(x)
    bad = torch.zeros(20, dtype=torch.bool, device="cuda")
    bad[3] = bad[7] = True
    assert bool(y[bad].isnan().any(1).all()) and bool(y[~bad].isfinite().all())
    clean = torch.where(bad[:, None], 0.0, x)
    assert torch.equal(ln.forward(clean)[0][~bad], y[~bad])
    dx, dw, db = ln.backward(torch.ones_like(x), x, mean, rstd)
    assert bool(dx[~bad].isfinite().all()) and bool(dx[bad].isnan().any(1).all())
    assert bool(dw.isnan().any()) and bool(db.isfinite().all())


@pytest.mark.parametrize("width", [64, 1000, 3000, 9000])
def test_norm_no_rows(width):
    ln = LayerNorm([width])
    x = torch.empty(0, width, device="cuda")
    y, mean, rstd = ln.forward(x)
    assert y.shape == (0, width) and mean.shape == (0, 1)
    dw, db = torch.full((2, width), 5.0, device="cuda").unbind(0)
    dx, dw, db = ln.backward(x, x, mean, rstd, dweight=dw, dbias=db)
    assert bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("width,dtype", [(128, "f32"), (2000, "f32"), (12000, "f32"), (20000, "f32"), (5, "f16"), (37, "f16"),
                                         (257, "f32"), (1001, "f16"), (4097, "bf16")])
def test_norm_in_place(width, dtype):
    s = norm_inputs(741, [width], dtype, dtype)
    ln = LayerNorm([width], DT[dtype], weight_dtype=torch.float32)
    s["weight"], s["bias"] = s["weight"].float(), s["bias"].float()
    y, mean, rstd = ln.forward(s["x"], s["weight"], s["bias"])
    dx, dw, db = ln.backward(s["dy"], s["x"], mean, rstd, s["weight"])
    x = s["x"].clone()
    assert torch.equal(ln.forward(x, s["weight"], s["bias"], y=x)[0], y)
    for target in ("x", "dy"):
        t = {k: s[k].clone() for k in ("x", "dy")}
        got = ln.backward(t["dy"], t["x"], mean, rstd, s["weight"], dx=t[target])
        assert got[0] is t[target] and all(torch.equal(a, b) for a, b in zip(got, (dx, dw, db)))


def test_norm_same_bits_every_time_and_on_another_stream():
    ln, s, out, grads = check_norm(3001, [128, 64, 256])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out2 = ln.forward(s["x"], s["weight"], s["bias"], stream=side)
    grads2 = ln.backward(s["dy"], s["x"], out2[1], out2[2], s["weight"], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out + grads, out2 + grads2))


@pytest.mark.parametrize("width", [128, 1001, 3000, 9000])
def test_norm_in_a_graph(width):
    s = norm_inputs(500, [width], "f32", "bf16")
    ln = LayerNorm([width], torch.float32, torch.bfloat16)
    y, mean, rstd = ln.forward(s["x"], s["weight"], s["bias"])
    grads = ln.backward(s["dy"], s["x"], mean, rstd, s["weight"])
    out = [torch.zeros_like(v) for v in (y, mean, rstd, *grads)]
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        ln.forward(s["x"], s["weight"], s["bias"], y=out[0], mean=out[1], rstd=out[2])
        ln.backward(s["dy"], s["x"], out[1], out[2], s["weight"], dx=out[3], dweight=out[4], dbias=out[5])
    for _ in range(2):
        for v in out:
            v.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, (y, mean, rstd, *grads)))


def test_norm_backward_is_the_difference_quotient_of_forward():
    """<dx, d> + <dweight, e> + <dbias, f> against the change of <y, dy> along (d, e, f).  y is fp32: with a step of
    2^-6 the quotient's rounding part is |dy|_1 2^-24 |y| 2^6 ~ 2^-14 of the sum's size; its cubic part, halved step
    against whole, is measured and allowed for."""
    g = gen(5)
    rows, widths = 24, [32, 100]
    s = norm_inputs(rows, widths, "f32", "f32", seed=9)
    ln = LayerNorm(widths)
    _, mean, rstd = ln.forward(s["x"], s["weight"], s["bias"])
    dx, dw, db = ln.backward(s["dy"], s["x"], mean, rstd, s["weight"])
    s["x"][1] = torch.randn(132, generator=g).cuda()  # an all-equal row has no usable quotient (its rstd is 1 / sqrt(eps))
    _, mean, rstd = ln.forward(s["x"], s["weight"], s["bias"])
    dx, dw, db = ln.backward(s["dy"], s["x"], mean, rstd, s["weight"])
    d = torch.randn(rows, 132, generator=g).cuda()
    e, f = torch.randn(2, 132, generator=g).cuda().unbind(0)
    along = (host(dx) * host(d)).sum() + (host(dw) * host(e)).sum() + (host(db) * host(f)).sum()

    def quotient(h):
        ys = [host(ln.forward(s["x"] + k * h * d, s["weight"] + k * h * e, s["bias"] + k * h * f)[0]) for k in (1, -1)]
        return ((ys[0] - ys[1]) * host(s["dy"])).sum() / (2 * h)

    q1, q2 = quotient(2.0 ** -6), quotient(2.0 ** -7)
    size = np.abs(host(s["dy"])).sum()
    assert abs(q2 - along) <= 2 * abs(q1 - q2) + 2.0 ** -13 * size


def test_norm_of_pooled_output_feeds_the_embedding_backward():
    """The path of a step: pooled rows -> layer norm by table -> dx -> backward_update, with the layer norm's dx
    as grad_out; empty bags give rows of zeros."""
    g = gen(2)
    D, E, B = [32, 64, 8], [50, 40, 30], 33
    lengths = torch.randint(0, 4, (len(D) * B,), generator=g)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    indices = torch.cat([torch.randint(0, E[t], (int(lengths[t * B:(t + 1) * B].sum()),), generator=g) for t in range(3)])
    tbe = TableBatchedEmbedding(D, E, B, indices.numel(), torch.float32)
    weights = (torch.rand(tbe.num_weights, generator=g) - 0.5).cuda()
    idx, off = indices.cuda(), offsets.cuda()
    pooled = tbe.forward(weights, idx, off)
    ln = LayerNorm(tbe.D)
    y, mean, rstd = ln.forward(pooled)
    empty = (lengths.view(3, B).T == 0).repeat_interleave(torch.tensor(D), 1)
    assert bool((y[empty.cuda()] == 0).all())
    dy = torch.randn(B, sum(D), generator=g).cuda()
    dx, _, _ = ln.backward(dy, pooled, mean, rstd)
    before = weights.clone()
    tbe.backward_update(weights, torch.zeros(tbe.total_rows, device="cuda"), idx, off, dx, optimizer="sgd", lr=0.1)
    # the row sums of an SGD step with unweighted bags: every lookup subtracts lr * dx of its bag
    want = host(before)
    at = np.concatenate([[0], np.cumsum([e * d for e, d in zip(E, D)])])
    col = np.concatenate([[0], np.cumsum(D)])
    for t in range(3):
        table = want[at[t]:at[t + 1]].reshape(E[t], D[t])
        for b in range(B):
            u = t * B + b
            for p in range(int(offsets[u]), int(offsets[u + 1])):
                table[int(indices[p])] -= 0.1 * host(dx)[b, col[t]:col[t + 1]]
    np.testing.assert_allclose(host(weights), want, rtol=1e-5, atol=1e-5 * np.abs(want).max())


def test_norm_refusals():
    ln = LayerNorm([64, 32])
    x = torch.randn(4, 96, device="cuda")
    with pytest.raises(TypeError):
        ln.forward(x.half())
    with pytest.raises(ValueError):
        ln.forward(x[:, :95])
    with pytest.raises(ValueError):
        ln.forward(x.t().contiguous().t())
    with pytest.raises(ValueError):
        ln.forward(x[:1].expand(4, 96))
    with pytest.raises(ValueError):
        ln.forward(x, weight=torch.ones(95, device="cuda"))
    with pytest.raises(TypeError):
        ln.forward(x, weight=torch.ones(96, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        ln.forward(x, mean=torch.empty(4, 2, device="cuda"))
    y, mean, rstd = ln.forward(x)
    with pytest.raises(ValueError):
        ln.backward(x[:3], x, mean, rstd)
    with pytest.raises(ValueError):
        ln.backward(x, x, mean[:3], rstd[:3])
    with pytest.raises(ValueError):
        ln.forward(x.cpu())
    with pytest.raises(TBEError):
        LayerNorm([64], torch.float16, torch.bfloat16)
    with pytest.raises(TBEError):
        LayerNorm([64, 0])
    with pytest.raises(TBEError):
        LayerNorm([64], eps=-1.0)
    wide = torch.randn(4, 200, device="cuda")
    with pytest.raises(TBEError):  # y over x with another stride
        ln.forward(wide[:, :96], y=wide.view(-1)[:384].view(4, 96))


# ------------------------------------------------------------------------------------------
# Gradient norm
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sizes", [[1], [7, 0, 3], [255, 256, 257, 2048, 2049], [100_003], [5] * 100, [3] * 1700, [1_500_000, 17]])
def test_grad_norm(sizes, dtype):
    g = gen(len(sizes))
    grads = [torch.randn(n, generator=g).to(DT[dtype]).cuda() for n in sizes]
    norm = GradNorm(grads)
    want = math.sqrt(sum((host(t) ** 2).sum() for t in grads))
    # squares and at most 9 sums of a thread's share of a chunk in fp32 (chunks of one pass at these sizes), the rest in fp64;
    # half of it in the root
    for max_norm in (math.inf, 0.5 * want, 2 * want, 0.0):
        got = host(norm.compute(max_norm))
        assert abs(got[0] - want) <= 20 * ref.U * want
        coef = min(1.0, max_norm / (got[0] + 1e-6))
        assert abs(got[1] - coef) <= 4 * ref.U * coef
    assert torch.equal(norm.compute(1.0), norm.compute(1.0))


def test_grad_norm_misaligned_views_and_nothing():
    flat = torch.randn(10_000, generator=gen(1)).to(torch.bfloat16).cuda()
    parts = [flat[1:4], flat[5:2054], flat[4099:4100], flat[4101:9999]]
    want = math.sqrt(sum((host(t) ** 2).sum() for t in parts))
    assert abs(host(GradNorm(parts).compute())[0] - want) <= 20 * ref.U * want
    assert host(GradNorm([]).compute(1.0)).tolist() == [0.0, 1.0]
    assert host(GradNorm([torch.empty(0, device="cuda")]).compute(1.0)).tolist() == [0.0, 1.0]


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_grad_norm_non_finite(bad):
    t = torch.ones(5000, device="cuda")
    t[4321] = bad
    got = host(GradNorm([torch.ones(3, device="cuda"), t]).compute(1.0))
    assert not math.isfinite(got[0])


def test_grad_norm_refusals():
    with pytest.raises(TypeError):
        GradNorm([torch.ones(3, device="cuda"), torch.ones(3, device="cuda", dtype=torch.float16)])
    with pytest.raises(TypeError):
        GradNorm([torch.ones(3, device="cuda", dtype=torch.float64)])
    with pytest.raises(ValueError):
        GradNorm([torch.ones(6, 4, device="cuda").t()])
    norm = GradNorm([torch.ones(3, device="cuda")])
    with pytest.raises(TBEError):
        norm.compute(-1.0)
    with pytest.raises(TBEError):
        norm.compute(math.nan)
    with pytest.raises(ValueError):
        norm.compute(1.0, out=torch.empty(3, device="cuda"))


# ------------------------------------------------------------------------------------------
# AdamW
# ------------------------------------------------------------------------------------------
LR, B1, B2, EPS = 1e-2, 0.9, 0.999, 1e-8


def adam_inputs(sizes, p, g, master, seed=0, offset=0):
    r = gen(seed)
    # `offset` elements before each tensor: views that start at no vector boundary
    view = lambda t: torch.cat([torch.zeros(offset, dtype=t.dtype), t]).cuda()[offset:]  # noqa: E731
    full = [torch.randn(n, generator=r) for n in sizes]
    s = dict(params=[view(t.to(DT[p])) for t in full],
             grads=[view((torch.randn(n, generator=r) * 10.0 ** torch.randint(-3, 2, (n,), generator=r)).to(DT[g]))
                    for n in sizes])
    s["master"] = [view(t) for t in full] if master else None
    return s


def check_steps(opt, s, p, steps, sizes, decay, lr_scale, states, clip=None, betas=(B1, B2), eps=EPS):
    """Each step against the 64-bit formula from the state before it."""
    coef = 1.0 if clip is None else float(clip[1])
    for _ in range(steps):
        t = int(opt.steps.item()) + 1
        before = []
        for i in range(len(sizes)):
            if states == "q8":
                m = ref.q8_decode(opt.exp_avg[i].cpu().numpy(), host(opt.exp_avg_scale[i]), True).astype(np.float32)
                v = ref.q8_decode(opt.exp_avg_sq[i].cpu().numpy(), host(opt.exp_avg_sq_scale[i]), False).astype(np.float32)
            else:
                m, v = host(opt.exp_avg[i]), host(opt.exp_avg_sq[i])
            before.append((host(s["master"][i] if s["master"] else s["params"][i]), m, v))
        opt.step(LR, clip=clip)
        assert int(opt.steps.item()) == t
        for i in range(len(sizes)):
            p0, m0, v0 = before[i]
            store = "f32" if s["master"] else p
            lr = float(np.float32(LR)) * lr_scale[i]
            (p1, m1, v1), (ep, em, ev) = ref.adamw(p0, host(s["grads"][i]), m0, v0, t, lr, *betas, eps, decay[i], coef, store)
            within(s["master"][i] if s["master"] else s["params"][i], p1, ep, f"p of tensor {i}")
            if s["master"]:
                assert torch.equal(s["params"][i], s["master"][i].to(DT[p]))
            if states == "f32":
                within(opt.exp_avg[i], m1, em, "m")
                within(opt.exp_avg_sq[i], v1, ev, "v")
            else:
                check_q8(opt, i, m1, v1, m0, v0, host(s["grads"][i]), coef, betas)


def fp32_moments(m, v, g, coef, betas):
    """The moments with each product and sum rounded to fp32, as documented."""
    f = np.float32
    m, v, g = (np.asarray(a, f) for a in (m, v, g))
    g = g * f(coef)
    return m * f(betas[0]) + g * f(1 - betas[0]), v * f(betas[1]) + (g * g) * f(1 - betas[1])


def check_q8(opt, i, m1, v1, m0, v0, g, coef, betas):
    """Codes are the nearest ones to the fp32 moments (one of the two nearest within 1e-6 of a middle); scales are
    the blocks' largest magnitudes, exactly."""
    m, v = fp32_moments(m0, v0, g, coef, betas)
    for got, got_scale, x, signed in ((opt.exp_avg[i], opt.exp_avg_scale[i], m, True),
                                      (opt.exp_avg_sq[i], opt.exp_avg_sq_scale[i], v, False)):
        codes, scale, gap = ref.q8_encode(x, signed)
        assert np.array_equal(host(got_scale), scale)
        got = got.cpu().numpy().astype(np.int64)
        off = got != codes
        zero = (codes & 127 if signed else codes) == 0
        assert np.array_equal(got[off & zero] & 127, codes[off & zero] & 127)  # -0 and 0
        off &= ~zero
        assert (np.abs(got[off] - codes[off]) <= 1).all() and (gap[off] <= 1e-6).all()
        if not signed:
            assert ((got > 0) == (x > 0))[np.repeat(scale, 256)[:x.size] > 0].all()
    mv, vv = opt.state_values()
    assert np.array_equal(host(mv[i]), (ref.q8_decode(opt.exp_avg[i].cpu().numpy(), host(opt.exp_avg_scale[i]), True)
                                        ).astype(np.float32))
    assert np.array_equal(host(vv[i]), (ref.q8_decode(opt.exp_avg_sq[i].cpu().numpy(), host(opt.exp_avg_sq_scale[i]), False)
                                        ).astype(np.float32))


SIZES = [1, 7, 8, 255, 256, 257, 2048, 2051, 0, 5000]


@pytest.mark.parametrize("states", ["f32", "q8"])
@pytest.mark.parametrize("p,g,master", [("f32", "f32", False), ("f32", "bf16", False), ("f32", "f16", False),
                                        ("bf16", "bf16", False), ("bf16", "f32", True), ("bf16", "bf16", True),
                                        ("bf16", "f16", False), ("f16", "f16", False), ("f16", "f32", True),
                                        ("f16", "bf16", True)])
def test_adamw_types(p, g, master, states):
    s = adam_inputs(SIZES, p, g, master)
    decay, scale = [0.01 * (i % 3) for i in range(len(SIZES))], [1.0 - 0.5 * (i % 2) for i in range(len(SIZES))]
    opt = DenseAdamW(s["params"], s["grads"], states, s["master"], weight_decay=decay, lr_scale=scale, betas=(B1, B2), eps=EPS)
    check_steps(opt, s, p, 3, SIZES, decay, scale, states)


@pytest.mark.parametrize("states", ["f32", "q8"])
@pytest.mark.parametrize("offset", [1, 3, 4, 5])
def test_adamw_misaligned_tensors(offset, states):
    for p, g, master in (("f32", "f32", False), ("bf16", "bf16", True)):
        s = adam_inputs([3, 100, 4099], p, g, master, offset=offset)
        n = [3, 100, 4099]
        state = {"exp_avg": [torch.zeros(k + offset, device="cuda", dtype=torch.uint8 if states == "q8" else torch.float32)[offset:]
                             for k in n]}
        opt = DenseAdamW(s["params"], s["grads"], states, s["master"], state=state, weight_decay=0.1, betas=(B1, B2), eps=EPS)
        check_steps(opt, s, p, 2, n, [0.1] * 3, [1.0] * 3, states)


def test_adamw_tensors_packed_tightly():
    """Tensors that follow one another in flat buffers share the vectors' alignment from their first elements on; whatever
    lies between the chunks' ends is updated once."""
    for p in ("f32", "bf16"):
        sizes = [2045, 2049, 3, 1, 8191, 5, 4100]
        starts = np.concatenate([[0], np.cumsum(sizes)])
        flat = {k: torch.randn(starts[-1], generator=gen(4)).to(DT[p] if k in ("params", "grads") else torch.float32).cuda()
                for k in ("params", "grads", "m", "v")}
        flat["v"].abs_()
        cut = lambda t: [t[a:b] for a, b in zip(starts[:-1], starts[1:])]  # noqa: E731
        s = dict(params=cut(flat["params"]), grads=cut(flat["grads"]), master=None)
        opt = DenseAdamW(s["params"], s["grads"], state={"exp_avg": cut(flat["m"]), "exp_avg_sq": cut(flat["v"])},
                         weight_decay=0.1, betas=(B1, B2), eps=EPS)
        check_steps(opt, s, p, 2, sizes, [0.1] * len(sizes), [1.0] * len(sizes), "f32")


@pytest.mark.parametrize("states", ["f32", "q8"])
@pytest.mark.parametrize("count", [39, 40, 41, 361, 800])
def test_adamw_many_tensors(count, states):
    sizes = [1 + (37 * i) % 600 for i in range(count)]
    s = adam_inputs(sizes, "bf16", "bf16", False)
    decay = [0.1 * (i % 2) for i in range(count)]
    opt = DenseAdamW(s["params"], s["grads"], states, weight_decay=decay, betas=(B1, B2), eps=EPS)
    check_steps(opt, s, "bf16", 1, sizes, decay, [1.0] * count, states)


@pytest.mark.parametrize("states", ["f32", "q8"])
def test_adamw_large_tensor(states):
    # more chunks than four to an SM: the long chunks
    n = [6_000_011]
    s = adam_inputs(n, "bf16", "f32", False)
    opt = DenseAdamW(s["params"], s["grads"], states, betas=(B1, B2), eps=EPS)
    g, p0 = s["grads"][0].clone(), s["params"][0].clone()
    opt.step(LR)
    m, v = (t[0] for t in opt.state_values()) if states == "q8" else (opt.exp_avg[0], opt.exp_avg_sq[0])
    gd = g.double()
    upd = gd / (gd.abs() + EPS)  # the first step: m / (1 - b1) = g, sqrt(v / (1 - b2)) = |g|
    want = p0.double() * (1 - float(np.float32(LR)) * 0.01) - float(np.float32(LR)) * upd
    assert bool(((s["params"][0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all())
    block = lambda t: torch.nn.functional.pad(t, (0, -n[0] % 256)).view(-1, 256)  # noqa: E731
    if states == "f32":
        assert torch.equal(m, g * np.float32(1 - B1).item()) and torch.equal(v, (g * g) * np.float32(1 - B2).item())
    else:
        # half the widest step between codes, by the interval that the magnitude lies in: 7/16 of its power of 8 at 2^-k
        for got, x, bits in ((m, g * np.float32(1 - B1).item(), 7), (v, (g * g) * np.float32(1 - B2).item(), 8)):
            a = block(x.abs()).amax(1, keepdim=True)
            r = (block(x.abs()) / a).double()
            levels = torch.from_numpy(ref.q8_levels(bits)).cuda()
            step = levels[1:] - levels[:-1]
            at = torch.bucketize(r, levels[1:]).clamp(max=step.numel() - 1)
            most = step[at] / 2
            if bits == 8:
                most[at == 0] = levels[1]
            else:
                most[at == 0] = levels[1] * 0.5626  # the lowest interval's line starts above zero
            assert bool(((block(got).double() - block(x).double()).abs() / a <= most * (1 + 1e-5) + 1e-7).all())


@pytest.mark.parametrize("states", ["f32", "q8"])
def test_adamw_clip_coefficient_and_skipped_steps(states):
    sizes = [300, 1000]
    s = adam_inputs(sizes, "f32", "f32", False)
    opt = DenseAdamW(s["params"], s["grads"], states, weight_decay=0.1, betas=(B1, B2), eps=EPS)
    norm = GradNorm(s["grads"])
    clip = norm.compute(0.25)
    assert 0 < float(clip[1]) < 1
    check_steps(opt, s, "f32", 2, sizes, [0.1] * 2, [1.0] * 2, states, clip=clip)
    s["grads"][1][77] = math.inf
    keep = [t.clone() for t in s["params"] + opt.exp_avg + opt.exp_avg_sq + [opt.steps]]
    opt.step(LR, clip=norm.compute(0.25))
    assert all(torch.equal(a, b) for a, b in zip(keep, s["params"] + opt.exp_avg + opt.exp_avg_sq + [opt.steps]))
    s["grads"][1][77] = 1.0
    check_steps(opt, s, "f32", 1, sizes, [0.1] * 2, [1.0] * 2, states, clip=norm.compute(0.25))


@pytest.mark.parametrize("states", ["f32", "q8"])
@pytest.mark.parametrize("betas,eps", [((0.0, 0.0), 1e-8), ((0.0, 0.999), 1e-3), ((0.95, 0.5), 0.0)])
def test_adamw_other_factors(betas, eps, states):
    sizes = [700]
    s = adam_inputs(sizes, "f32", "f32", False)
    opt = DenseAdamW(s["params"], s["grads"], states, betas=betas, eps=eps)
    check_steps(opt, s, "f32", 2, sizes, [0.01], [1.0], states, betas=betas, eps=eps)


def test_adamw_late_steps():
    # t far on: the corrections are 1; t given with the state
    s = adam_inputs([500], "f32", "f32", False)
    opt = DenseAdamW(s["params"], s["grads"], state={"step": torch.full((1,), 10 ** 7, device="cuda")}, betas=(B1, B2), eps=EPS)
    check_steps(opt, s, "f32", 2, [500], [0.01], [1.0], "f32")


def test_adamw_q8_zero_blocks_and_vanishing_gradients():
    """Blocks of zeros keep scale 0; a second moment that falls below its block's lowest code stays positive, so a
    coordinate whose gradient stops is not left with m / eps."""
    p = torch.zeros(1024, device="cuda")
    g = torch.zeros(1024, device="cuda")
    g[256:512] = 1e-6
    g[300] = 1e3
    opt = DenseAdamW([p], [g], "q8", weight_decay=0.0)
    opt.step(1e-3)
    assert host(opt.exp_avg_scale[0])[[0, 2, 3]].tolist() == [0, 0, 0]
    assert bool((opt.exp_avg_sq[0][256:512] > 0).all())
    g.zero_()
    before = p.clone()
    opt.step(1e-3)
    assert bool(((p - before).abs() <= 1e-3 * 2).all()) and bool(p.isfinite().all())
    assert bool((p[:256] == 0).all()) and bool((p[512:] == 0).all())


def test_adamw_q8_non_finite_gradient_stays_in_its_block():
    p, g = torch.zeros(1024, device="cuda"), torch.ones(1024, device="cuda")
    g[300] = math.nan
    opt = DenseAdamW([p], [g], "q8")
    opt.step(1e-3)
    m, v = (t[0] for t in opt.state_values())
    ok = torch.ones(1024, dtype=torch.bool, device="cuda")
    ok[256:512] = False
    assert bool(m[ok].isfinite().all()) and bool(p[ok].isfinite().all()) and bool(m[~ok].isnan().all())
    assert bool(p[300].isnan())


def test_adamw_q8_trains_like_f32():
    """A least-squares problem of coordinates on very different scales: both forms reach the same loss (to 10%)."""
    losses = {}
    for states in ("f32", "q8"):
        r = gen(11)
        a = (torch.randn(512, 128, generator=r) * 10 ** torch.linspace(-1, 0.5, 128)).cuda()
        truth = torch.randn(128, generator=r).cuda()
        b = a @ truth + 0.5 * torch.randn(512, generator=r).cuda()
        x = torch.zeros(128, device="cuda")
        g = torch.empty(128, device="cuda")
        opt = DenseAdamW([x], [g], states, weight_decay=0.0)
        for k in range(600):
            torch.matmul(a.T, a @ x - b, out=g)
            g.div_(512)
            opt.step(0.05 * (1 - k / 600))
        losses[states] = float(((a @ x - b) ** 2).mean())
    assert losses["q8"] <= 1.1 * losses["f32"] and losses["f32"] < 0.5


def test_adamw_step_and_norm_in_a_graph():
    """Captured once, replayed: the step count lives on the device, so each replay has its own corrections."""
    s = adam_inputs([3000, 50], "f32", "f32", False)
    s2 = adam_inputs([3000, 50], "f32", "f32", False)
    opt, opt2 = (DenseAdamW(x["params"], x["grads"]) for x in (s, s2))
    norm, norm2 = GradNorm(s["grads"]), GradNorm(s2["grads"])
    clip = torch.empty(2, device="cuda")
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        norm.compute(0.5, out=clip)
        opt.step(LR, clip=clip)
    for _ in range(3):
        graph.replay()
        opt2.step(LR, clip=norm2.compute(0.5))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(s["params"], s2["params"])) and int(opt.steps) == 3


def test_objects_made_and_used_on_different_streams():
    """Made on one stream, used on another at once and dropped while the work may still run: the object's memory is
    complete when the constructor returns and is not handed out again before the other stream is done."""
    side = torch.cuda.Stream()
    p, g = torch.zeros(1 << 20, device="cuda"), torch.ones(1 << 20, device="cuda")
    x = torch.randn(1 << 14, 64, device="cuda")
    want = LayerNorm([64]).forward(x)
    grads = LayerNorm([64]).backward(x, x, want[1], want[2])
    torch.cuda.synchronize()
    for _ in range(5):
        opt = DenseAdamW([p], [g], "q8", weight_decay=0.0)
        opt.step(1e-3, clip=GradNorm([g]).compute(stream=side), stream=side)
        got = LayerNorm([64]).backward(x, x, want[1], want[2], stream=side)
        steps = opt.steps
        del opt
        torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")  # would land in freed memory
        side.synchronize()
        assert int(steps) == 1 and all(torch.equal(a, b) for a, b in zip(got, grads))
    np.testing.assert_allclose(host(p), -5e-3, rtol=1e-5)


@pytest.mark.parametrize("states", ["f32", "q8"])
def test_adamw_nothing_to_update(states):
    """No tensor, or tensors without elements: the step is counted, unless the norm calls it off."""
    for params in ([], [torch.empty(0, device="cuda")] * 2):
        opt = DenseAdamW(params, [p.clone() for p in params], states)
        opt.step(LR)
        opt.step(LR, clip=torch.tensor([1.0, 1.0], device="cuda"))
        opt.step(LR, clip=torch.tensor([math.inf, 0.0], device="cuda"))
        opt.step(LR, clip=torch.tensor([math.nan, math.nan], device="cuda"))
        assert int(opt.steps) == 2


def test_adamw_rebound_gradients():
    s = adam_inputs([100], "f32", "f32", False)
    opt = DenseAdamW(s["params"], s["grads"], weight_decay=0.0)
    other = [torch.full((100,), -2.0, dtype=torch.bfloat16, device="cuda")]
    opt.bind_grads(other)
    before = s["params"][0].clone()
    opt.step(LR)
    np.testing.assert_allclose(host(s["params"][0] - before), LR, rtol=1e-4)


def test_adamw_refusals():
    p, g = torch.zeros(10, device="cuda"), torch.zeros(10, device="cuda")
    with pytest.raises(ValueError):
        DenseAdamW([p], [])
    with pytest.raises(ValueError):
        DenseAdamW([p], [g[:9]])
    with pytest.raises(TypeError):
        DenseAdamW([p], [g], master=[g])
    with pytest.raises(TypeError):
        DenseAdamW([p], [g], state={"moment": [g]})
    with pytest.raises(TypeError):
        DenseAdamW([p], [g], "q8", state={"exp_avg": [g]})
    with pytest.raises(ValueError):
        DenseAdamW([p], [g], weight_decay=[0.1, 0.2])
    with pytest.raises(KeyError):
        DenseAdamW([p], [g], states="f64")
    with pytest.raises(TBEError):
        DenseAdamW([p], [g], betas=(1.0, 0.9)).step(LR)
    with pytest.raises(TBEError):
        DenseAdamW([p], [g], eps=-1.0).step(LR)
    opt = DenseAdamW([p], [g])
    with pytest.raises(TBEError):
        opt.step(math.nan)
    with pytest.raises(TBEError):
        opt.state_values()
    with pytest.raises(ValueError):
        opt.step(LR, clip=torch.ones(1, device="cuda"))
    with pytest.raises(TypeError):
        opt.step(LR, clip=torch.ones(2, device="cuda", dtype=torch.float64))
    assert int(opt.steps) == 0
