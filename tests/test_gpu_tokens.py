"""The lookup of a table's rows with its gradient and the softmax cross entropy over them (include/tbe_tokens.h) against
their formulas in 64 bits (tests/tokens_reference.py, whose bounds follow from the roundings), at the sizes, strides,
ids and values where they can go wrong."""
import numpy as np
import pytest
import torch

import tokens_reference as ref
from bwd_tbe_fwd_gb300 import STAT_NAMES, SoftmaxLoss, TokenEmbedding

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
IT = {"i32": torch.int32, "i64": torch.int64}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def host(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what):
    got = host(got)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside; first at {tuple(np.argwhere(bad)[0])}: "
                           f"{got[bad][0]!r} for {want[bad][0]!r} +- {bound[bad][0]!r}")


def strided(t, pad):
    """The same values as a view of a wider matrix whose other columns are NaN."""
    if not pad:
        return t.cuda()
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]]


def make_ids(g, n, rows, kind, itype):
    """"spread": uniform; "hot": half of them one row; "one": all the same; "run": sorted; some padding in each but "full"."""
    ids = torch.randint(0, rows, (n,), generator=g)
    if kind == "hot":
        ids = torch.where(torch.rand(n, generator=g) < 0.5, torch.full_like(ids, rows - 1), ids)
    if kind == "one":
        ids = torch.full_like(ids, rows // 2)
    if kind == "none":
        ids = torch.full_like(ids, -1)
    if kind not in ("full", "one"):
        ids = torch.where(torch.rand(n, generator=g) < 0.15, torch.full_like(ids, -1), ids)
    if kind == "run":
        ids = ids.sort().values
    return ids.to(IT[itype])


# ------------------------------------------------------------------------------------------
# Lookup
# ------------------------------------------------------------------------------------------
def check_lookup(tokens, rows, dim, table="f32", out="f32", ids="spread", itype="i64", pad=0, scale=1.0, accumulate=False, seed=0,
                 room=0):
    g = gen(seed)
    emb = TokenEmbedding(rows, dim, tokens + room, DT[table], DT[out], IT[itype], scale)
    i = make_ids(g, tokens, rows, ids, itype)
    i_d, i_h = i.cuda(), i.numpy().astype(np.int64)
    t = strided(torch.randn(rows, dim, generator=g).to(DT[table]), pad)
    y = emb.forward(t, i_d, out=strided(torch.zeros(tokens, dim, dtype=DT[out]), pad))
    within(y, *ref.lookup(host(t), i_h, scale, out), "out")
    dout = strided(torch.randn(tokens, dim, generator=g).to(DT[out]), pad)
    old = torch.randn(rows, dim, generator=g).to(DT[table]) if accumulate else torch.full((rows, dim), float("nan"), dtype=DT[table])
    grad = strided(old, pad)
    got = emb.backward(dout, i_d, grad=grad, accumulate=accumulate)
    assert got is grad
    want, bound = ref.lookup_gradient(host(dout), i_h, rows, scale, table, host(old) if accumulate else None)
    within(got, want, bound, "grad")
    if pad:  # columns past a row's are nobody's
        assert bool(torch.isnan(grad.as_strided((rows, pad), grad.stride(), dim)).all())
    again = emb.backward(dout, i_d, grad=strided(old, pad), accumulate=accumulate)
    assert torch.equal(again.cpu(), got.cpu())
    assert not emb.stats.any()


TYPES = [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("table,out", TYPES)
@pytest.mark.parametrize("dim", [1, 4, 8, 33, 128, 260, 1001])
def test_lookup_types_and_widths(dim, table, out):
    check_lookup(75, 40, dim, table, out, scale=1.7, seed=dim)


@pytest.mark.parametrize("tokens", [1, 2, 31, 32, 33, 63, 64, 65, 255, 1000, 4095, 4096, 4097, 8192, 8193, 20000])
@pytest.mark.parametrize("kind", ["spread", "hot", "one", "run", "none", "full"])
def test_lookup_every_length(tokens, kind):
    check_lookup(tokens, 100, 24, "bf16", "f32", ids=kind, seed=tokens)


@pytest.mark.parametrize("rows", [1, 2, 255, 256, 257, 70000, 300_001])
def test_lookup_row_counts(rows):
    check_lookup(3000, rows, 16, "f16", "f16", itype="i32", seed=rows)


@pytest.mark.parametrize("pad", [1, 3, 8, 64])
@pytest.mark.parametrize("accumulate", [False, True])
def test_lookup_strides_and_accumulation(pad, accumulate):
    check_lookup(500, 70, 64, "bf16", "bf16", pad=pad, accumulate=accumulate, scale=-0.5, seed=pad)
    check_lookup(500, 70, 30, "f32", "bf16", ids="hot", pad=pad, accumulate=accumulate, itype="i32", seed=pad)


def test_lookup_of_more_than_a_cluster_sorts():
    check_lookup(70_001, 5000, 8, "f32", "f32", ids="hot", seed=5)
    check_lookup(200_000, 1_000_003, 4, "f32", "f32", seed=6)


def test_lookup_of_no_tokens():
    emb = TokenEmbedding(10, 8, 4)
    ids = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert emb.forward(torch.ones(10, 8, device="cuda"), ids).shape == (0, 8)
    grad = torch.ones(10, 8, device="cuda")
    assert float(emb.backward(torch.zeros(0, 8, device="cuda"), ids, grad=grad, accumulate=True).sum()) == 80
    assert float(emb.backward(torch.zeros(0, 8, device="cuda"), ids, grad=grad).abs().sum()) == 0


def test_lookup_counts_ids_past_the_table():
    emb = TokenEmbedding(10, 8, 6)
    ids = torch.tensor([-1, 0, 10, 9, 2 ** 40, -2 ** 60], device="cuda")
    out = emb.forward(torch.ones(10, 8, device="cuda"), ids)
    assert out[:, 0].tolist() == [0, 1, 0, 1, 0, 0]
    assert dict(zip(STAT_NAMES, emb.stats.tolist()))["unrepaired"] == 2
    grad = emb.backward(torch.ones(6, 8, device="cuda"), ids)
    assert grad[:, 0].tolist() == [1, 0, 0, 0, 0, 0, 0, 0, 0, 1]
    assert dict(zip(STAT_NAMES, emb.stats.tolist()))["unrepaired"] == 4


def test_lookup_padding_may_hold_anything():
    emb = TokenEmbedding(4, 8, 3)
    dout = torch.ones(3, 8, device="cuda")
    dout[1] = float("nan")
    grad = emb.backward(dout, torch.tensor([2, -1, 2], device="cuda"))
    assert grad[:, 0].tolist() == [0, 0, 2, 0]


# ------------------------------------------------------------------------------------------
# Softmax cross entropy
# ------------------------------------------------------------------------------------------
def loss_inputs(tokens, rows, dim, dtype, ids="spread", itype="i64", scale=1.0, pad=0, spread=2.0, seed=0):
    g = gen(seed)
    w = (torch.randn(rows, dim, generator=g) * (spread / (scale * dim ** 0.5))).to(DT[dtype])
    h = torch.randn(tokens, dim, generator=g).to(DT[dtype])
    t = make_ids(g, tokens, rows, ids, itype)
    h[(t < 0)] = float("nan")  # what padding holds is nobody's business
    return strided(h, pad), strided(w, pad if dim % 8 or pad % 8 == 0 else 8), t.cuda(), t.numpy().astype(np.int64)


def check_loss(tokens, rows, dim, dtype="bf16", ids="spread", itype="i64", scale=1.0, pad=0, spread=2.0, seed=0, upstream="mean",
               room=0):
    h, w, t, t_h = loss_inputs(tokens, rows, dim, dtype, ids, itype, scale, pad, spread, seed)
    op = SoftmaxLoss(rows, dim, tokens + room, DT[dtype], IT[itype], scale)
    out = op.forward(h, w, t)
    want, bound = ref.loss(host(h), host(w), t_h, scale)
    for got, v, b, name in zip(out, want, bound, ("loss", "lse", "mean")):
        within(got, v, b, name)
    loss, lse, mean = out
    dloss = None
    coef = np.full(tokens, float(mean[1]))
    if upstream == "tokens":
        dloss = torch.randn(tokens, generator=gen(seed + 1)).cuda()
        coef = host(dloss)
    grads = op.backward(h, w, t, lse, dloss=dloss, mean=None if upstream == "tokens" else mean,
                        dhidden=strided(torch.full((tokens, dim), float("nan"), dtype=DT[dtype]), pad),
                        dweight=strided(torch.full((rows, dim), float("nan"), dtype=DT[dtype]), pad))
    want, bound = ref.loss_gradients(host(h), host(w), t_h, host(lse), coef, scale, dtype)
    for got, v, b, name in zip(grads, want, bound, ("dhidden", "dweight")):
        within(got, v, b, name)
    again = op.backward(h, w, t, lse, dloss=dloss, mean=None if upstream == "tokens" else mean)
    assert all(torch.equal(x, y) for x, y in zip(grads, again))
    assert not op.stats.any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,rows,dim", [(1, 1, 1), (1, 2, 8), (32, 1000, 64), (256, 256, 64), (257, 257, 65), (300, 700, 128),
                                             (128, 255, 301), (5, 3000, 1000)])
def test_loss_sizes(tokens, rows, dim, dtype):
    check_loss(tokens, rows, dim, dtype, seed=tokens, upstream="tokens")


@pytest.mark.parametrize("dim", [1, 7, 8, 16, 63, 64, 72, 127, 128, 129, 136, 255, 256, 257, 320, 513, 1024])
def test_loss_widths(dim):
    check_loss(77, 333, dim, "bf16", seed=dim)


@pytest.mark.parametrize("rows", [1, 2, 127, 128, 129, 255, 256, 257, 511, 513, 4097])
def test_loss_row_counts(rows):
    check_loss(40, rows, 40, "f16", itype="i32", seed=rows, upstream="tokens")


@pytest.mark.parametrize("tokens", [1, 2, 127, 128, 129, 255, 256, 257, 511, 513, 1025])
def test_loss_token_counts(tokens):
    check_loss(tokens, 300, 48, "bf16", ids="hot", seed=tokens)


@pytest.mark.parametrize("pad", [1, 8, 24])
def test_loss_strides(pad):
    check_loss(100, 500, 96, "bf16", pad=pad, seed=pad)
    check_loss(100, 500, 45, "f16", pad=pad, seed=pad, upstream="tokens", room=1000)


@pytest.mark.parametrize("kind", ["one", "none", "full", "run"])
def test_loss_targets(kind):
    check_loss(200, 400, 64, "bf16", ids=kind, seed=3)


@pytest.mark.parametrize("scale,spread", [(20.0, 2.0), (0.125, 2.0), (1.0, 30.0), (1.0, 0.0)])
def test_loss_scales(scale, spread):
    check_loss(150, 600, 64, "bf16", scale=scale, spread=spread, seed=4)


def test_loss_of_no_tokens():
    op = SoftmaxLoss(10, 16, 4)
    h, w = torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda"), torch.ones(10, 16, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    loss, lse, mean = op.forward(h, w, t)
    assert loss.shape == lse.shape == (0,) and mean.tolist() == [0, 0]
    dh, dw = op.backward(h, w, t, lse, mean=mean)
    assert dh.shape == (0, 16) and float(dw.abs().sum()) == 0


@pytest.mark.parametrize("tokens,kind", [(1023, "spread"), (1024, "spread"), (1500, "hot"), (4097, "none"), (4100, "run"), (1100, "full")])
def test_loss_selects_the_tokens_that_count(tokens, kind):
    check_loss(tokens, 290, 40, "bf16", ids=kind, seed=tokens)


@pytest.mark.parametrize("dim", [24, 136, 200])
@pytest.mark.parametrize("rows", [1500, 1600, 9000])
def test_loss_sums_of_dhidden_in_one_and_in_many_splits(rows, dim):
    check_loss(90, rows, dim, "f16", seed=rows, upstream="tokens")
    check_loss(600, rows, dim, "bf16", seed=rows)


@pytest.mark.parametrize("tokens", [1, 16, 31, 32, 33])
def test_loss_of_few_tokens_over_many_rows(tokens):
    """One tile of tokens, more tiles of the table than pairs of CTAs: the pairs join their parts."""
    check_loss(tokens, 30_011, 72, "bf16", ids="hot", seed=tokens)


@pytest.mark.parametrize("rows,dim", [(1, 8), (17, 48), (300, 40), (257, 300)])
@pytest.mark.parametrize("kind", ["spread", "none", "one"])
def test_loss_of_many_tokens_over_few_rows(rows, dim, kind):
    """dweight's sums over the tokens are split, into as many parts as there are blocks of tokens that count at most."""
    check_loss(6000, rows, dim, "bf16", ids=kind, seed=rows)


def test_loss_of_many_tokens_of_which_few_count():
    h, w, t, t_h = loss_inputs(8000, 20, 64, "bf16", seed=1)
    t[130:] = -1
    t_h[130:] = -1
    op = SoftmaxLoss(20, 64, 8000)
    _, lse, mean = op.forward(h, w, t)
    grads = op.backward(h, w, t, lse, mean=mean)
    want, bound = ref.loss_gradients(host(h), host(w), t_h, host(lse), np.full(8000, float(mean[1])), 1.0, "bf16")
    for got, v, b, name in zip(grads, want, bound, ("dhidden", "dweight")):
        within(got, v, b, name)


@pytest.mark.parametrize("table,out", TYPES)
@pytest.mark.parametrize("dim", [63, 64, 66, 127, 130, 914, 1597])
def test_lookup_wide_rows_without_vectors(dim, table, out):
    check_lookup(333, 50, dim, table, out, pad=1 if dim % 2 else 2, scale=0.3, seed=dim)
    check_lookup(50, 20, dim, table, out, seed=dim + 1)


@pytest.mark.parametrize("at", [1, 2, 4])
def test_lookup_buffers_may_begin_anywhere(at):
    """Tables, gradients and rows that begin at any element of a buffer, whose other elements stay as they are."""
    g = gen(at)
    rows, dim, tokens = 90, 64, 400
    emb = TokenEmbedding(rows, dim, tokens, torch.float16, torch.float16)
    ids = torch.randint(-1, rows, (tokens,), generator=g).cuda()
    wide = [torch.full((n * dim + 8,), 7.0, dtype=torch.float16, device="cuda") for n in (rows, tokens, rows, tokens)]
    table, out, grad, dout = (t[at:at + n * dim].view(n, dim) for t, n in zip(wide, (rows, tokens, rows, tokens)))
    table.copy_(torch.randn(rows, dim, generator=g))
    dout.copy_(torch.randn(tokens, dim, generator=g))
    emb.forward(table, ids, out=out)
    emb.backward(dout, ids, grad=grad)
    want = emb.forward(table.clone(), ids), emb.backward(dout.clone(), ids)
    assert torch.equal(out, want[0]) and torch.equal(grad, want[1])
    for t, n in zip(wide, (rows, tokens, rows, tokens)):
        assert bool((t[:at] == 7).all()) and bool((t[at + n * dim:] == 7).all())


@pytest.mark.parametrize("tokens", [8193, 16384, 16385, 65535, 65537, 131072, 131073])
def test_lookup_at_the_borders_of_the_sorts(tokens):
    check_lookup(tokens, 3000, 4, "f32", "f32", ids="hot", seed=tokens, room=1000)
    check_lookup(tokens, 1_500_000, 4, "f32", "f32", accumulate=True, seed=tokens + 1)
