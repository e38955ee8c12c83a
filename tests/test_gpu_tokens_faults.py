"""The token side (include/tbe_tokens.h) where it once went wrong, or where no test had looked."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import tokens_reference as ref
from bwd_tbe_fwd_gb300 import SoftmaxLoss, TokenEmbedding
from test_gpu_tokens import check_lookup, check_loss, gen, host, loss_inputs, within

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


# ------------------------------------------------------------------------------------------
# Coefficients of different sizes in fp16
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("tokens,rows,dim", [(48, 131072, 16), (100, 1500, 24), (600, 20011, 37), (1500, 900, 64)])
def test_fp16_gradients_of_coefficients_of_different_sizes(tokens, rows, dim):
    """Coefficients from 1 down to 10^-6, dhidden row by row against the row's own size.  The table's rows have a common part, so
    that the probabilities' sum counts.  What dz loses to fp16's least values is, at a coefficient c, no more than 2^-13 c / rows
    an entry: 2^-25 where the largest coefficient is 2^13 and c = 2^-k of it has a factor 2^e, e >= k + log2(rows) - 24.  That
    holds where hidden's rows reach 2^(k + log2(rows) - 34): 8 for k = 20 and 2^17 rows.  dweight's product takes hidden's
    rows to 2^-15 of their largest element."""
    g = gen(rows)
    h = torch.randn(tokens, dim, generator=g).clamp(-7, 7)
    h[:, 0] = 8
    w = torch.randn(rows, dim, generator=g) * 0.05 + 0.25
    h, w = h.half().cuda(), w.half().cuda()
    t = torch.randint(0, rows, (tokens,), generator=g).cuda()
    t[5] = -1
    c = 2.0 ** 10 * 10.0 ** (-6 * torch.rand(tokens, generator=g).sort().values)
    c[::3] *= -1
    c[0], c[-1], c[7] = 2.0 ** 10, 2.0 ** 10 * 1e-6, 0
    op = SoftmaxLoss(rows, dim, tokens, dtype=torch.float16)
    lse = op.forward(h, w, t)[1]
    dh, dw = op.backward(h, w, t, lse, dloss=c.cuda())
    hh, wh, th, lh, ch = host(h), host(w), t.cpu().numpy(), host(lse), host(c)
    for i in range(tokens):
        one = slice(i, i + 1)
        (want, _), (bound, _) = ref.loss_gradients(hh[one], wh, th[one], lh[one], ch[one], 1.0, "f16")
        within(dh[one], want, bound + (th[i] >= 0) * abs(ch[i]) * 2.0 ** -13 * np.abs(wh).mean(0), f"dhidden {i}")
    (_, want), (_, bound) = ref.loss_gradients(hh, wh, th, lh, ch, 1.0, "f16")
    z, _ = ref.logits(hh, wh, 1.0)
    dz = np.exp(z - lh[:, None])
    dz[np.arange(tokens), np.maximum(th, 0)] -= 1
    low = np.abs(np.where(th >= 0, ch, 0.0)[:, None] * dz).T @ np.broadcast_to(2.0 ** -15 * np.abs(hh).max(1, keepdims=True), hh.shape)
    within(dw, want, bound + low, "dweight")
    again = op.backward(h, w, t, lse, dloss=c.cuda())
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)
    assert not op.stats.any()


def test_fp16_coefficients_that_are_not_finite():
    """They spoil their own token's gradient, and with it the table's; the other tokens' rows are as without them."""
    h, w, t, _ = loss_inputs(60, 200, 32, "f16", ids="full", seed=2)
    op = SoftmaxLoss(200, 32, 60, dtype=torch.float16)
    lse = op.forward(h, w, t)[1]
    c = torch.full((60,), 1e-5, device="cuda")
    c[1] = 1.0
    want = op.backward(h, w, t, lse, dloss=c)[0].clone()
    c[10], c[20] = float("inf"), float("nan")
    got = op.backward(h, w, t, lse, dloss=c)[0]
    keep = torch.ones(60, dtype=torch.bool, device="cuda")
    keep[10] = keep[20] = False
    assert torch.equal(got[keep], want[keep]) and not bool(torch.isfinite(got[~keep]).any())


# ------------------------------------------------------------------------------------------
# Statistics that pairs of CTAs carry from tile to tile
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("tokens", [128, 129, 130, 200, 255, 256])
def test_loss_of_one_tile_of_tokens_over_many_rows(tokens):
    """128 tokens: single CTAs; from 129 on pairs, more tiles of 256 rows than there are pairs, each pair's statistics one part."""
    check_loss(tokens, 30_011, 72, "bf16", ids="hot", seed=tokens)
    check_loss(tokens, 19_457, 40, "f16", itype="i32", seed=tokens, upstream="tokens")


def test_loss_and_its_statistics_of_256_tokens_over_70000_rows():
    h, w, t, t_h = loss_inputs(256, 70_000, 16, "f16", seed=3)
    op = SoftmaxLoss(70_000, 16, 256, dtype=torch.float16)
    out = op.forward(h, w, t)
    want, bound = ref.loss(host(h), host(w), t_h, 1.0)
    for got, v, b, name in zip(out, want, bound, ("loss", "lse", "mean")):
        within(got, v, b, name)


# ------------------------------------------------------------------------------------------
# The forward's workspace
# ------------------------------------------------------------------------------------------
def sampled_loss(tokens, rows, dim, dtype, seed, check):
    """A loss over a large table, its tokens `check` against the formula; targets at the pieces' borders and in each part."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(rows, dim, generator=g, device="cuda") * 2 / dim ** 0.5).to(dtype)
    h = torch.randn(tokens, dim, generator=g, device="cuda").to(dtype)
    t = torch.randint(0, rows, (tokens,), generator=g, device="cuda")
    t[1::9] = -1
    op = SoftmaxLoss(rows, dim, tokens, dtype=dtype)
    piece = -(-(-(-rows // 256)) // 2) * 256  # of two
    for k, at in enumerate((0, piece - 1, piece, rows - 1)):
        t[check[k % len(check)]] = at
        loss, lse, mean = op.forward(h, w, t)
        if k >= len(check) - 1:
            want, bound = ref.loss(host(h[check]), host(w), t[check].cpu().numpy(), 1.0)
            within(loss[check], want[0], bound[0], "loss")
            within(lse[check], want[1], bound[1], "lse")
    live = t >= 0
    assert not bool(loss[~live].any()) and not bool(lse[~live].any())
    n = int(live.sum())
    assert float(mean[1]) == pytest.approx(1 / n, rel=1e-6)
    assert float(mean[0]) == pytest.approx(float(loss.double().sum()) / n, rel=1e-6)
    assert not op.stats.any()


@pytest.mark.parametrize("tokens,rows,dim,check", [
    (1500, 3_000_001, 8, [0, 700, 1400, 1499]),        # tokens that count are gathered; several tiles of them
    (1_050_000, 5003, 16, [0, 255, 524_288, 1_049_999]),
    (300, 16_000_000, 8, [0, 299]),                    # two tiles, not gathered
])
def test_loss_in_two_pieces(tokens, rows, dim, check):
    """More than 2^32 logits, whose statistics are joined piece by piece."""
    sampled_loss(tokens, rows, dim, torch.bfloat16, tokens, check)


def test_loss_of_one_tile_of_tokens_in_two_pieces():
    """One tile of tokens over so many rows that it takes two pieces, whose statistics pairs carry (256 tokens)."""
    sampled_loss(256, 17_000_003, 8, torch.float16, 5, [0, 255])


def test_loss_of_few_tokens_in_two_pieces():
    """... and single CTAs (120)."""
    sampled_loss(120, 34_000_003, 8, torch.bfloat16, 6, [0, 119])


def test_a_piece_of_nothing_has_no_part_in_the_next():
    """The first piece's logits are all -inf, the second's -200: the sum of exponentials is the second's.  Its 8.5M terms are added
    in a chain of some 25000 additions at most, each within 2^-24; the logits and their constants lose 2^-13 at this size."""
    rows, piece = 17_000_003, -(-(-(-17_000_003 // 256)) // 2) * 256
    w = torch.full((rows, 8), -25.0, dtype=torch.float16, device="cuda")
    w[:piece] = float("-inf")
    h = torch.ones(256, 8, dtype=torch.float16, device="cuda")
    t = torch.full((256,), rows - 1, device="cuda")
    loss, lse, mean = SoftmaxLoss(rows, 8, 256, dtype=torch.float16).forward(h, w, t)
    n = np.log(rows - piece)
    err = 25000 * ref.U + 2.0 ** -13
    assert float((loss.double() - n).abs().max()) <= err and float((lse.double() - (n - 200)).abs().max()) <= err
    assert abs(float(mean[0]) - n) <= err


# ------------------------------------------------------------------------------------------
# Calls that the header allows and no test made
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dim", [1500, 4099, 65535, 65536])
def test_loss_of_wide_rows(dim):
    check_loss(70, 300, dim, "bf16", seed=dim, spread=1.0)
    check_loss(300, 40, dim, "f16", seed=dim, spread=1.0, upstream="tokens")


@pytest.mark.parametrize("dim,pad", [(45, 3), (301, 3), (8, 8), (1, 7)])
def test_loss_rows_of_odd_widths_at_aligned_strides(dim, pad):
    """Rows of which the last piece of 16 bytes is not whole, read where they lie."""
    check_loss(90, 400, dim, "bf16", pad=pad, seed=dim)
    check_loss(1100, 300, dim, "f16", pad=pad, seed=dim, upstream="tokens")


@pytest.mark.parametrize("dim,table,out", [(65536, "bf16", "bf16"), (65535, "f16", "f32"), (4100, "f32", "bf16")])
def test_lookup_of_wide_rows(dim, table, out):
    check_lookup(90, 30, dim, table, out, ids="hot", scale=0.7, seed=dim)
    check_lookup(700, 20, dim, table, out, accumulate=True, scale=0.7, seed=dim)


@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("accumulate", [False, True])
def test_lookup_gradient_of_more_than_a_cluster_sorts_into_rows_apart(pad, accumulate):
    check_lookup(140_001, 9000, 6, "bf16", "f32", ids="hot", itype="i32", pad=pad, accumulate=accumulate, seed=pad)


def test_the_tables_gradients_add_up_to_nothing():
    """The sum over the table's rows of dz is (sum of p) - 1 = 0 for every token, as far as lse is that of the logits and p
    of both.  Each entry of dz is rounded to bf16, each row of dweight too: half a step of its size; the sums over the tokens
    lose 2 N u of them."""
    tokens, rows, dim = 1000, 5000, 40
    h, w, t, t_h = loss_inputs(tokens, rows, dim, "bf16", seed=8)
    op = SoftmaxLoss(rows, dim, tokens)
    _, lse, mean = op.forward(h, w, t)
    dw = host(op.backward(h, w, t, lse, mean=mean)[1])
    live, hh = ref.masked(host(h), t_h, rows)
    l64 = host(lse)[:, None]
    z, ez = ref.logits(hh, host(w), 1.0)
    p = np.exp(z - l64)
    off = (p * (ref.exponent_error(z, l64, ez) * 1.01 + 4 * ref.U)).sum(1) + ref.loss(hh, host(w), t_h, 1.0)[1][1]  # of a token's sum
    dz = p.copy()
    dz[np.nonzero(live)[0], t_h[live]] -= 1
    size = np.abs(dz[live]).T @ np.abs(hh[live])
    bound = (size * (ref.STORE["bf16"] + 2 * tokens * ref.U)).sum(0) + off[live] @ np.abs(hh[live])
    bound = (bound * float(mean[1]) + np.abs(dw).sum(0) * ref.STORE["bf16"]) * 1.02
    assert (np.abs(dw.sum(0)) <= bound).all()


CAPTURE = """
import torch
from bwd_tbe_fwd_gb300 import SoftmaxLoss, TokenEmbedding
g = torch.Generator().manual_seed(1)
w = torch.randn({rows}, 72, generator=g).to(torch.bfloat16).cuda()
t = torch.randint(-1, {rows}, ({tokens},), generator=g).cuda()
emb = TokenEmbedding({rows}, 72, {tokens}, table_dtype=torch.bfloat16)
op = SoftmaxLoss({rows}, 72, {tokens})
def step():
    h = emb.forward(w, t)
    loss, lse, mean = op.forward(h, w, t)
    dh, dw = op.backward(h, w, t, lse, mean=mean)
    return [h, loss, lse, mean, dh, emb.backward(dh, t, grad=dw, accumulate=True), emb.backward(dh, t)]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in got]
want = step()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert not emb.stats.any() and not op.stats.any()
print("captured")
"""


@pytest.mark.parametrize("tokens,rows", [(40, 500), (3000, 4000), (140_000, 300)])
def test_a_graph_may_hold_a_process_s_first_calls(tokens, rows):
    """Nothing is loaded, asked or set up by a first call that a capture does not allow."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE.format(tokens=tokens, rows=rows)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "captured\n", r.stdout[-2000:] + r.stderr[-3000:]


def test_objects_for_no_tokens_and_calls_of_none():
    emb, op = TokenEmbedding(10, 8, 0, table_dtype=torch.float16), SoftmaxLoss(10, 8, 0, dtype=torch.float16)
    w = torch.ones(10, 8, dtype=torch.float16, device="cuda")
    ids = torch.zeros(0, 5, dtype=torch.int64, device="cuda")
    out = emb.forward(w, ids)
    assert out.shape == (0, 5, 8)
    wide = torch.full((10, 9), 7.0, dtype=torch.float16, device="cuda")
    assert not bool(emb.backward(out, ids, grad=wide[:, :8]).any()) and bool((wide[:, 8] == 7).all())
    wide[:, :8] = 7
    loss, lse, mean = op.forward(out.view(0, 8), w, ids.view(-1))
    dh, dw = op.backward(out.view(0, 8), w, ids.view(-1), lse, dloss=loss, mean=mean, dweight=wide[:, :8])
    assert loss.shape == lse.shape == (0,) and dh.shape == (0, 8) and mean.tolist() == [0, 0]
    assert not bool(dw.any()) and bool((wide[:, 8] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_upstream_gradients_of_padding_are_not_looked_at(dtype):
    h, w, t, t_h = loss_inputs(300, 200, 40, dtype, seed=11)
    op = SoftmaxLoss(200, 40, 300, dtype=w.dtype)
    lse = op.forward(h, w, t)[1]
    c = torch.rand(300, generator=gen(12)).cuda() + 0.5
    want = op.backward(h, w, t, lse, dloss=c)
    c[t < 0], lse[t < 0] = float("inf"), float("nan")
    assert all(torch.equal(a, b) for a, b in zip(op.backward(h, w, t, lse, dloss=c), want))
    assert not bool(want[0][t < 0].any())
