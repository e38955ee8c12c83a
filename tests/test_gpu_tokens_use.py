"""The token side (include/tbe_tokens.h) as programs use it: both ends of a model on one table, other streams, captured
graphs, two objects at once, values at the arithmetic's ends, and sizes that only large calls reach."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import tokens_reference as ref
from bwd_tbe_fwd_gb300 import SoftmaxLoss, TokenEmbedding
from test_gpu_tokens import check_loss, gen, host, loss_inputs, within

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------
# Together
# ------------------------------------------------------------------------------------------
def test_both_gradients_of_a_shared_table():
    """The loss's gradient of the table with the lookup's added to it.  The second is rounded once more in the sum: half a step
    of the sum's size."""
    tokens, rows, dim = 500, 300, 64
    g = gen(0)
    table = (torch.randn(rows, dim, generator=g) * 0.3).to(torch.bfloat16).cuda()
    ids = torch.randint(-1, rows, (tokens,), generator=g).cuda()
    targets = torch.randint(-1, rows, (tokens,), generator=g).cuda()
    emb = TokenEmbedding(rows, dim, tokens, table_dtype=torch.bfloat16, scale=2.0)
    op = SoftmaxLoss(rows, dim, tokens)
    hidden = emb.forward(table, ids)
    _, lse, mean = op.forward(hidden, table, targets)
    dhidden, dtable = op.backward(hidden, table, targets, lse, mean=mean)
    alone = dtable.clone()
    both = emb.backward(dhidden, ids, grad=dtable, accumulate=True)
    assert both is dtable
    coef = np.full(tokens, float(mean[1]))
    (_, want), (_, bound) = ref.loss_gradients(host(hidden), host(table), targets.cpu().numpy(), host(lse), coef, 1.0, "bf16")
    within(alone, want, bound, "loss")
    want, bound = ref.lookup_gradient(host(dhidden), ids.cpu().numpy(), rows, 2.0, "bf16", host(alone))
    within(both, want, bound, "both")


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_items.py")
    spec = importlib.util.spec_from_file_location("train_items", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_examples_gradients_are_autograds():
    """The gradients that a step leaves, against autograd in 64 bits on the same parameters.  Between them lie five values that
    are rounded to bf16 on the way (y, hidden, dz, d_hidden, d_y) and the gradients themselves, each off by 2^-9 of its
    size; what cancels in the sums makes that up to five times as much of the result's norm: 6 * 5 * 2^-9 < 6e-2."""
    m = example()
    model = m.Model()
    ids, targets = model.batch()
    table, dense, gain, shift = params = [p.double().requires_grad_() for p in model.params]
    flat, t = ids.view(-1), targets.view(-1)
    rows = torch.where((flat >= 0)[:, None], m.WIDTH ** 0.5 * table[flat.clamp(min=0)], 0.0)
    y = torch.nn.functional.layer_norm(rows, (m.WIDTH,), gain, shift, 1e-5)
    loss = torch.nn.functional.cross_entropy((y + y @ dense) @ table.T, t, ignore_index=-1)
    loss.backward()
    got = model.step(ids, targets, 1e-3)
    loss = float(loss.detach())
    assert abs(float(got[0]) - loss) <= 2 ** -6 * loss
    assert float(got[1]) == pytest.approx(1 / int((t >= 0).sum()), rel=1e-6)
    for g, p in zip(model.grads, params):
        assert float((g.double() - p.grad).norm()) <= 6e-2 * float(p.grad.norm())


def test_the_example_runs():
    model = example().Model()
    results = torch.stack([model.step(*model.batch(), lr=3e-3) for _ in range(5)])
    assert bool(torch.isfinite(results).all())


# ------------------------------------------------------------------------------------------
# Streams and graphs
# ------------------------------------------------------------------------------------------
class Both:
    """A lookup and a loss with their gradients, everything in given memory."""

    def __init__(self, seed, tokens=1500, rows=3000, dim=72, stream=None):
        self.h, self.w, self.t, _ = loss_inputs(tokens, rows, dim, "bf16", seed=seed)
        self.h = torch.where(torch.isnan(self.h), torch.zeros_like(self.h), self.h)
        self.emb = TokenEmbedding(rows, dim, tokens, table_dtype=torch.bfloat16, out_dtype=torch.float32)
        self.op = SoftmaxLoss(rows, dim, tokens)
        f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.out, self.grad = f(tokens, dim), torch.empty_like(self.w)
        self.loss, self.lse, self.mean = f(tokens), f(tokens), f(2)
        self.dh, self.dw = torch.empty_like(self.h), torch.empty_like(self.w)

    def run(self, stream=None):
        self.emb.forward(self.w, self.t, out=self.out, stream=stream)
        self.emb.backward(self.out, self.t, grad=self.grad, stream=stream)
        self.op.forward(self.h, self.w, self.t, loss=self.loss, lse=self.lse, mean=self.mean, stream=stream)
        self.op.backward(self.h, self.w, self.t, self.lse, mean=self.mean, dhidden=self.dh, dweight=self.dw, stream=stream)
        return [self.out, self.grad, self.loss, self.lse, self.mean, self.dh, self.dw]

    def results(self):
        return [x.clone() for x in (self.out, self.grad, self.loss, self.lse, self.mean, self.dh, self.dw)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_same_bits_on_another_stream():
    b = Both(1)
    b.run()
    want = b.results()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for x in (b.grad, b.dh, b.dw):
        x.fill_(1.0)
    side.wait_stream(torch.cuda.current_stream())
    b.run(stream=side)
    side.synchronize()
    assert same(b.results(), want)
    with torch.cuda.stream(side):
        out = b.op.forward(b.h, b.w, b.t)
        grads = b.op.backward(b.h, b.w, b.t, out[1], mean=out[2])
    side.synchronize()
    assert same([*out, *grads], want[2:])


def test_two_objects_at_once_on_two_streams():
    one, two = Both(2), Both(3, tokens=700, rows=5001, dim=136)
    wants = []
    for b in (one, two):
        b.run()
        torch.cuda.synchronize()
        wants.append(b.results())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for b, s in zip((one, two), streams):
            b.run(stream=s)
    torch.cuda.synchronize()
    assert same(one.results(), wants[0]) and same(two.results(), wants[1])


def test_in_a_graph_with_other_inputs():
    b = Both(4)
    stream = torch.cuda.Stream()
    b.run(stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        b.run()
        b.run()
    for seed in (5, 6):
        other = Both(seed)
        other.run()
        b.h.copy_(other.h), b.w.copy_(other.w), b.t.copy_(other.t)
        graph.replay()
        torch.cuda.synchronize()
        assert same(b.results(), other.results())


def test_objects_made_and_dropped_while_their_work_runs():
    side = torch.cuda.Stream()
    b = Both(7)
    b.run()
    want = b.results()
    torch.cuda.synchronize()
    for _ in range(3):
        op = SoftmaxLoss(3000, 72, 1500)
        grads = op.backward(b.h, b.w, b.t, b.lse, mean=b.mean, stream=side)
        del op
        trash = torch.full((1 << 28,), 7, dtype=torch.uint8, device="cuda")
        side.synchronize()
        assert same(grads, want[5:])
        del trash


def test_an_object_serves_fewer_tokens():
    """What the splits and pieces take for fewer tokens fits a workspace for more."""
    op = SoftmaxLoss(2000, 264, 5000)
    for tokens in (1, 40, 300, 1024, 3000, 5000):
        h, w, t, t_h = loss_inputs(tokens, 2000, 264, "bf16", seed=tokens)
        own = SoftmaxLoss(2000, 264, tokens)
        out, want = op.forward(h, w, t), own.forward(h, w, t)
        assert same(out, want)
        assert same(op.backward(h, w, t, out[1], mean=out[2]), own.backward(h, w, t, out[1], mean=out[2]))


def test_hidden_may_begin_anywhere():
    g = gen(8)
    wide = torch.randn(60, 96, generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(500, 72, generator=g).to(torch.bfloat16).cuda()
    t = torch.randint(0, 500, (60,), generator=g).cuda()
    op = SoftmaxLoss(500, 72, 60)
    want = None
    for at in (0, 1, 4, 8):
        h = wide.clone()
        h = torch.cat([h[:, :72], h], 1)[:, :168].contiguous()
        h[:, at:at + 72] = wide[:, :72]
        h = h[:, at:at + 72]
        out = op.forward(h, w, t)
        res = [*out, *op.backward(h, w, t, out[1], mean=out[2])]
        want = want or [x.clone() for x in res]
        assert same(res, want)


# ------------------------------------------------------------------------------------------
# Values
# ------------------------------------------------------------------------------------------
def test_a_row_that_is_not_finite_spoils_its_own_loss_alone():
    h, w, t, _ = loss_inputs(300, 400, 64, "bf16", ids="full", seed=9)
    op = SoftmaxLoss(400, 64, 300)
    want = op.forward(h, w, t)[0].clone()
    h[17, 3], h[200, 5] = float("inf"), float("nan")
    loss = op.forward(h, w, t)[0]
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[17] = keep[200] = False
    assert torch.equal(loss[keep], want[keep]) and not bool(torch.isfinite(loss[~keep]).any())


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-12, 1e12, 1e30])
def test_upstream_gradients_of_any_size(size):
    """dz is scaled by a factor that the largest coefficient gives: bf16's gradients keep their accuracy at any size."""
    h, w, t, t_h = loss_inputs(100, 200, 64, "bf16", seed=10)
    op = SoftmaxLoss(200, 64, 100)
    lse = op.forward(h, w, t)[1]
    dloss = torch.randn(100, generator=gen(11)).cuda() * size
    grads = op.backward(h, w, t, lse, dloss=dloss)
    want, bound = ref.loss_gradients(host(h), host(w), t_h, host(lse), host(dloss), 1.0, "bf16")
    for got, v, b, name in zip(grads, want, bound, ("dhidden", "dweight")):
        within(got, v, b, name)


def test_fp16_gradients_of_a_mean_over_many_rows():
    """Probabilities of 2^-17 times coefficients of 2^-8 lie below fp16's least value; what they add up to does not."""
    g = gen(12)
    tokens, rows, dim = 256, 70_000, 16
    h = torch.ones(tokens, dim).half().cuda()
    w = torch.zeros(rows, dim).half().cuda()
    w[::2] = 2.0 ** -6
    t = torch.randint(0, rows, (tokens,), generator=g).cuda()
    op = SoftmaxLoss(rows, dim, tokens, dtype=torch.float16)
    _, lse, mean = op.forward(h, w, t)
    dh, dw = op.backward(h, w, t, lse, dloss=torch.full((tokens,), 2.0 ** 8, device="cuda"), mean=mean)
    coef = np.full(tokens, 2.0 ** 8 * float(mean[1]))
    want, bound = ref.loss_gradients(host(h), host(w), t.cpu().numpy(), host(lse), coef, 1.0, "f16")
    within(dh, want[0], bound[0], "dhidden")
    within(dw, want[1], bound[1], "dweight")
    assert float(dw.float().abs().min()) > 0


# ------------------------------------------------------------------------------------------
# Sizes
# ------------------------------------------------------------------------------------------
def sampled_loss_check(h, w, t, scale, store, loss, lse, coef, dh, dw, rows, tokens):
    """`rows` of dweight and `tokens` of loss, lse and dhidden against the formulas; lse, where it is an input, as given."""
    t_h = t.cpu().numpy()
    hs, ws = host(h[tokens]), host(w)
    want, bound = ref.loss(hs, ws, t_h[tokens], scale)
    within(loss[tokens], want[0], bound[0], "loss")
    within(lse[tokens], want[1], bound[1], "lse")
    top = np.abs(coef).max()
    (g, _), (e, _) = ref.loss_gradients(hs, ws, t_h[tokens], host(lse[tokens]), coef[tokens], scale, store)
    within(dh[tokens], g, e + top * 2.0 ** -13 * ref.TINY[store] * 2 * np.abs(ws).sum(0) * scale, "dhidden")
    # the rows of dweight: the table cut down to them, with lse of the whole, targets elsewhere gone but the tokens live
    at = np.full(len(ws), -1)
    at[rows] = np.arange(len(rows))
    hall, wr = host(h), ws[rows]
    live = t_h >= 0
    z, ez = ref.logits(np.where(live[:, None], hall, 0.0), wr, scale)
    l64 = np.where(live, host(lse), 0.0)[:, None]
    p = np.exp(z - l64)
    dz = p.copy()
    mine = np.nonzero(live & (at[np.where(live, t_h, 0)] >= 0))[0]
    dz[mine, at[t_h[mine]]] -= 1
    c = np.where(live, coef, 0.0)[:, None]
    edz = np.abs(c) * p * (ref.exponent_error(z, l64, ez) * 1.01 + 4 * ref.U) + np.abs(c * dz) * (ref.STORE[store] * 1.01 + 4 * ref.U) \
        + top * 2.0 ** -13 * ref.TINY[store] * 2
    hall = np.where(live[:, None], hall, 0.0)
    got = scale * ((c * dz).T @ hall)
    err = scale * (edz.T @ np.abs(hall) * 1.01 + (2 * len(hall) + 64) * ref.U * (np.abs(c * dz).T @ np.abs(hall)))
    within(dw[rows], got, err + ref.rounded(got, store), "dweight")


def big_loss(tokens, rows, dim, dtype, store, seed, sample):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(rows, dim, generator=g, device="cuda") * 2 / dim ** 0.5).to(dtype)
    h = torch.randn(tokens, dim, generator=g, device="cuda").to(dtype)
    t = torch.randint(0, rows, (tokens,), generator=g, device="cuda")
    t[::7] = -1
    op = SoftmaxLoss(rows, dim, tokens, dtype=dtype)
    loss, lse, mean = op.forward(h, w, t)
    dh, dw = op.backward(h, w, t, lse, mean=mean)
    coef = np.full(tokens, float(mean[1]))
    sampled_loss_check(h, w, t, 1.0, store, loss, lse, coef, dh, dw, np.array(sorted(set(sample))), np.arange(0, tokens, max(1, tokens // 23)))
    assert not op.stats.any()
    # the sum over the table's rows of dz is zero for every token, so dweight adds up to nothing but rounding
    return dw


def test_loss_in_several_pieces_of_the_table():
    """4096 tokens by 200000 rows: dz takes 512 MB for 65536 rows, so four pieces, the last one shorter; odd rows at the borders."""
    rows = 200_003
    piece = -(-(-(-rows // 4)) // 256) * 256
    sample = [0, 1, 255, 256, piece - 1, piece, piece + 1, 2 * piece - 1, 2 * piece, 3 * piece - 1, 3 * piece, rows - 2, rows - 1]
    big_loss(4096, rows, 40, torch.bfloat16, "bf16", 1, sample)
    big_loss(4100, rows, 33, torch.bfloat16, "bf16", 2, sample)


def test_loss_over_a_table_of_more_than_2_to_the_31_elements():
    rows, dim = 4_200_000, 520
    dw = big_loss(8, rows, dim, torch.bfloat16, "bf16", 3, [0, rows // 2, 4_130_055, 4_130_056, rows - 1])
    assert bool(torch.isfinite(dw[-1].float()).all())


def test_lookup_in_a_table_of_more_than_2_to_the_32_elements():
    rows, dim = 34_000_000, 128
    emb = TokenEmbedding(rows, dim, 5000, table_dtype=torch.float16, index_dtype=torch.int32, scale=0.5)
    table = torch.empty(rows, dim, dtype=torch.float16, device="cuda")
    table.fill_(1.0)
    ids = torch.randint(rows - 1000, rows, (5000,), generator=gen(13), dtype=torch.int32).cuda()
    ids[:3] = torch.tensor([0, rows - 1, 33_554_433], dtype=torch.int32)
    where = torch.arange(rows - 1000, rows, device="cuda")
    table[where] = (torch.arange(1000, device="cuda") % 512).half()[:, None].expand(-1, dim)
    out = emb.forward(table, ids)
    assert torch.equal(out, (table[ids.long()].float() * 0.5).half())
    dout = torch.ones(5000, dim, dtype=torch.float16, device="cuda")
    grad = emb.backward(dout, ids, grad=table)
    count = torch.bincount((ids.long() - (rows - 1000)).clamp(min=0), minlength=1000)
    count[0] -= 2 if int(ids[2]) < rows - 1000 else 1
    assert torch.equal(grad[where][:, 0].float(), count.float() * 0.5)
    assert float(grad[0, 0]) == 0.5 and float(grad[33_554_433, 5]) == 0.5
    total = sum(float(part.float().sum()) for part in grad.split(1 << 20))
    assert total == 5000 * dim * 0.5
