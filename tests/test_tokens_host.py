"""The token side (include/tbe_tokens.h) on the host: refusals of its entry points before any launch, what the binding
refuses, the device and stream that it calls them with, and the 64-bit references' own soundness.  No GPU is needed."""
import ctypes
import math
import types

import numpy as np
import pytest
import torch

import tokens_reference as ref
from bwd_tbe_fwd_gb300 import build as tbe_build
from bwd_tbe_fwd_gb300 import dense, tbe, tokens

INVALID, UNSUPPORTED, WORKSPACE = tbe.TBE_ERR_INVALID_ARG, tbe.TBE_ERR_UNSUPPORTED, tbe.TBE_ERR_WORKSPACE
A = ctypes.c_void_p(1 << 16)       # stands for an aligned buffer; no call below gets as far as using it
B = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 16) + 1)
EIGHT = ctypes.c_void_p((1 << 16) + 8)


@pytest.fixture(scope="module")
def lib():
    tbe_build.build()
    return tokens._bind(tbe.load())


# ------------------------------------------------------------------------------------------
# Lookup
# ------------------------------------------------------------------------------------------
def lookup(**kw):
    f = dict(tokens=4, rows=10, dim=8, table_stride=8, out_stride=8, tdtype=tbe.TBE_F32, odtype=tbe.TBE_F32, itype=tbe.TBE_I64,
             scale=1.0)
    f.update(kw)
    return tokens.LookupProblem(*f.values())


def lookup_forward(lib, p, table=A, ids=A, out=B, stats=None):
    return lib.tbe_lookup_forward(ctypes.byref(p), table, ids, out, stats, None)


def lookup_backward(lib, p, dout=A, ids=A, grad=B, ws=A, n=1 << 40, stats=None):
    return lib.tbe_lookup_backward(ctypes.byref(p), dout, ids, grad, 0, ws, n, stats, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(tokens=-1), INVALID), (dict(rows=0), INVALID), (dict(dim=0), INVALID), (dict(table_stride=7), INVALID),
    (dict(out_stride=7), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(tokens=(1 << 31) - (1 << 16) + 1), UNSUPPORTED), (dict(dim=65537, table_stride=1 << 20, out_stride=1 << 20), UNSUPPORTED),
    (dict(tokens=1 << 30, dim=1025, table_stride=1025, out_stride=1025), UNSUPPORTED),
    (dict(rows=(1 << 31) - 1, table_stride=1 << 40), UNSUPPORTED), (dict(out_stride=1 << 62), UNSUPPORTED),
    (dict(tdtype=5), UNSUPPORTED), (dict(odtype=-1), UNSUPPORTED), (dict(itype=2), UNSUPPORTED),
    (dict(tdtype=tbe.TBE_F16, odtype=tbe.TBE_BF16), UNSUPPORTED),
])
def test_lookup_refuses_bad_problems(lib, kw, expect):
    p = lookup(**kw)
    assert lookup_forward(lib, p) == expect
    assert lookup_backward(lib, p) == expect
    assert lib.tbe_lookup_backward_workspace_size(ctypes.byref(p)) == 0


def test_lookup_refuses_bad_buffers(lib):
    p = lookup()
    for kw in (dict(table=None), dict(ids=None), dict(out=None), dict(table=ODD), dict(out=ODD), dict(ids=ctypes.c_void_p((1 << 16) + 4)),
               dict(stats=ctypes.c_void_p((1 << 16) + 4))):
        assert lookup_forward(lib, p, **kw) == INVALID, kw
    for kw in (dict(dout=None), dict(ids=None), dict(grad=None), dict(dout=ODD), dict(grad=ODD), dict(ids=EIGHT, grad=ODD)):
        assert lookup_backward(lib, p, **kw) == INVALID, kw
    assert lookup_forward(lib, lookup(tokens=0), table=None, ids=None, out=None) == tbe.TBE_OK
    assert lib.tbe_lookup_forward(None, A, A, B, None, None) == INVALID


# ------------------------------------------------------------------------------------------
# Softmax cross entropy
# ------------------------------------------------------------------------------------------
def softmax(**kw):
    f = dict(tokens=4, rows=10, dim=8, hidden_stride=8, weight_stride=8, dhidden_stride=8, dweight_stride=8, dtype=tbe.TBE_BF16,
             itype=tbe.TBE_I64, scale=1.0)
    f.update(kw)
    return tokens.SoftmaxProblem(*f.values())


def loss_forward(lib, p, hidden=A, weight=A, targets=A, loss=B, lse=B, mean=B, ws=A, n=1 << 40, stats=None):
    return lib.tbe_softmax_loss_forward(ctypes.byref(p), hidden, weight, targets, loss, lse, mean, ws, n, stats, None)


def loss_backward(lib, p, hidden=A, weight=A, targets=A, lse=A, dloss=A, mean=A, dhidden=B, dweight=B, ws=A, n=1 << 40, stats=None):
    return lib.tbe_softmax_loss_backward(ctypes.byref(p), hidden, weight, targets, lse, dloss, mean, dhidden, dweight, ws, n, stats, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(tokens=-1), INVALID), (dict(rows=0), INVALID), (dict(dim=0), INVALID), (dict(hidden_stride=7), INVALID),
    (dict(weight_stride=7), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(tokens=(1 << 24) + 1), UNSUPPORTED), (dict(rows=(1 << 31) - (1 << 16)), UNSUPPORTED),
    (dict(tokens=1 << 24, rows=1 << 30), UNSUPPORTED), (dict(dim=65537, hidden_stride=1 << 17, weight_stride=1 << 17, dhidden_stride=1 << 17, dweight_stride=1 << 17), UNSUPPORTED),
    (dict(dtype=tbe.TBE_F32), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(itype=7), UNSUPPORTED), (dict(hidden_stride=1 << 39), UNSUPPORTED),
])
def test_loss_refuses_bad_problems(lib, kw, expect):
    p = softmax(**kw)
    assert loss_forward(lib, p) == expect
    assert loss_backward(lib, p) == expect
    assert lib.tbe_softmax_loss_workspace_size(ctypes.byref(p)) == 0
    assert lib.tbe_softmax_loss_backward_workspace_size(ctypes.byref(p)) == 0


def test_loss_refuses_bad_buffers(lib):
    p = softmax()
    for kw in (dict(hidden=None), dict(weight=None), dict(targets=None), dict(loss=None), dict(lse=None), dict(mean=None), dict(hidden=ODD),
               dict(weight=EIGHT), dict(targets=ctypes.c_void_p((1 << 16) + 4)), dict(loss=ODD), dict(lse=ODD), dict(mean=ODD), dict(ws=EIGHT),
               dict(stats=ctypes.c_void_p(4))):
        assert loss_forward(lib, p, **kw) == INVALID, kw
    for kw in (dict(hidden=None), dict(weight=None), dict(targets=None), dict(lse=None), dict(dhidden=None), dict(dweight=None), dict(hidden=ODD),
               dict(weight=EIGHT), dict(dloss=ODD), dict(mean=ODD), dict(dhidden=ODD), dict(dweight=ODD)):
        assert loss_backward(lib, p, **kw) == INVALID, kw
    for kw in (dict(dhidden_stride=7), dict(dweight_stride=7)):
        assert loss_backward(lib, softmax(**kw)) == INVALID
    need = lib.tbe_softmax_loss_workspace_size(ctypes.byref(p))
    assert need > 0 and loss_forward(lib, p, n=need - 1) == WORKSPACE and loss_forward(lib, p, ws=None) == WORKSPACE
    assert lib.tbe_softmax_loss_forward(None, A, A, A, B, B, B, A, need, None, None) == INVALID


def test_loss_workspace_serves_fewer_tokens(lib):
    """The forward's (the backward's asks the device for its size): never less for more tokens, whatever the strides of hidden."""
    for dim in (8, 301):
        last = 0
        for n in (1, 31, 33, 255, 257, 1023, 1025, 5000, 70_000):
            sizes = {lib.tbe_softmax_loss_workspace_size(ctypes.byref(softmax(tokens=n, dim=dim, rows=5000, weight_stride=dim, hidden_stride=s)))
                     for s in (dim, dim + 1, dim + 8)}
            assert len(sizes) == 1 and min(sizes) >= last
            last = min(sizes)


# ------------------------------------------------------------------------------------------
# Binding
# ------------------------------------------------------------------------------------------
class FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            if name.endswith("size"):
                return 16
            self.calls.append((name, getattr(args[-1], "value", args[-1])))
            return tbe.TBE_OK
        return fn


@pytest.fixture
def fake(monkeypatch):
    fake = FakeLib()
    for module in (dense, tokens):
        monkeypatch.setattr(module, "load", lambda: fake)
        monkeypatch.setattr(module, "_bind", lambda lib: lib)
    entered = []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)

        def __exit__(self, *exc):
            return False

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=1000))
    fake.entered = entered
    return fake


def test_every_call_runs_on_the_tensors_device_and_stream(fake):
    emb = tokens.TokenEmbedding(10, 8, 6, device="cpu")
    op = tokens.SoftmaxLoss(10, 8, 6, device="cpu")
    ids, table = torch.zeros(6, dtype=torch.int64), torch.zeros(10, 8)
    h, w = torch.zeros(6, 8, dtype=torch.bfloat16), torch.zeros(10, 8, dtype=torch.bfloat16)
    mine = types.SimpleNamespace(cuda_stream=4242)
    for stream, expect in ((None, 1000), (mine, 4242)):
        fake.calls.clear(), fake.entered.clear()
        out = emb.forward(table, ids, out=torch.zeros(6, 8), stream=stream)
        emb.backward(out, ids, grad=table, stream=stream)
        loss, lse, mean = op.forward(h, w, ids, loss=torch.zeros(6), lse=torch.zeros(6), mean=torch.zeros(2), stream=stream)
        op.backward(h, w, ids, lse, mean=mean, dhidden=h, dweight=w, stream=stream)
        assert [c[0] for c in fake.calls] == ["tbe_lookup_forward", "tbe_lookup_backward", "tbe_softmax_loss_forward",
                                              "tbe_softmax_loss_backward"]
        assert all(s == expect for _, s in fake.calls)
        assert fake.entered == [torch.device("cpu")] * 4


def test_the_binding_refuses(fake):
    emb = tokens.TokenEmbedding(10, 8, 6, table_dtype=torch.float16, out_dtype=torch.float32, device="cpu")
    ids, table, dout = torch.zeros(6, dtype=torch.int64), torch.zeros(10, 8, dtype=torch.float16), torch.zeros(6, 8)
    for args, error in (((table, ids.int()), TypeError), ((table.float(), ids), TypeError), ((table[:9], ids), ValueError),
                        ((table, torch.zeros(7, dtype=torch.int64)), ValueError), ((table.T.contiguous().T, ids), ValueError),
                        ((table, torch.zeros(12, dtype=torch.int64)[::2]), ValueError), ((table[:1].expand(10, 8), ids), ValueError)):
        with pytest.raises(error):
            emb.forward(*args)
    for args, kw, error in (((dout.half(), ids), {}, TypeError), ((dout[:5], ids), {}, ValueError), ((dout, ids), dict(grad=table.float()), TypeError),
                            ((dout, ids), dict(accumulate=True), ValueError), ((dout.view(6, 1, 8), ids), {}, ValueError)):
        with pytest.raises(error):
            emb.backward(*args, **kw)
    assert emb.forward(table, ids.view(2, 3)).shape == (2, 3, 8)
    assert emb.backward(dout.view(2, 3, 8), ids.view(2, 3)).shape == (10, 8)
    with pytest.raises(TypeError):
        tokens.TokenEmbedding(10, 8, 6, index_dtype=torch.int16, device="cpu")

    op = tokens.SoftmaxLoss(10, 8, 6, device="cpu")
    h, w, lse = torch.zeros(6, 8, dtype=torch.bfloat16), torch.zeros(10, 8, dtype=torch.bfloat16), torch.zeros(6)
    for args, kw, error in (((h.float(), w, ids), {}, TypeError), ((h, w[:9], ids), {}, ValueError), ((h[:5], w, ids), {}, ValueError),
                            ((h, torch.zeros(10, 9, dtype=torch.bfloat16)[:, :8], ids), {}, ValueError),
                            ((h, torch.zeros(84, dtype=torch.bfloat16)[4:].view(10, 8), ids), {}, ValueError),
                            ((h, w, ids), dict(loss=torch.zeros(5)), ValueError), ((h, w, ids), dict(mean=torch.zeros(2).double()), TypeError)):
        with pytest.raises(error):
            op.forward(*args, **kw)
    for args, kw, error in (((h, w, ids, lse[:5]), {}, ValueError), ((h, w, ids, lse), dict(dloss=lse.double()), TypeError),
                            ((h, w, ids, lse), dict(mean=lse), ValueError), ((h, w, ids, lse), dict(dweight=w[:, :7]), ValueError)):
        with pytest.raises(error):
            op.backward(*args, **kw)


# ------------------------------------------------------------------------------------------
# The references
# ------------------------------------------------------------------------------------------
def test_reference_gradients_are_difference_quotients():
    r = np.random.default_rng(0)
    h, w, t = r.standard_normal((5, 3)), r.standard_normal((7, 3)), np.array([2, -1, 6, 0, 2])
    coef, scale = r.standard_normal(5), 0.5
    (_, lse, _), _ = ref.loss(h, w, t, scale)
    (dh, dw), _ = ref.loss_gradients(h, w, t, lse, coef, scale, "f32")
    step = 1e-6  # central quotient: step^2 and 1e-16 / step

    def total(h, w):
        return (ref.loss(h, w, t, scale)[0][0] * coef).sum()

    for grad, k in ((dh, 0), (dw, 1)):
        for at in np.ndindex(grad.shape):
            args = [[h.copy(), w.copy()] for _ in range(2)]
            args[0][k][at] += step
            args[1][k][at] -= step
            assert abs((total(*args[0]) - total(*args[1])) / (2 * step) - grad[at]) <= 1e-7 * (1 + np.abs(grad).max())


def test_reference_loss_is_torchs():
    r = torch.Generator().manual_seed(1)
    h, w = torch.randn(9, 4, generator=r, dtype=torch.float64), torch.randn(11, 4, generator=r, dtype=torch.float64)
    t = torch.tensor([0, 10, -1, 3, 3, -1, 7, 8, 9])
    (loss, _, mean), _ = ref.loss(h.numpy(), w.numpy(), t.numpy(), 2.0)
    want = torch.nn.functional.cross_entropy(2.0 * h @ w.T, t, ignore_index=-1, reduction="none")
    np.testing.assert_allclose(loss, want.numpy(), rtol=1e-12, atol=1e-12)
    assert abs(mean[0] - float(want[t >= 0].mean())) < 1e-12 and mean[1] == 1 / 7


def test_reference_lookup():
    table = np.arange(12.0).reshape(4, 3)
    out, _ = ref.lookup(table, np.array([3, -1, 9, 0]), 2.0, "f32")
    assert out.tolist() == [[18, 20, 22], [0, 0, 0], [0, 0, 0], [0, 2, 4]]
    grad, bound = ref.lookup_gradient(np.ones((4, 3)), np.array([1, 1, -1, 4]), 4, 0.5, "f32")
    assert grad[:, 0].tolist() == [0, 1, 0, 0] and (bound[[0, 2, 3]] == 0).all()
