"""The dense side (include/tbe_dense.h) on the host: refusals of its entry points before any launch, the device and
stream that the binding calls them with, and the 64-bit references' own soundness.  No GPU is needed."""
import ctypes
import math
import types

import numpy as np
import pytest
import torch

import dense_reference as ref
from bwd_tbe_fwd_gb300 import build as tbe_build
from bwd_tbe_fwd_gb300 import dense, tbe

OK, INVALID, UNSUPPORTED, WORKSPACE = tbe.TBE_OK, tbe.TBE_ERR_INVALID_ARG, tbe.TBE_ERR_UNSUPPORTED, tbe.TBE_ERR_WORKSPACE
A = ctypes.c_void_p(4096)      # stands for an aligned buffer; no call below gets as far as using it
ODD = ctypes.c_void_p(4096 + 1)


@pytest.fixture(scope="module")
def lib():
    tbe_build.build()
    return dense._bind(tbe.load())


def norm_problem(widths=(64,), rows=4, **kw):
    w = (ctypes.c_int32 * len(widths))(*widths)
    n = sum(widths)
    f = dict(rows=rows, segments=len(widths), widths=w, col_offsets=4096, x_stride=n, y_stride=n, dx_stride=n,
             xdtype=tbe.TBE_F32, ydtype=tbe.TBE_F32, wdtype=tbe.TBE_F32, eps=1e-5)
    f.update(kw)
    p = dense.NormProblem(*f.values())
    p._keep = w
    return p


def forward(lib, p, x=A, w=A, b=A, y=ctypes.c_void_p(8192), mean=A, rstd=A):
    return lib.tbe_layer_norm_forward(ctypes.byref(p), x, w, b, y, mean, rstd, None)


def backward(lib, p, dy=A, x=ctypes.c_void_p(8192), mean=A, rstd=A, w=A, dx=ctypes.c_void_p(1 << 14), dw=A, db=A, ws=A,
             n=1 << 30):
    return lib.tbe_layer_norm_backward(ctypes.byref(p), dy, x, mean, rstd, w, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=-1), INVALID), (dict(segments=0), INVALID), (dict(widths=(64, 0)), INVALID), (dict(widths=(-4,)), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(xdtype=7), UNSUPPORTED), (dict(wdtype=-1), UNSUPPORTED), (dict(xdtype=tbe.TBE_F16, ydtype=tbe.TBE_BF16), UNSUPPORTED),
    (dict(widths=(64, 32), col_offsets=None), INVALID), (dict(x_stride=63), INVALID), (dict(y_stride=0), INVALID),
    (dict(widths=(4,) * 4097), UNSUPPORTED), (dict(widths=(1 << 30, 1 << 30)), UNSUPPORTED),
])
def test_norm_refuses_bad_problems(lib, kw, expect):
    p = norm_problem(**kw)
    assert forward(lib, p) == expect
    assert backward(lib, p) == expect
    if "x_stride" not in kw and "y_stride" not in kw:
        assert lib.tbe_layer_norm_backward_workspace_size(ctypes.byref(p)) == 0


def test_norm_refuses_bad_buffers(lib):
    p = norm_problem()
    for kw in (dict(x=None), dict(y=None), dict(x=ODD), dict(y=ODD), dict(w=ODD), dict(b=ODD), dict(mean=None), dict(rstd=None),
               dict(mean=ODD, rstd=ODD)):
        assert forward(lib, p, **kw) == INVALID, kw
    for kw in (dict(x=None), dict(dy=None), dict(mean=None), dict(rstd=None), dict(x=ODD), dict(dy=ODD), dict(dx=ODD),
               dict(dw=ODD), dict(db=ODD), dict(w=ODD), dict(mean=ODD)):
        assert backward(lib, p, **kw) == INVALID, kw
    assert backward(lib, norm_problem(dx_stride=1)) == INVALID
    # in place only with the same type and stride
    assert forward(lib, norm_problem(ydtype=tbe.TBE_BF16), x=A, y=A) == INVALID
    assert forward(lib, norm_problem(y_stride=128), x=A, y=A) == INVALID
    assert backward(lib, norm_problem(ydtype=tbe.TBE_BF16), dy=A, dx=A) == INVALID
    assert backward(lib, norm_problem(dx_stride=128), x=A, dx=A) == INVALID
    assert forward(lib, norm_problem(rows=0)) == OK
    assert backward(lib, norm_problem(), dx=None, dw=None, db=None) == OK
    assert lib.tbe_layer_norm_forward(None, A, A, A, A, A, A, None) == INVALID


def test_grad_norm_refuses(lib):
    n = lib.tbe_grad_norm_workspace_size()
    ptrs, sizes = (ctypes.c_void_p * 2)(4096, 8192), (ctypes.c_int64 * 2)(3, 5)

    def call(count=2, ptrs=ptrs, sizes=sizes, dtype=tbe.TBE_F32, max_norm=1.0, out=A, ws=A, size=n):
        return lib.tbe_grad_norm(count, ptrs, sizes, dtype, max_norm, out, ws, size, None)

    for kw in (dict(count=-1), dict(ptrs=None), dict(sizes=None), dict(out=None), dict(out=ODD), dict(max_norm=-1.0),
               dict(max_norm=math.nan), dict(ws=ODD), dict(sizes=(ctypes.c_int64 * 2)(3, -1)),
               dict(ptrs=(ctypes.c_void_p * 2)(4096, None)), dict(ptrs=(ctypes.c_void_p * 2)(4096, 8193))):
        assert call(**kw) == INVALID, kw
    assert call(dtype=9) == UNSUPPORTED
    assert call(sizes=(ctypes.c_int64 * 2)(3, 1 << 41)) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(size=n - 1) == WORKSPACE


def adamw_problem(states=dense.TBE_STATE_F32, pdtype=tbe.TBE_F32, betas=(0.9, 0.999), eps=1e-8, **kw):
    f = dict(param=4096, grad=8192, master=None, exp_avg=1 << 14, exp_avg_sq=1 << 15, exp_avg_scale=1 << 16,
             exp_avg_sq_scale=1 << 17, numel=10, lr_scale=1.0, weight_decay=0.0)
    f.update(kw)
    t = (dense.DenseTensor * 2)(dense.DenseTensor(*f.values()), dense.DenseTensor(*f.values()))
    p = dense.AdamWProblem(2, t, pdtype, tbe.TBE_F32, states, *betas, eps)
    p._keep = t
    return p


def test_adamw_refuses(lib):
    n = lib.tbe_adamw_workspace_size()

    def call(p, lr=0.1, clip=None, step=A, ws=A, size=n):
        return lib.tbe_adamw_update(ctypes.byref(p), lr, clip, step, ws, size, None)

    q8 = dense.TBE_STATE_Q8
    for kw in (dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None), dict(param=4097), dict(grad=8194),
               dict(exp_avg=(1 << 14) + 2), dict(master=4098), dict(numel=-1), dict(lr_scale=math.nan),
               dict(weight_decay=math.inf), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(betas=(math.nan, 0.9)),
               dict(eps=-1.0), dict(eps=math.inf), dict(states=5), dict(states=q8, exp_avg_scale=None),
               dict(states=q8, exp_avg_sq_scale=(1 << 17) + 2)):
        assert call(adamw_problem(**kw)) == INVALID, kw
    for kw in (dict(lr=math.nan), dict(lr=math.inf), dict(step=None), dict(step=ctypes.c_void_p(4100)), dict(clip=ODD),
               dict(ws=ODD)):
        assert call(adamw_problem(), **kw) == INVALID, kw
    assert call(adamw_problem(pdtype=4)) == UNSUPPORTED
    assert call(adamw_problem(numel=1 << 41)) == UNSUPPORTED
    assert call(adamw_problem(master=4096)) == UNSUPPORTED  # fp32 params are their own master
    p = adamw_problem(pdtype=tbe.TBE_BF16, master=4096)
    p.tensors[1].master = None
    assert call(p) == UNSUPPORTED  # all tensors have one, or none
    assert call(adamw_problem(), ws=None) == WORKSPACE and call(adamw_problem(), size=n - 1) == WORKSPACE
    p = adamw_problem()
    p.count = -1
    assert call(p) == INVALID
    assert lib.tbe_adamw_update(None, 0.1, None, A, A, n, None) == INVALID
    assert lib.tbe_adamw_state_values(ctypes.byref(adamw_problem()), None, None, None) == INVALID  # fp32 states
    odd = (ctypes.c_void_p * 2)(4096, 4098)
    assert lib.tbe_adamw_state_values(ctypes.byref(adamw_problem(states=q8)), odd, None, None) == INVALID


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
    monkeypatch.setattr(dense, "load", lambda: fake)
    monkeypatch.setattr(dense, "_bind", lambda lib: lib)
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
    x = torch.zeros(3, 12)
    ln = dense.LayerNorm([8, 4], device="cpu")
    opt = dense.DenseAdamW([x], [x.clone()], "q8", device="cpu")
    norm = dense.GradNorm([x])
    mine = types.SimpleNamespace(cuda_stream=4242)
    for stream, expect in ((None, 1000), (mine, 4242)):
        fake.calls.clear(), fake.entered.clear()
        y, mean, rstd = ln.forward(x, y=x.clone(), mean=torch.zeros(3, 2), rstd=torch.zeros(3, 2), stream=stream)
        ln.backward(x, x, mean, rstd, dx=y, dweight=torch.zeros(12), dbias=torch.zeros(12), stream=stream)
        norm.compute(1.0, out=torch.zeros(2), stream=stream)
        opt.step(0.1, stream=stream)
        opt.state_values([torch.zeros(36)], [torch.zeros(36)], stream=stream)
        assert [c[0] for c in fake.calls] == ["tbe_layer_norm_forward", "tbe_layer_norm_backward", "tbe_grad_norm",
                                              "tbe_adamw_update", "tbe_adamw_state_values"]
        assert all(s == expect for _, s in fake.calls)
        assert fake.entered == [torch.device("cpu")] * 5


# ------------------------------------------------------------------------------------------
# The references
# ------------------------------------------------------------------------------------------
def test_reference_gradients_are_difference_quotients():
    r = np.random.default_rng(0)
    widths, rows = [5, 8], 4
    x, dy = r.standard_normal((2, rows, 13))
    w, b = 1 + 0.3 * r.standard_normal(13), r.standard_normal(13)
    (y, mean, rstd), _ = ref.layer_norm(x, widths, w, b, 1e-5)
    (dx, dw, db), _ = ref.layer_norm_gradients(dy, x, mean, rstd, widths, w)
    h = 1e-6  # central quotient: h^2 and 1e-16 / h

    def loss(x, w, b):
        return (ref.layer_norm(x, widths, w, b, 1e-5)[0][0] * dy).sum()

    for grad, k in ((dx, 0), (dw, 1), (db, 2)):
        for at in np.ndindex(grad.shape):
            args = [[x.copy(), w.copy(), b.copy()] for _ in range(2)]
            args[0][k][at] += h
            args[1][k][at] -= h
            assert abs((loss(*args[0]) - loss(*args[1])) / (2 * h) - grad[at]) <= 1e-7 * (1 + np.abs(dx).max() + np.abs(grad).max())


@pytest.mark.parametrize("signed", [True, False])
def test_reference_codes(signed):
    levels = ref.q8_levels(7 if signed else 8)
    assert (np.diff(levels) > 0).all() and levels[0] == 0 and levels[-1] == 1
    assert np.array_equal(levels.astype(np.float16).astype(np.float64), levels)  # exact in fp16
    x = np.concatenate([levels, -levels[1:] if signed else levels[1:]]) * 3.5
    codes, scale, _ = ref.q8_encode(x, signed, block=x.size)
    assert scale.tolist() == [3.5]
    assert np.array_equal(ref.q8_decode(codes, scale, signed, block=x.size), x)


def test_reference_adamw_agrees_with_torch():
    r = torch.Generator().manual_seed(3)
    p = torch.randn(50, generator=r, dtype=torch.float64)
    q = torch.nn.Parameter(p.clone())
    opt = torch.optim.AdamW([q], lr=0.01, betas=(0.5, 0.75), eps=1e-8, weight_decay=0.1)  # exact in fp32
    m = v = np.zeros(50)
    x = p.numpy()
    for t in range(1, 4):
        g = torch.randn(50, generator=r, dtype=torch.float64)
        q.grad = g.clone()
        opt.step()
        (x, m, v), _ = ref.adamw(x, g.numpy(), m, v, t, 0.01, 0.5, 0.75, 1e-8, 0.1)
        np.testing.assert_allclose(q.detach().numpy(), x, rtol=1e-12)
