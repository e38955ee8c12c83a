"""ctypes binding of include/tbe_tokens.h: the lookup of a table's rows by token with its gradient, and the softmax
cross entropy over a table's rows with its gradient.

As in ``dense.py``, argument marshalling only: the two classes hold what a program sets up once (descriptions,
workspaces), a call checks its tensors and launches.  An object is ready for any stream when its constructor
returns.  Its workspace is used by its calls in order: calls of one object must not overlap on different streams or
host threads, and neither must two captured graphs that hold its calls.
"""
from __future__ import annotations

import ctypes

import torch

from .dense import _device, _empty, _flat, _Handle
from .tbe import _WDTYPE, TBE_I32, TBE_I64, TBE_NUM_STATS, TBEError, c_f32, c_i32, c_i64, load, vp

_ITYPE = {torch.int32: TBE_I32, torch.int64: TBE_I64}


class LookupProblem(ctypes.Structure):
    _fields_ = [("tokens", c_i64), ("rows", c_i64), ("dim", c_i32), ("table_stride", c_i64), ("out_stride", c_i64),
                ("tdtype", ctypes.c_int), ("odtype", ctypes.c_int), ("itype", ctypes.c_int), ("scale", c_f32)]


class SoftmaxProblem(ctypes.Structure):
    _fields_ = [("tokens", c_i64), ("rows", c_i64), ("dim", c_i32), ("hidden_stride", c_i64), ("weight_stride", c_i64),
                ("dhidden_stride", c_i64), ("dweight_stride", c_i64), ("dtype", ctypes.c_int), ("itype", ctypes.c_int),
                ("scale", c_f32)]


def _bind(lib):
    """Argument types of the tbe_tokens.h entry points (once per loaded library)."""
    if getattr(lib, "_tokens_bound", False):
        return lib
    L, S, size = ctypes.POINTER(LookupProblem), ctypes.POINTER(SoftmaxProblem), ctypes.c_size_t
    lib.tbe_lookup_forward.argtypes = [L, vp, vp, vp, vp, vp]
    lib.tbe_lookup_backward_workspace_size.argtypes = [L]
    lib.tbe_lookup_backward.argtypes = [L, vp, vp, vp, c_i32, vp, size, vp, vp]
    lib.tbe_softmax_loss_workspace_size.argtypes = [S]
    lib.tbe_softmax_loss_forward.argtypes = [S, vp, vp, vp, vp, vp, vp, vp, size, vp, vp]
    lib.tbe_softmax_loss_backward_workspace_size.argtypes = [S]
    lib.tbe_softmax_loss_backward.argtypes = [S, vp, vp, vp, vp, vp, vp, vp, vp, vp, size, vp, vp]
    for name in ("tbe_lookup_backward_workspace_size", "tbe_softmax_loss_workspace_size",
                 "tbe_softmax_loss_backward_workspace_size"):
        getattr(lib, name).restype = size
    for name in ("tbe_lookup_forward", "tbe_lookup_backward", "tbe_softmax_loss_forward", "tbe_softmax_loss_backward"):
        getattr(lib, name).restype = ctypes.c_int
    lib._tokens_bound = True
    return lib


def _matrix(t, name, dtype, rows, cols, handle):
    """Row stride of a [rows, cols] matrix with contiguous columns and rows that do not overlap."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols:
        raise ValueError(f"{name} must be [{rows}, {cols}]")
    stride = t.stride()
    if t.get_device() != handle._index or (cols > 1 and stride[1] != 1):
        raise ValueError(f"{name} must be on {handle.device} with contiguous columns")
    if rows <= 1:
        return cols
    if stride[0] < cols:
        raise ValueError(f"the rows of {name} overlap")
    return stride[0]


class _Tokens(_Handle):
    """What the two classes share: the table's size, the workspace for as many tokens as a call may have, and the counters
    (``stats``, int64 [TBE_NUM_STATS]: ids past the table, and waits that gave up)."""

    def _setup(self, rows, dim, tokens, index_dtype, device):
        self.lib = _bind(load())
        self._on(_device(device))
        if index_dtype not in _ITYPE:
            raise TypeError("index_dtype must be int32 or int64")
        self.rows, self.dim, self.tokens, self.index_dtype = int(rows), int(dim), int(tokens), index_dtype

    def _workspace(self, *queries):
        """Room for the largest call: `queries` are (entry point, problem) pairs of which each problem's size counts."""
        need = 0
        with torch.cuda.device(self.device):
            for fn, prob in queries:
                n = fn(ctypes.byref(prob))
                if n == 0:
                    raise TBEError(f"{fn.__name__} rejected the problem")
                need = max(need, n)
        self.ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        self._ws, self._ws_bytes = self.ws.data_ptr(), need
        self.stats = torch.zeros(TBE_NUM_STATS, dtype=torch.int64, device=self.device)
        self._stats = self.stats.data_ptr()
        self._own(self.ws, self.stats)

    def _count(self, ids, name):
        n = ids.numel()
        if n > self.tokens:
            raise ValueError(f"{name} has {n} elements, the object was made for {self.tokens}")
        _flat(ids, name, self.index_dtype, n, self.device)
        return n


class TokenEmbedding(_Tokens):
    """One table's rows by token: ``out[i] = scale * table[ids[i]]`` and the table's gradient
    ``grad[v] = scale * sum of dout[i] over ids[i] == v``.  Ids that are no row of the table (padding: any negative one) give
    rows of zeros and have no part in the gradient; those past the table are counted in ``stats``.

    table and grad are [rows, dim] of ``table_dtype``, out and dout [tokens, dim] of ``out_dtype`` (default the same; the
    two are equal or one of them is float32); ids hold at most ``tokens`` of ``index_dtype``.  Rows may be strided
    (views of a wider matrix); columns are contiguous."""

    def __init__(self, rows: int, dim: int, tokens: int, table_dtype=torch.float32, out_dtype=None, index_dtype=torch.int64,
                 scale: float = 1.0, device="cuda"):
        self._setup(rows, dim, tokens, index_dtype, device)
        self.table_dtype, self.out_dtype, self.scale = table_dtype, out_dtype or table_dtype, float(scale)
        self.prob = LookupProblem(self.tokens, self.rows, self.dim, self.dim, self.dim, _WDTYPE[self.table_dtype],
                                  _WDTYPE[self.out_dtype], _ITYPE[index_dtype], self.scale)
        self._prob = ctypes.byref(self.prob)
        self._workspace((self.lib.tbe_lookup_backward_workspace_size, self.prob))

    def forward(self, table, ids, out=None, stream=None):
        """Returns out, [*ids.shape, dim] (a given one: [ids.numel(), dim])."""
        p = self.prob
        p.tokens = n = self._count(ids, "ids")
        p.table_stride = _matrix(table, "table", self.table_dtype, self.rows, self.dim, self)
        if out is None:
            out = _empty((*ids.shape, self.dim), self.out_dtype, self.device, stream)
            p.out_stride = self.dim
        else:
            p.out_stride = _matrix(out, "out", self.out_dtype, n, self.dim, self)
        self._launch(self.lib.tbe_lookup_forward, (self._prob, table.data_ptr(), ids.data_ptr(), out.data_ptr(), self._stats),
                     stream, "tbe_lookup_forward")
        return out

    def backward(self, dout, ids, grad=None, accumulate: bool = False, stream=None):
        """Returns grad, [rows, dim]; with ``accumulate`` a given one is added to (as the loss's gradient of a shared
        table), else overwritten.  dout: [*ids.shape, dim] or [ids.numel(), dim]."""
        p = self.prob
        p.tokens = n = self._count(ids, "ids")
        if dout.dim() != 2:
            if dout.shape != (*ids.shape, self.dim) or not dout.is_contiguous():
                raise ValueError(f"dout must be [*ids.shape, {self.dim}] and contiguous, or [{n}, {self.dim}]")
            dout = dout.view(n, self.dim)
        p.out_stride = _matrix(dout, "dout", self.out_dtype, n, self.dim, self)
        if grad is None:
            if accumulate:
                raise ValueError("accumulate needs a grad to add to")
            grad = _empty((self.rows, self.dim), self.table_dtype, self.device, stream)
            p.table_stride = self.dim
        else:
            p.table_stride = _matrix(grad, "grad", self.table_dtype, self.rows, self.dim, self)
        self._launch(self.lib.tbe_lookup_backward,
                     (self._prob, dout.data_ptr(), ids.data_ptr(), grad.data_ptr(), int(accumulate), self._ws, self._ws_bytes,
                      self._stats), stream, "tbe_lookup_backward")
        return grad


class SoftmaxLoss(_Tokens):
    """Softmax cross entropy of each token over the rows of a table, ``z = scale * hidden @ weight.T``, without keeping the
    logits, and its gradient.  Targets that are no row of the table (padding: any negative one) have loss 0 and no part
    in the gradients, whatever their hidden row holds; those past the table are counted in ``stats``.

    hidden and dhidden are [tokens, dim], weight and dweight [rows, dim], all of ``dtype`` (float16 or bfloat16); targets hold
    at most ``tokens`` of ``index_dtype``.  Rows may be strided (those of weight by
    multiples of 8 where dim is one, from a multiple of 16 bytes on); columns are contiguous.  The workspace has room for both
    directions: up to 512 MB of the logits' gradient (or 512 bytes a token), 100 MB and copies of hidden."""

    def __init__(self, rows: int, dim: int, tokens: int, dtype=torch.bfloat16, index_dtype=torch.int64, scale: float = 1.0,
                 device="cuda"):
        self._setup(rows, dim, tokens, index_dtype, device)
        self.dtype, self.scale = dtype, float(scale)
        d = self.dim
        self.prob = SoftmaxProblem(self.tokens, self.rows, d, d, d, d, d, _WDTYPE[dtype], _ITYPE[index_dtype], self.scale)
        self._prob = ctypes.byref(self.prob)
        self._workspace((self.lib.tbe_softmax_loss_workspace_size, self.prob),
                        (self.lib.tbe_softmax_loss_backward_workspace_size, self.prob))

    def _weight(self, weight):
        stride = _matrix(weight, "weight", self.dtype, self.rows, self.dim, self)
        if stride % 8 and self.dim % 8 == 0:  # the workspace has no room for a copy that TMA can address
            raise ValueError("the rows of weight must be a multiple of 8 elements apart")
        if stride % 8 == 0 and weight.data_ptr() % 16:
            raise ValueError("weight must begin at a multiple of 16 bytes")
        return stride

    def forward(self, hidden, weight, targets, loss=None, lse=None, mean=None, stream=None):
        """Returns (loss, lse, mean): float32 [tokens] each, and [2]: the mean loss of the tokens that count, and one over
        their number."""
        p = self.prob
        p.tokens = n = self._count(targets, "targets")
        p.hidden_stride = _matrix(hidden, "hidden", self.dtype, n, self.dim, self)
        p.weight_stride = self._weight(weight)
        out = []
        for t, name, k in ((loss, "loss", n), (lse, "lse", n), (mean, "mean", 2)):
            if t is None:
                t = _empty(k, torch.float32, self.device, stream)
            else:
                _flat(t, name, torch.float32, k, self.device)
            out.append(t)
        self._launch(self.lib.tbe_softmax_loss_forward,
                     (self._prob, hidden.data_ptr(), weight.data_ptr(), targets.data_ptr(), *(t.data_ptr() for t in out),
                      self._ws, self._ws_bytes, self._stats), stream, "tbe_softmax_loss_forward")
        return tuple(out)

    def backward(self, hidden, weight, targets, lse, dloss=None, mean=None, dhidden=None, dweight=None, stream=None):
        """Returns (dhidden, dweight) of sum_i c[i] loss[i], c[i] = dloss[i] (float32 [tokens]; 1 when None) times mean[1]
        (1 when None): the forward's ``mean`` alone gives the gradient of the mean loss."""
        p = self.prob
        p.tokens = n = self._count(targets, "targets")
        p.hidden_stride = _matrix(hidden, "hidden", self.dtype, n, self.dim, self)
        p.weight_stride = self._weight(weight)
        _flat(lse, "lse", torch.float32, n, self.device)
        if dloss is not None:
            _flat(dloss, "dloss", torch.float32, n, self.device)
        if mean is not None:
            _flat(mean, "mean", torch.float32, 2, self.device)
        if dhidden is None:
            dhidden = _empty((n, self.dim), self.dtype, self.device, stream)
            p.dhidden_stride = self.dim
        else:
            p.dhidden_stride = _matrix(dhidden, "dhidden", self.dtype, n, self.dim, self)
        if dweight is None:
            dweight = _empty((self.rows, self.dim), self.dtype, self.device, stream)
            p.dweight_stride = self.dim
        else:
            p.dweight_stride = _matrix(dweight, "dweight", self.dtype, self.rows, self.dim, self)
        self._launch(self.lib.tbe_softmax_loss_backward,
                     (self._prob, hidden.data_ptr(), weight.data_ptr(), targets.data_ptr(), lse.data_ptr(),
                      None if dloss is None else dloss.data_ptr(), None if mean is None else mean.data_ptr(),
                      dhidden.data_ptr(), dweight.data_ptr(), self._ws, self._ws_bytes, self._stats), stream,
                     "tbe_softmax_loss_backward")
        return dhidden, dweight
