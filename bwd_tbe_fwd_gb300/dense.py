"""ctypes binding of include/tbe_dense.h: layer norm over each table's columns of the pooled
output, the global norm of many gradients, and one AdamW step of many tensors.

As in ``tbe.py``, argument marshalling only: torch supplies device memory and the current stream,
every step runs in the CUDA library, and there is nothing to fall back on.  The three classes hold
what a program sets up once (descriptions, workspaces); a call checks its tensors and launches.  An
object is ready for any stream when its constructor returns.  Its workspace is used by its calls in
order: calls of one object must not overlap on different streams or host threads.
"""
from __future__ import annotations

import array
import ctypes
import math

import torch

from .tbe import _WDTYPE, TBE_OK, TBEError, _check, c_f32, c_i32, c_i64, load, vp

TBE_STATE_F32, TBE_STATE_Q8 = 0, 1
TBE_Q8_BLOCK = 256


class NormProblem(ctypes.Structure):
    _fields_ = [("rows", c_i64), ("segments", c_i32), ("widths", ctypes.POINTER(c_i32)), ("col_offsets", vp),
                ("x_stride", c_i64), ("y_stride", c_i64), ("dx_stride", c_i64), ("xdtype", ctypes.c_int),
                ("ydtype", ctypes.c_int), ("wdtype", ctypes.c_int), ("eps", c_f32)]


class DenseTensor(ctypes.Structure):
    _fields_ = [("param", vp), ("grad", vp), ("master", vp), ("exp_avg", vp), ("exp_avg_sq", vp),
                ("exp_avg_scale", vp), ("exp_avg_sq_scale", vp), ("numel", c_i64), ("lr_scale", c_f32),
                ("weight_decay", c_f32)]


class AdamWProblem(ctypes.Structure):
    _fields_ = [("count", c_i32), ("tensors", ctypes.POINTER(DenseTensor)), ("pdtype", ctypes.c_int),
                ("gdtype", ctypes.c_int), ("states", ctypes.c_int), ("beta1", ctypes.c_double),
                ("beta2", ctypes.c_double), ("eps", c_f32)]


def _bind(lib):
    """Argument types of the tbe_dense.h entry points (once per loaded library)."""
    if getattr(lib, "_dense_bound", False):
        return lib
    N, A, size = ctypes.POINTER(NormProblem), ctypes.POINTER(AdamWProblem), ctypes.c_size_t
    lib.tbe_layer_norm_forward.argtypes = [N, vp, vp, vp, vp, vp, vp, vp]
    lib.tbe_layer_norm_backward_workspace_size.argtypes = [N]
    lib.tbe_layer_norm_backward.argtypes = [N, vp, vp, vp, vp, vp, vp, vp, vp, vp, size, vp]
    lib.tbe_grad_norm_workspace_size.argtypes = []
    lib.tbe_grad_norm.argtypes = [c_i32, vp, vp, ctypes.c_int, c_f32, vp, vp, size, vp]
    lib.tbe_adamw_workspace_size.argtypes = []
    lib.tbe_adamw_update.argtypes = [A, c_f32, vp, vp, vp, size, vp]
    lib.tbe_adamw_state_values.argtypes = [A, vp, vp, vp]
    for name in ("tbe_layer_norm_backward_workspace_size", "tbe_grad_norm_workspace_size", "tbe_adamw_workspace_size"):
        getattr(lib, name).restype = size
    for name in ("tbe_layer_norm_forward", "tbe_layer_norm_backward", "tbe_grad_norm", "tbe_adamw_update",
                 "tbe_adamw_state_values"):
        getattr(lib, name).restype = ctypes.c_int
    lib._dense_bound = True
    return lib


def _device(device) -> torch.device:
    dev = torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    return dev


# The current stream's handle without making a Stream object (which costs 2 to 4 us of a small call's 10).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, device):
    """The cudaStream_t of `stream`, or of the device's current one when None."""
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None and device.type == "cuda":
        return _current_raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


class _Handle:
    """What the three classes share: the device, memory of their own, and the launch of an entry point."""

    def _on(self, device):
        self.device = device
        self._index = -1 if device.index is None else device.index  # as Tensor.get_device

    def _own(self, *tensors):
        """Memory that the object's kernels use: complete when the constructor returns, and kept from reuse
        while a call on another stream than the constructor's may be at work on it."""
        self._kept = tensors
        self._home = _raw_stream(None, self.device)
        if self._index >= 0:
            torch.cuda.current_stream(self.device).synchronize()

    def _launch(self, fn, args, stream, what):
        """Calls the library with the device current, on `stream` (default: the device's current one)."""
        s = _raw_stream(stream, self.device)
        if s != self._home and self._index >= 0:
            for t in self._kept:
                t.record_stream(stream or torch.cuda.current_stream(self.device))
        if self._index >= 0 and torch.cuda.current_device() == self._index:
            status = fn(*args, s)
        else:
            with torch.cuda.device(self.device):
                status = fn(*args, s)
        if status != TBE_OK:
            _check(load(), status, what)


def _empty(shape, dtype, device, stream):
    """A result's memory, belonging to the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _flat(t, name, dtype, numel, device):
    """Address of a contiguous tensor of that type and size on that device."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.get_device() != (-1 if device.index is None else device.index) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous on {device}")
    if t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements")
    return t.data_ptr()


class LayerNorm(_Handle):
    """Layer norm of [rows, sum(widths)] matrices, each segment of ``widths[s]`` columns on its own: one
    segment is the ordinary layer norm; ``LayerNorm(tbe.D, ...)`` normalises every table's part of
    TableBatchedEmbedding.forward's output, and its dx is backward_update's grad_out.

    x and dx have ``x_dtype``, y and dy ``y_dtype`` (default the same; the two are equal or one of them
    is float32), weight, bias and their gradients ``weight_dtype``; mean and rstd are float32
    [rows, len(widths)].  Rows may be strided (views of a wider matrix); columns are contiguous."""

    def __init__(self, widths, x_dtype=torch.float32, y_dtype=None, weight_dtype=torch.float32, eps: float = 1e-5,
                 device="cuda"):
        self.lib = _bind(load())
        self._on(_device(device))
        self.widths = [int(w) for w in ([widths] if isinstance(widths, int) else widths)]
        self.cols = sum(self.widths)
        self.x_dtype, self.y_dtype, self.weight_dtype = x_dtype, y_dtype or x_dtype, weight_dtype
        self._widths = (c_i32 * len(self.widths))(*self.widths)
        offsets = [0]
        for w in self.widths:
            offsets.append(offsets[-1] + w)
        self.col_offsets = torch.tensor(offsets, dtype=torch.int32, device=self.device)
        self.prob = NormProblem(((1 << 39) - 1) // max(1, self.cols), len(self.widths), self._widths, self.col_offsets.data_ptr(), self.cols, self.cols,
                                self.cols, _WDTYPE[self.x_dtype], _WDTYPE[self.y_dtype], _WDTYPE[weight_dtype], eps)
        self._prob = ctypes.byref(self.prob)
        with torch.cuda.device(self.device):  # the most that any number of rows takes
            n = self.lib.tbe_layer_norm_backward_workspace_size(self._prob)
        if n == 0:
            raise TBEError("tbe_layer_norm_backward_workspace_size rejected the problem")
        self.ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        self._ws, self._ws_bytes = self.ws.data_ptr(), n
        self._own(self.col_offsets, self.ws)

    def _rows(self, t, name, dtype, rows=None):
        """Row stride of a [rows, cols] matrix."""
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}")
        shape = t.shape
        if len(shape) != 2 or shape[1] != self.cols or (rows is not None and shape[0] != rows):
            raise ValueError(f"{name} must be [{'rows' if rows is None else rows}, {self.cols}]")
        stride = t.stride()
        if t.get_device() != self._index or (self.cols > 1 and stride[1] != 1):
            raise ValueError(f"{name} must be on {self.device} with contiguous columns")
        if shape[0] <= 1:
            return self.cols
        if stride[0] < self.cols:
            raise ValueError(f"the rows of {name} overlap")
        return stride[0]

    def _param(self, t, name):
        return None if t is None else _flat(t, name, self.weight_dtype, self.cols, self.device)

    def _stat(self, t, name, rows):
        return _flat(t, name, torch.float32, rows * len(self.widths), self.device)

    def forward(self, x, weight=None, bias=None, y=None, mean=None, rstd=None, stream=None):
        """Returns (y, mean, rstd); y may be x itself where the types agree."""
        p = self.prob
        p.x_stride = self._rows(x, "x", self.x_dtype)
        p.rows = rows = x.shape[0]
        if y is None:
            y = _empty((rows, self.cols), self.y_dtype, self.device, stream)
            p.y_stride = self.cols
        else:
            p.y_stride = self._rows(y, "y", self.y_dtype, rows)
        if (mean is None) != (rstd is None):
            raise ValueError("mean and rstd are given together")
        if mean is None:
            mean = _empty((rows, len(self.widths)), torch.float32, self.device, stream)
            rstd = _empty((rows, len(self.widths)), torch.float32, self.device, stream)
            stats = mean.data_ptr(), rstd.data_ptr()
        else:
            stats = self._stat(mean, "mean", rows), self._stat(rstd, "rstd", rows)
        self._launch(self.lib.tbe_layer_norm_forward,
                (self._prob, x.data_ptr(), self._param(weight, "weight"), self._param(bias, "bias"), y.data_ptr(), *stats),
                stream, "tbe_layer_norm_forward")
        return y, mean, rstd

    def backward(self, dy, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, stream=None):
        """Returns (dx, dweight, dbias); dx may be x or dy itself where the types agree."""
        p = self.prob
        p.x_stride = self._rows(x, "x", self.x_dtype)
        p.rows = rows = x.shape[0]
        p.y_stride = self._rows(dy, "dy", self.y_dtype, rows)
        if dx is None:
            dx = _empty((rows, self.cols), self.x_dtype, self.device, stream)
            p.dx_stride = self.cols
        else:
            p.dx_stride = self._rows(dx, "dx", self.x_dtype, rows)
        if dweight is None:
            dweight = _empty(self.cols, self.weight_dtype, self.device, stream)
        if dbias is None:
            dbias = _empty(self.cols, self.weight_dtype, self.device, stream)
        self._launch(self.lib.tbe_layer_norm_backward,
                (self._prob, dy.data_ptr(), x.data_ptr(), self._stat(mean, "mean", rows), self._stat(rstd, "rstd", rows),
                 self._param(weight, "weight"), dx.data_ptr(), self._param(dweight, "dweight"),
                 self._param(dbias, "dbias"), self._ws, self._ws_bytes), stream, "tbe_layer_norm_backward")
        return dx, dweight, dbias


def _tensor_list(tensors, name, device=None):
    tensors = list(tensors)
    for t in tensors:
        device = device or t.device
        if t.dtype != tensors[0].dtype:
            raise TypeError(f"all {name} must be of one dtype")
        if t.dtype not in _WDTYPE:
            raise TypeError(f"{name} must be float32, float16 or bfloat16")
        if t.device != device or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous on {device}")
    return tensors


def _pointers(tensors):
    return (vp * max(1, len(tensors)))(*[t.data_ptr() for t in tensors])


class GradNorm(_Handle):
    """The norm of many gradients together and the coefficient that clips it, left on the device.  The
    gradients are those tensors' memory: refill it in place, or make a new object."""

    def __init__(self, grads, device="cuda"):
        self.lib = _bind(load())
        self.grads = _tensor_list(grads, "gradients")
        self._on(self.grads[0].device if self.grads else _device(device))
        self._dtype = _WDTYPE[self.grads[0].dtype] if self.grads else _WDTYPE[torch.float32]
        self._ptrs = _pointers(self.grads)
        self._numels = (c_i64 * max(1, len(self.grads)))(*[t.numel() for t in self.grads])
        self.ws = torch.zeros(self.lib.tbe_grad_norm_workspace_size(), dtype=torch.uint8, device=self.device)
        self._ws, self._ws_bytes = self.ws.data_ptr(), self.ws.numel()
        self._own(self.ws)

    def compute(self, max_norm: float = math.inf, out=None, stream=None):
        """Returns out: float32 [2], the norm and min(1, max_norm / (norm + 1e-6))."""
        if out is None:
            out = _empty(2, torch.float32, self.device, stream)
            address = out.data_ptr()
        else:
            address = _flat(out, "out", torch.float32, 2, self.device)
        self._launch(self.lib.tbe_grad_norm,
                     (len(self.grads), self._ptrs, self._numels, self._dtype, max_norm, address, self._ws, self._ws_bytes),
                     stream, "tbe_grad_norm")
        return out


class DenseAdamW(_Handle):
    """AdamW over many tensors at once.  ``params`` and ``grads`` are updated from and in their own memory
    (refill gradients in place, or call bind_grads).  ``states``: "f32", or "q8" for 8-bit states with
    a float32 scale for each 256 elements.  ``master``: None, or float32 tensors that hold 16-bit
    parameters at full precision.  ``weight_decay`` and ``lr_scale``: one number or one for each
    tensor.  ``state``: tensors to go on from (exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale:
    lists; step: int64 [1]); what it lacks starts at zero.  They are attributes of the object."""

    def __init__(self, params, grads, states: str = "f32", master=None, state=None, weight_decay=0.01, lr_scale=1.0,
                 betas=(0.9, 0.999), eps: float = 1e-8, device="cuda"):
        self.lib = _bind(load())
        self.params = _tensor_list(params, "params")
        n = len(self.params)
        self._on(self.params[0].device if n else _device(device))
        q8 = {"f32": False, "q8": True}[states]
        self.states = states
        self._numels = numels = [p.numel() for p in self.params]
        self.master = None if master is None else list(master)
        if self.master is not None and n and self.params[0].dtype == torch.float32:
            raise TypeError("float32 params take no master")
        state = dict(state or {})
        made = []

        def held(key, dtype, sizes):
            got = state.pop(key, None)
            if got is None:
                got = [torch.zeros(k, dtype=dtype, device=self.device) for k in sizes]
                made.extend(got)
            got = list(got)
            self._same_count(got, key)
            for t, k in zip(got, sizes):
                _flat(t, key, dtype, k, self.device)
            return got

        self.exp_avg = held("exp_avg", torch.uint8 if q8 else torch.float32, numels)
        self.exp_avg_sq = held("exp_avg_sq", torch.uint8 if q8 else torch.float32, numels)
        blocks = [-(-k // TBE_Q8_BLOCK) for k in numels]
        self.exp_avg_scale = held("exp_avg_scale", torch.float32, blocks) if q8 else None
        self.exp_avg_sq_scale = held("exp_avg_sq_scale", torch.float32, blocks) if q8 else None
        self.steps = state.pop("step", None)
        if self.steps is None:
            self.steps = torch.zeros(1, dtype=torch.int64, device=self.device)
            made.append(self.steps)
        _flat(self.steps, "step", torch.int64, 1, self.device)
        if state:
            raise TypeError(f"unknown state {sorted(state)}")
        if self.master is not None:
            self._same_count(self.master, "master")
            for t, k in zip(self.master, numels):
                _flat(t, "master", torch.float32, k, self.device)
        self.weight_decay = self._each(weight_decay, "weight_decay")
        self.lr_scale = self._each(lr_scale, "lr_scale")
        self._tensors = (DenseTensor * max(1, n))()
        for i, p in enumerate(self.params):
            d = self._tensors[i]
            d.param, d.numel = p.data_ptr(), numels[i]
            d.exp_avg, d.exp_avg_sq = self.exp_avg[i].data_ptr(), self.exp_avg_sq[i].data_ptr()
            d.master = self.master[i].data_ptr() if self.master is not None else None
            if q8:
                d.exp_avg_scale, d.exp_avg_sq_scale = (self.exp_avg_scale[i].data_ptr(),
                                                       self.exp_avg_sq_scale[i].data_ptr())
            d.lr_scale, d.weight_decay = self.lr_scale[i], self.weight_decay[i]
        self.prob = AdamWProblem(n, self._tensors, _WDTYPE[self.params[0].dtype] if n else 0, 0,
                                 TBE_STATE_Q8 if q8 else TBE_STATE_F32, betas[0], betas[1], eps)
        self._prob = ctypes.byref(self.prob)
        self.bind_grads(grads)
        self.ws = torch.zeros(self.lib.tbe_adamw_workspace_size(), dtype=torch.uint8, device=self.device)
        self._own(self.ws, *made)

    def _same_count(self, tensors, name):
        if len(tensors) != len(self.params):
            raise ValueError(f"{name}: {len(tensors)} tensors for {len(self.params)} params")

    def _each(self, v, name):
        v = [float(x) for x in v] if isinstance(v, (list, tuple)) else [float(v)] * len(self.params)
        self._same_count(v, name)
        return v

    def bind_grads(self, grads):
        """The gradients' memory from now on: one tensor for each of params, of one dtype."""
        grads = _tensor_list(grads, "grads", self.device)
        self._same_count(grads, "grads")
        for g, p in zip(grads, self.params):
            if g.numel() != p.numel():
                raise ValueError("grads and params differ in size")
        self.grads = grads
        for i, g in enumerate(grads):
            self._tensors[i].grad = g.data_ptr()
        self.prob.gdtype = _WDTYPE[grads[0].dtype] if grads else 0

    def step(self, lr: float, clip=None, stream=None):
        """One update.  clip: the result of GradNorm.compute (where its norm is not finite nothing changes)."""
        self._launch(self.lib.tbe_adamw_update,
                (self._prob, lr, None if clip is None else _flat(clip, "clip", torch.float32, 2, self.device),
                 self.steps.data_ptr(), self.ws.data_ptr(), self.ws.numel()), stream, "tbe_adamw_update")

    def state_values(self, exp_avg=None, exp_avg_sq=None, stream=None):
        """What the 8-bit states stand for: two lists of float32 tensors (given ones are written)."""
        lists = []
        T = torch.Tensor
        for given, name in ((exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq")):
            if given is None:
                given = [_empty(n, torch.float32, self.device, stream) for n in self._numels]
            self._same_count(given, name)
            # all at once, and one by one only to say what is wrong
            if given and not ([*map(T.numel, given)] == self._numels and all(map(T.is_contiguous, given))
                              and {*map(T.get_device, given)} == {self._index}
                              and {t.dtype for t in given} == {torch.float32}):
                for t, n in zip(given, self._numels):
                    _flat(t, name, torch.float32, n, self.device)
            lists.append((given, array.array("Q", map(T.data_ptr, given))))
        self._launch(self.lib.tbe_adamw_state_values,
                     (self._prob, lists[0][1].buffer_info()[0], lists[1][1].buffer_info()[0]), stream,
                     "tbe_adamw_state_values")
        return lists[0][0], lists[1][0]
