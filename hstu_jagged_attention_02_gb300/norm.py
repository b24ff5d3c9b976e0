"""Layer norm with weight and bias over rows of features, through hstu_ln_fwd /
_bwd of libhstu_attn.so: what a projection's input goes through.  Marshalling
and checks of arguments only."""
from __future__ import annotations

from typing import Optional

import numpy as np
import torch

from . import binding as C
from .attention import _ptr
from .qk import Launch, _need, _same_device, device_error

_DTYPES = {torch.bfloat16: C.HSTU_BF16, torch.float32: C.HSTU_FP32}


def _as_rows(t, name):
    """[rows, D] with contiguous features and rows that are not in each other's
    way; any other layout is copied."""
    _need(t.dim() == 2, f"{name} must be [rows, D], got {tuple(t.shape)}")
    if t.numel() and ((t.shape[1] > 1 and t.stride(1) != 1) or t.stride(0) < 0):
        return t.contiguous()
    return t


def _own_rows(t, name):
    """Of an output: contiguous features, a place of its own for each."""
    _need(t.dim() == 2, f"{name} must be [rows, D], got {tuple(t.shape)}")
    _need(t.numel() == 0 or ((t.shape[1] == 1 or t.stride(1) == 1) and (t.shape[0] == 1 or t.stride(0) >= t.shape[1])),
          f"{name} needs contiguous features and rows that do not overlap")


def _runs(t):
    """(first byte, bytes of a run, bytes from run to run, runs) of the memory
    behind a vector, or a matrix whose features are contiguous."""
    size, at = t.element_size(), t.data_ptr()
    if t.is_contiguous() or t.dim() != 2:
        return at, t.numel() * size, 0, 1
    rows, width = t.shape
    run, pitch = ((width - 1) * t.stride(1) + 1) * size, t.stride(0) * size
    return (at, run, pitch, rows) if pitch > run else (at, (rows - 1) * pitch + run, 0, 1)


def _touch(a, b):
    """Whether two tensors (vectors, rows of features, or dense) share a byte.
    Cuts of the columns of one buffer lie apart."""
    if a is None or b is None or a.numel() == 0 or b.numel() == 0:
        return False
    a, b = sorted((_runs(a), _runs(b)), key=lambda r: -r[3])
    hull = lambda r: r[0] + r[2] * (r[3] - 1) + r[1]  # noqa: E731
    if hull(a) <= b[0] or hull(b) <= a[0]:
        return False
    if a[3] == 1:
        return True
    # the runs of a that begin last at or before a run of b, and the next ones
    starts = b[0] + b[2] * np.arange(b[3], dtype=np.int64)
    i = (starts - a[0]) // a[2]
    for k in (i, i + 1):
        at = a[0] + a[2] * np.clip(k, 0, a[3] - 1)
        if np.any((at < starts + b[1]) & (starts < at + a[1])):
            return True
    return False


def _same_rows(a, b):
    """Whether two matrices are the same rows, of the same type."""
    return (a is not None and b is not None and a.data_ptr() == b.data_ptr() and a.dtype == b.dtype and a.shape == b.shape and
            (a.shape[0] == 1 or a.stride(0) == b.stride(0)))


def _apart(name, out, may_be=(), **others):
    """An output shares no memory with the others, but for those that it may be."""
    for other, t in others.items():
        _need(not _touch(out, t) or (other in may_be and _same_rows(out, t)),
              f"{name} shares memory with {other}" + (", and is not the same rows" if other in may_be else ""))


def _step(t):
    return 0 if t is None or t.numel() == 0 else t.stride(0)


class LNProblem:
    """x [rows, D] (BF16 or FP32), weight and bias [D] FP32 (either may be
    None), the outputs and the workspace, with the C argument structs filled
    once; forward() fills y, mean, rstd; backward() fills dx, d_weight, d_bias
    from dy (and adds dres, the gradient that reached x past the norm).

    x, dy, dres are used in place where their features are contiguous, else
    copied once, here.  The outputs are allocated unless given; y may be x
    (without a backward), dx may be x, dy or dres, of the same type and strides;
    they share no memory otherwise with what their call reads.  mean and rstd
    may be those of an earlier forward; with them want_y=False makes a problem of
    the backward alone."""

    def __init__(self, x, weight=None, bias=None, *, eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None,
                 dy=None, dres=None, y=None, dx=None, mean=None, rstd=None, num_rows=None, want_weight_grad=None,
                 want_bias_grad=None, want_y: bool = True, workspace=None):
        _need(x.dim() == 2, f"x must be [rows, D], got {tuple(x.shape)}")
        _need(x.dtype in _DTYPES, f"x must be BF16 or FP32, got {x.dtype}")
        dev = x.device
        self.device = dev
        _same_device(dev, weight=weight, bias=bias, dy=dy, dres=dres, y=y, dx=dx, mean=mean, rstd=rstd, num_rows=num_rows,
                     workspace=workspace)
        rows, D = x.shape
        if out_dtype is None:
            out_dtype = y.dtype if y is not None else (dy.dtype if dy is not None else x.dtype)
        _need(out_dtype in _DTYPES, f"the output must be BF16 or FP32, got {out_dtype}")
        for name, t in (("weight", weight), ("bias", bias)):
            _need(t is None or (t.shape == (D,) and t.dtype == torch.float32 and t.is_contiguous()), f"{name} must be FP32 [D]")
        for name, t, dt in (("y", y, out_dtype), ("dy", dy, None), ("dres", dres, x.dtype), ("dx", dx, x.dtype)):
            _need(t is None or (t.shape == x.shape and t.dtype in _DTYPES and (dt is None or t.dtype == dt)),
                  f"{name} does not match x in shape or type")
        for name, t in (("mean", mean), ("rstd", rstd)):
            _need(t is None or (t.shape == (rows,) and t.dtype == torch.float32 and t.is_contiguous()),
                  f"{name} must be FP32 [rows]")
        _need((mean is None) == (rstd is None), "mean and rstd go together")
        _need(num_rows is None or (num_rows.dtype == torch.int64 and num_rows.numel() == 1),
              "num_rows must be one int64 on the device")
        _need(dres is None or dy is not None, "dres is of the backward, which needs dy")
        self.x, self.weight, self.bias, self.num_rows = _as_rows(x, "x"), weight, bias, num_rows
        f32 = dict(device=dev, dtype=torch.float32)
        _need(want_y or (y is None and dy is not None and mean is not None),
              "a problem without y is one of the backward alone, which needs the forward's mean and rstd")
        self.y = y if y is not None or not want_y else torch.empty(rows, D, device=dev, dtype=out_dtype)
        if want_y:
            _own_rows(self.y, "y")
        _need(dy is None or y is None or y.numel() == 0 or y.data_ptr() != self.x.data_ptr(),
              "the backward needs x, which a forward in place overwrites")
        if y is not None:
            _apart("y", y, ("x",), x=self.x, weight=weight, bias=bias, num_rows=num_rows, mean=mean, rstd=rstd)
        if mean is not None and dy is None:   # (with dy they are those of an earlier forward: read)
            for name, t in (("mean", mean), ("rstd", rstd)):
                _apart(name, t, x=self.x, weight=weight, bias=bias, num_rows=num_rows)
            _apart("mean", mean, rstd=rstd)
        self.dy, self.dres = (None if t is None else _as_rows(t, name) for name, t in (("dy", dy), ("dres", dres)))
        if dx is not None:
            _own_rows(dx, "dx")
            _apart("dx", dx, ("x", "dy", "dres"), x=self.x, dy=self.dy, dres=self.dres, weight=weight, num_rows=num_rows,
                   mean=mean, rstd=rstd)
        self.mean = mean if mean is not None else torch.empty(rows, **f32)
        self.rstd = rstd if rstd is not None else torch.empty(rows, **f32)
        backward = dy is not None
        self.dx = self.d_weight = self.d_bias = None
        d = C.hstu_ln_desc()
        d.struct_size = C.ctypes.sizeof(d)
        d.x_dtype, d.y_dtype, d.D, d.eps, d.rows = _DTYPES[x.dtype], _DTYPES[out_dtype], D, eps, rows
        d.x_stride, d.y_stride = _step(self.x), _step(self.y)
        self.desc = d
        fwd_b, bwd_b = C.hstu_ln_workspace_size(d)
        need = max(fwd_b, bwd_b if backward else 0)
        if workspace is None:
            workspace = torch.empty(need, device=dev, dtype=torch.uint8)
            workspace[:fwd_b].zero_()   # the header
        _need(workspace.dtype == torch.uint8 and workspace.is_contiguous(), "workspace must be contiguous uint8")
        self.ws, self.ws_bytes = workspace, workspace.numel()
        lib, w = C.load(), (self.ws.data_ptr(), self.ws_bytes)
        self.fwd_args = C.hstu_ln_fwd_args(_ptr(num_rows), _ptr(self.x), _ptr(weight), _ptr(bias), _ptr(self.y),
                                           _ptr(self.mean), _ptr(self.rstd))
        self._forward = Launch(dev, lib.hstu_ln_fwd, "hstu_ln_fwd", self.desc, self.fwd_args, *w)
        if backward:
            self.dx = dx if dx is not None else torch.empty(rows, D, device=dev, dtype=x.dtype)
            if want_weight_grad if want_weight_grad is not None else weight is not None:
                self.d_weight = torch.empty(D, **f32)
            if want_bias_grad if want_bias_grad is not None else bias is not None:
                self.d_bias = torch.empty(D, **f32)
            b = C.hstu_ln_desc.from_buffer_copy(d)
            b.y_dtype, b.y_stride = _DTYPES[self.dy.dtype], _step(self.dy)
            b.dx_stride, b.dres_stride = _step(self.dx), _step(self.dres)
            self.bwd_desc = b
            self.bwd_args = C.hstu_ln_bwd_args(_ptr(num_rows), _ptr(self.x), _ptr(weight), _ptr(self.mean), _ptr(self.rstd),
                                               _ptr(self.dy), _ptr(self.dres), _ptr(self.dx), _ptr(self.d_weight),
                                               _ptr(self.d_bias))
            self._backward = Launch(dev, lib.hstu_ln_bwd, "hstu_ln_bwd", self.bwd_desc, self.bwd_args, *w)

    def forward(self, stream=None):
        _need(self.y is not None, "a problem without y has no forward")
        self._forward(stream)

    def backward(self, stream=None):
        self._backward(stream)

    def device_error(self, stream=None) -> int:
        return device_error(self.device, self.ws, stream)


class LNFunction(torch.autograd.Function):
    """y of x, weight, bias; gradients for the three."""

    @staticmethod
    def forward(ctx, x, weight, bias, num_rows, eps, out_dtype, workspace):
        det = lambda t: None if t is None else t.detach()  # noqa: E731
        pr = LNProblem(det(x), det(weight), det(bias), eps=eps, out_dtype=out_dtype, num_rows=num_rows, workspace=workspace)
        if num_rows is not None:   # rows behind the batch are written by nobody
            pr.y.zero_()
        pr.forward()
        ctx.save_for_backward(x, weight, bias, num_rows, pr.mean, pr.rstd)
        ctx.eps = eps
        return pr.y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, bias, num_rows, mean, rstd = ctx.saved_tensors
        pr = LNProblem(x, weight, bias, eps=ctx.eps, dy=dy, mean=mean, rstd=rstd, num_rows=num_rows, want_y=False)
        if num_rows is not None:
            pr.dx.zero_()
        pr.backward()
        return (pr.dx, pr.d_weight, pr.d_bias) + (None,) * 4


def hstu_ln(x, weight=None, bias=None, *, eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None, num_rows=None,
            workspace=None):
    """Differentiable layer norm of the rows of x [rows, D] (BF16 or FP32), in
    out_dtype (default: x's): the input of a projection, or of
    hstu_group_linear.  num_rows: one int64 on the device, rows in use of a
    padded batch (rows behind it come back as zeros).  A count outside
    [0, rows] raises nothing here: the device records it in the forward's
    workspace.  Give one to look (256 zeroed bytes, uint8, 256-byte aligned;
    qk.device_error(device, workspace) != 0), or use LNProblem, which keeps its
    own.  There is no second derivative.  Into a CUDA graph goes LNProblem's
    forward and backward, rather than autograd's."""
    return LNFunction.apply(x, weight, bias, num_rows, float(eps), out_dtype, workspace)
