"""Products of ragged groups of rows with a weight matrix each (a projection
per kind of token, scenario or expert) and their gradients, through
hstu_group_fwd / _bwd of libhstu_attn.so.  Marshalling and checks of arguments
only."""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as C
from .attention import _ptr
from .norm import _DTYPES, _apart, _own_rows
from .qk import Launch, _need, _same_device, device_error


def group_rows(group_of_row, groups: int):
    """Order and offsets of rows by group: x[order] lies as GroupProblem takes
    it (rows of a group in their old order), offsets int64 [groups + 1];
    y_of_x = torch.empty_like(y).index_copy_(0, order, y) puts results back."""
    order = torch.sort(group_of_row, stable=True).indices
    counts = torch.bincount(group_of_row, minlength=groups)
    _need(counts.numel() == groups, f"a row's group is not below {groups}")
    offsets = torch.zeros(groups + 1, dtype=torch.int64, device=group_of_row.device)
    offsets[1:] = counts.cumsum(0)
    return order, offsets


def _rows16(t, name):
    """[rows, features] BF16 as tile loads take it: contiguous features, rows a
    multiple of 16 bytes apart; any other layout is copied."""
    if t.numel() and (t.stride(1) != 1 or t.data_ptr() % 16 or
                      (t.shape[0] > 1 and (t.stride(0) % 8 or t.stride(0) < t.shape[1]))):
        t = t.contiguous()
        if t.data_ptr() % 16:   # a cut of a larger buffer, contiguous already
            t = t.clone()
    return t


def _check_out(t, name):
    _own_rows(t, name)
    _need(t.numel() == 0 or (t.data_ptr() % 16 == 0 and (t.shape[0] == 1 or t.stride(0) % 8 == 0)),
          f"{name} needs 16-byte aligned rows, a multiple of 8 elements apart")


def _step(t, width):
    return width if t is None or t.numel() == 0 else t.stride(0)


class GroupProblem:
    """x [rows, K] BF16, w [groups, K, N] BF16, group_offsets int64
    [groups + 1] on the device (group g: rows [offsets[g], offsets[g + 1])), the
    outputs and the workspace, with the C argument structs filled once.
    forward() fills y [rows, N]; backward() fills dx [rows, K] and dw
    [groups, K, N] FP32 from dy [rows, N] BF16.

    x and dy are used in place where their features are contiguous and rows a
    multiple of 16 bytes apart, else copied once, here.  The outputs are
    allocated unless given (no y without want_y: the backward alone) and lie apart from the inputs (columns of one buffer
    do), dx and dw from each other.  Rows behind the last
    group are left as they are.  A workspace that is given (uint8, 256-byte
    aligned, as hstu_group_workspace_size says) has zeros in its first 256 bytes
    before its first use; it may serve problems of any shape, one call at a time."""

    def __init__(self, x, w, group_offsets, *, out_dtype: Optional[torch.dtype] = None, dy=None, y=None, dx=None, dw=None,
                 dx_dtype: Optional[torch.dtype] = None, want_y: bool = True, want_dx: bool = True, want_dw: bool = True,
                 workspace=None, flags: int = 0):
        _need(x.dim() == 2 and w.dim() == 3 and w.shape[1] == x.shape[1],
              f"x must be [rows, K] and w [groups, K, N], got {tuple(x.shape)} and {tuple(w.shape)}")
        _need(x.dtype == torch.bfloat16 and w.dtype == torch.bfloat16, f"x and w must be BF16, got {x.dtype} and {w.dtype}")
        _need(w.is_contiguous(), "w must be contiguous")
        dev = x.device
        self.device = dev
        _same_device(dev, w=w, group_offsets=group_offsets, dy=dy, y=y, dx=dx, dw=dw, workspace=workspace)
        (rows, K), (E, _, N) = x.shape, w.shape
        _need(group_offsets.dtype == torch.int64 and group_offsets.shape == (E + 1,) and group_offsets.is_contiguous(),
              "group_offsets must be int64 [groups + 1]")
        out_dtype = out_dtype if out_dtype is not None else (y.dtype if y is not None else torch.bfloat16)
        dx_dtype = dx_dtype if dx_dtype is not None else (dx.dtype if dx is not None else torch.bfloat16)
        _need(out_dtype in _DTYPES and dx_dtype in _DTYPES, "outputs are BF16 or FP32")
        for name, t, shape, dt in (("y", y, (rows, N), out_dtype), ("dy", dy, (rows, N), torch.bfloat16),
                                   ("dx", dx, (rows, K), dx_dtype), ("dw", dw, (E, K, N), torch.float32)):
            _need(t is None or (t.shape == shape and t.dtype == dt), f"{name} must be {dt} {shape}")
        _need(dw is None or dw.is_contiguous(), "dw must be contiguous")
        read = {t.data_ptr() for t in (x, w, dy) if t is not None and t.numel()}
        for name, t in (("y", y), ("dx", dx), ("dw", dw)):
            _need(t is None or t.numel() == 0 or t.data_ptr() not in read, f"{name} must lie apart from what is read")
        self.x, self.w, self.offsets = _rows16(x, "x"), w, group_offsets
        self.dy = None if dy is None else _rows16(dy, "dy")
        for name, t in (("y", y), ("dx", dx), ("dw", dw)):
            if t is not None:
                _apart(name, t, x=self.x, w=w, dy=self.dy, group_offsets=group_offsets)
        _apart("dx", dx, dw=dw)
        backward = dy is not None
        _need(want_y or (backward and y is None), "a problem without y is one of the backward alone")
        self.y = y if y is not None or not want_y else torch.empty(rows, N, device=dev, dtype=out_dtype)
        if want_y:
            _check_out(self.y, "y")
        self.dx = self.dw = None
        d = C.hstu_group_desc()
        d.struct_size = C.ctypes.sizeof(d)
        d.groups, d.K, d.N, d.rows, d.flags = E, K, N, rows, flags
        d.y_dtype, d.dx_dtype = _DTYPES[out_dtype], _DTYPES[dx_dtype]
        d.x_stride, d.y_stride = _step(self.x, K), _step(self.y, N)
        self.desc = d
        fwd_b, bwd_b, zero = C.hstu_group_workspace_size(d)
        need = max(fwd_b, bwd_b if backward else 0)
        if workspace is None:
            workspace = torch.empty(need, device=dev, dtype=torch.uint8)
            workspace[:zero].zero_()
        _need(workspace.dtype == torch.uint8 and workspace.is_contiguous(), "workspace must be contiguous uint8")
        self.ws, self.ws_bytes = workspace, workspace.numel()
        lib, at = C.load(), (self.ws.data_ptr(), self.ws_bytes)
        self.fwd_args = C.hstu_group_fwd_args(_ptr(group_offsets), _ptr(self.x), _ptr(w), _ptr(self.y))
        self._forward = Launch(dev, lib.hstu_group_fwd, "hstu_group_fwd", self.desc, self.fwd_args, *at)
        if backward:
            _need(want_dx or want_dw, "the backward needs something to compute")
            if want_dx:
                self.dx = dx if dx is not None else torch.empty(rows, K, device=dev, dtype=dx_dtype)
                _check_out(self.dx, "dx")
            if want_dw:
                self.dw = dw if dw is not None else torch.empty(E, K, N, device=dev, dtype=torch.float32)
            b = C.hstu_group_desc.from_buffer_copy(d)
            b.y_stride, b.dx_stride = _step(self.dy, N), _step(self.dx, K)
            self.bwd_desc = b
            self.bwd_args = C.hstu_group_bwd_args(_ptr(group_offsets), _ptr(self.x), _ptr(w), _ptr(self.dy), _ptr(self.dx),
                                                  _ptr(self.dw))
            self._backward = Launch(dev, lib.hstu_group_bwd, "hstu_group_bwd", self.bwd_desc, self.bwd_args, *at)

    def forward(self, stream=None):
        _need(self.y is not None, "a problem without y has no forward")
        self._forward(stream)

    def backward(self, stream=None):
        self._backward(stream)

    def device_error(self, stream=None) -> int:
        return device_error(self.device, self.ws, stream)


class GroupFunction(torch.autograd.Function):
    """y of x and w; gradients for both."""

    @staticmethod
    def forward(ctx, x, w, group_offsets, out_dtype, workspace):
        pr = GroupProblem(x.detach(), w.detach(), group_offsets, out_dtype=out_dtype, workspace=workspace,
                          y=torch.zeros(x.shape[0], w.shape[2], device=x.device, dtype=out_dtype))
        pr.forward()
        ctx.save_for_backward(x, w, group_offsets)
        return pr.y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, off = ctx.saved_tensors
        want_dx, want_dw = ctx.needs_input_grad[:2]
        pr = GroupProblem(x, w, off, dy=dy.to(torch.bfloat16), want_y=False, want_dx=want_dx, want_dw=want_dw,
                          dx=torch.zeros_like(x, memory_format=torch.contiguous_format) if want_dx else None)
        pr.backward()
        return pr.dx, None if pr.dw is None else pr.dw.to(w.dtype), None, None, None


def hstu_group_linear(x, w, group_offsets, *, out_dtype: torch.dtype = torch.bfloat16, workspace=None):
    """Differentiable y[r] = x[r] w[g] for the rows r of group g: x [rows, K]
    and w [groups, K, N] BF16, group_offsets as GroupProblem (group_rows makes
    them).  Rows behind the last group come back as zeros.  The backward rounds
    an FP32 gradient of y to BF16, the tensor cores' operand; the gradient of w
    is FP32 sums rounded to w's type (GroupProblem keeps FP32).  Offsets that are
    out of order raise nothing here: the device records it in the forward's
    workspace (256 zeroed bytes, uint8, 256-byte aligned;
    qk.device_error(device, workspace) != 0), or use GroupProblem.  There is no
    second derivative.  Into a CUDA graph goes GroupProblem's forward and
    backward, rather than autograd's."""
    return GroupFunction.apply(x, w, group_offsets, out_dtype, workspace)
