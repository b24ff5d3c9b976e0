"""AdamW over many tensors in one launch, moments in 32 or in 8 bits, through
hstu_adamw_* of libhstu_attn.so.  Marshalling and checks of arguments only."""
from __future__ import annotations

import bisect
from typing import NamedTuple, Optional

import torch

from . import binding as C
from .attention import _ptr
from .norm import _DTYPES
from .qk import Launch, _need, device_error

BLOCK = 256   # elements that share an exponent byte


class Moments8(NamedTuple):
    """A tensor's moments in 8 bits: codes uint8 (as many as the tensor has
    elements) and a byte for every 256 of them, of each moment (the format is in
    hstu_attn.h)."""
    m: torch.Tensor
    v: torch.Tensor
    m_exp: torch.Tensor
    v_exp: torch.Tensor


def zero_moments(param, bits: int = 32):
    """Moments of a tensor that has not been stepped."""
    _need(bits in (32, 8), f"moments have 32 or 8 bits, not {bits}")
    n, dev = param.numel(), param.device
    if bits == 32:
        return tuple(torch.zeros(n, device=dev, dtype=torch.float32) for _ in range(2))
    byte = dict(device=dev, dtype=torch.uint8)
    return Moments8(*(torch.zeros(n, **byte) for _ in range(2)),
                    *(torch.full(((n + BLOCK - 1) // BLOCK,), 16, **byte) for _ in range(2)))


def _apart(spans, t):
    """Whether t shares no byte with spans (sorted, apart from each other)."""
    lo, hi = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
    i = bisect.bisect_right(spans, (lo, hi))
    return lo == hi or ((i == 0 or spans[i - 1][1] <= lo) and (i == len(spans) or spans[i][0] >= hi))


class AdamW:
    """AdamW for a list of FP32 tensors: step() updates the parameters, their
    moments and their BF16 copies in place, in one launch.

    grads: a list of tensors that every step reads (all BF16 or all FP32; None:
    that parameter is left as it is, while the steps count on: there is one
    count for all, so one whose gradients begin later has no correction of its
    own for its young moments, and moves by up to (1 - beta1) / sqrt(1 - beta2)
    lr at first, 3.2 lr with the usual betas; give such parameters an AdamW of
    their own), or None: the parameters' .grad of the
    moment, looked up at every step (a list that changed is sent anew, which
    waits for the stream; into a CUDA graph goes a step with a list given).
    Gradients at the copies, where those are autograd's leaves, are not
    followed: a step that finds one is refused, and wants a list.
    copies: BF16 tensors (or None) written with the rounded parameters, the
    projections' operands.  weight_decay and lr_scale: a number, or one for
    each tensor.  moments: (m, v) FP32 or Moments8 for each tensor, of the same
    kind; allocated as zeros with state_bits unless given.  steps: steps that
    the moments have seen.  lr, grad_scale (FP32) and skip (int32) may be
    one-element tensors on the device, read at every step; skip: not zero, the
    step changes and counts nothing.  seed: of the 8-bit moments' rounding.

    A step changes the parameters and copies in place as autograd sees it: the
    backward of a graph that saved them before raises (a replayed CUDA graph's
    steps are not seen).

    All tensors are contiguous and 16-byte aligned (copies to 8 bytes, exponent
    bytes to any), must not overlap and stay where they are."""

    def __init__(self, params, grads=None, *, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.0, lr_scale=1.0,
                 copies=None, moments=None, state_bits: int = 32, grad_scale=None, skip=None, steps: int = 0, seed: int = 0,
                 grad_dtype: Optional[torch.dtype] = None):
        self.params = list(params)
        n = len(self.params)
        _need(n > 0, "AdamW needs a tensor")
        dev = self.params[0].device
        self.device = dev
        self.copies = list(copies) if copies is not None else [None] * n
        self.moments = list(moments) if moments is not None else [zero_moments(p, state_bits) for p in self.params]
        self.dynamic = grads is None
        self.grads = [p.grad for p in self.params] if self.dynamic else list(grads)
        each = lambda x, name: [float(x)] * n if isinstance(x, (int, float)) else [float(v) for v in x]  # noqa: E731
        wd, ls = each(weight_decay, "weight_decay"), each(lr_scale, "lr_scale")
        for name, l in (("grads", self.grads), ("copies", self.copies), ("moments", self.moments), ("weight_decay", wd),
                        ("lr_scale", ls)):
            _need(len(l) == n, f"{name}: {len(l)} for {n} tensors")
        bits = 8 if isinstance(self.moments[0], Moments8) else 32
        if grad_dtype is None:
            grad_dtype = next((g.dtype for g in self.grads if g is not None), torch.float32)
        _need(grad_dtype in _DTYPES, f"gradients must be BF16 or FP32, got {grad_dtype}")
        self.grad_dtype = grad_dtype
        spans, rows = [], []
        half = torch.uint8 if bits == 8 else torch.float32
        for i, (p, c, m) in enumerate(zip(self.params, self.copies, self.moments)):
            n_i, at = p.numel(), p.data_ptr()
            if p.device != dev or p.dtype != torch.float32 or not p.is_contiguous() or at % 16:
                raise ValueError(f"parameter {i} must be contiguous FP32 on {dev}, 16-byte aligned")
            spans.append((at, at + 4 * n_i))
            c_at = None
            if c is not None:
                c_at = c.data_ptr()
                if c.device != dev or c.dtype != torch.bfloat16 or c.numel() != n_i or not c.is_contiguous() or c_at % 8:
                    raise ValueError(f"copy {i} must be contiguous BF16 of its parameter's size, on {dev}")
                spans.append((c_at, c_at + 2 * n_i))
            if isinstance(m, Moments8) != (bits == 8):
                raise ValueError("all moments have 32 bits, or all 8")
            m_at = [t.data_ptr() for t in m]
            blocks = (n_i + BLOCK - 1) // BLOCK
            for k, t in enumerate(m):
                size, kind = (n_i, half) if k < 2 else (blocks, torch.uint8)
                if t.device != dev or t.dtype != kind or t.numel() != size or not t.is_contiguous() or (k < 2 and m_at[k] % 16):
                    raise ValueError(f"moments {i} do not match their parameter ({'values' if k < 2 else f'a byte for every {BLOCK}'})")
                spans.append((m_at[k], m_at[k] + size * t.element_size()))
            rows.append((at, c_at, m_at, n_i))
        spans = sorted(x for x in spans if x[1] > x[0])
        _need(all(a[1] <= b[0] for a, b in zip(spans, spans[1:])), "parameters, copies and moments must not overlap")
        self._written = spans
        for i, g in enumerate(self.grads):
            self._check_grad(i, g)
        # what the device writes stays where it is while this object lives, even if a parameter's data moves
        self._held = [t.detach() for t in self.params]
        self._changed = [t for t in (*self.params, *self.copies) if t is not None]
        self.lr_at = lr if isinstance(lr, torch.Tensor) else None
        for name, t, dt in (("lr", self.lr_at, torch.float32), ("grad_scale", grad_scale, torch.float32), ("skip", skip, torch.int32)):
            _need(t is None or (t.dtype == dt and t.numel() == 1 and t.device == dev), f"{name} must be one {dt} on {dev}")
        self.grad_scale, self.skip = grad_scale, skip
        d = C.hstu_adamw_desc()
        d.struct_size = C.ctypes.sizeof(d)
        d.state_bits, d.grad_dtype, d.num_tensors = bits, _DTYPES[grad_dtype], n
        d.lr = 0.0 if self.lr_at is not None else float(lr)
        d.beta1, d.beta2, d.eps = float(betas[0]), float(betas[1]), float(eps)
        d.seed, d.steps_done = int(seed) & 0xFFFFFFFFFFFFFFFF, int(steps)
        self.desc = d
        self._table = (C.hstu_adamw_tensor * n)()
        for i, (at, c_at, m_at, n_i) in enumerate(rows):
            self._table[i] = C.hstu_adamw_tensor(at or None, _ptr(self.grads[i]), c_at, *m_at, *([None] * (4 - len(m_at))), n_i,
                                                 wd[i], ls[i])
        _need(steps >= 0, "steps must not be negative")
        need = C.hstu_adamw_workspace_size(d, self._table)
        self.ws, self.ws_bytes = torch.zeros(need, device=dev, dtype=torch.uint8), need
        self.args = C.hstu_adamw_step_args(_ptr(self.lr_at), _ptr(grad_scale), _ptr(skip))
        self._step = Launch(dev, C.load().hstu_adamw_step, "hstu_adamw_step", d, self.args, self.ws.data_ptr(), need)
        with torch.cuda.device(dev):
            C.hstu_adamw_init(d, self._table, self.ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        self._sent = True

    def _check_grad(self, i, g):
        if g is None:
            return
        p = self.params[i]
        if (g.device != p.device or g.numel() != p.numel() or g.dtype != self.grad_dtype or not g.is_contiguous() or
                g.data_ptr() % 16):
            raise ValueError(f"gradient {i} must be contiguous {self.grad_dtype} of its parameter's size, 16-byte aligned")
        if not _apart(self._written, g):
            raise ValueError(f"gradient {i} overlaps what a step writes")

    @property
    def lr(self):
        return self.lr_at if self.lr_at is not None else self.desc.lr

    @lr.setter
    def lr(self, value):
        _need(self.lr_at is None, "lr lies on the device: write it there")
        _need(0.0 <= float(value) < 1e30, f"lr {value}")
        self.desc.lr = float(value)

    def _follow_grads(self, stream):
        """The parameters' present .grad; a list that changed is sent anew.  A
        step that raises leaves the device's list to be sent by the next one."""
        for i, (p, c) in enumerate(zip(self.params, self.copies)):
            g = p.grad
            if g is None and c is not None and c.is_leaf and c.grad is not None:
                raise ValueError(f"the gradient of parameter {i} lies at its copy, which a step without a list does not follow: give grads")
            if g is not self.grads[i] or _ptr(g) != self._table[i].grad:
                self._check_grad(i, g)
                self._sent = self._sent and _ptr(g) == self._table[i].grad
                self._table[i].grad, self.grads[i] = _ptr(g), g
            if p.data_ptr() != (self._table[i].param or 0):
                raise ValueError(f"parameter {i} is not where it was")
        if not self._sent:
            self.desc.steps_done = -1   # what the device has counted stays
            with torch.cuda.device(self.device):
                s = stream if stream is not None else torch.cuda.current_stream()
                C.hstu_adamw_init(self.desc, self._table, self.ws.data_ptr(), self.ws_bytes, s.cuda_stream)
            self._sent = True

    def step(self, stream=None):
        if self.dynamic:
            self._follow_grads(stream)
        self._step(stream)
        torch.autograd.graph.increment_version(self._changed)   # a backward that saved them finds out

    def steps(self, stream=None) -> int:
        """Steps counted so far.  Waits for the stream (default: the current one)."""
        with torch.cuda.device(self.device):
            s = stream if stream is not None else torch.cuda.current_stream()
            return C.hstu_adamw_steps(self.ws.data_ptr(), s.cuda_stream)

    def reader(self, outs):
        """A MomentsReader that writes the moments as values into outs, a pair
        (m, v) of tensors for each parameter (either may be None), all FP32 or all BF16."""
        return MomentsReader(self, outs)

    def read_moments(self, dtype: torch.dtype = torch.float32):
        """The moments' values, a new pair (m, v) shaped like each parameter."""
        outs = [tuple(torch.empty(p.shape, device=self.device, dtype=dtype) for _ in range(2)) for p in self.params]
        MomentsReader(self, outs).run()
        return outs

    def device_error(self, stream=None) -> int:
        return device_error(self.device, self.ws, stream)


class MomentsReader:
    """run() writes an AdamW's moments as values (8-bit ones decoded) into the
    tensors given, in one launch."""

    def __init__(self, optimizer: AdamW, outs):
        self.optimizer, self.outs = optimizer, list(outs)
        dev = optimizer.device
        _need(len(self.outs) == len(optimizer.params), f"{len(self.outs)} pairs for {len(optimizer.params)} tensors")
        dtype = next((t.dtype for pair in self.outs for t in pair if t is not None), torch.float32)
        _need(dtype in _DTYPES, f"moments are read as BF16 or FP32, not {dtype}")
        for p, pair in zip(optimizer.params, self.outs):
            _need(len(pair) == 2, "a pair (m, v) for each tensor")
            for t in pair:
                if t is not None and (t.device != dev or t.dtype != dtype or t.numel() != p.numel() or not t.is_contiguous() or
                                      t.data_ptr() % 16):
                    raise ValueError("a moment's values must be contiguous, 16-byte aligned, of one type")
                if t is not None and not _apart(optimizer._written, t):
                    raise ValueError("a moment's values overlap what a step writes")
        d = C.hstu_adamw_desc.from_buffer_copy(optimizer.desc)
        self.desc = d
        table = (C.hstu_adamw_moments * len(self.outs))(*(C.hstu_adamw_moments(_ptr(a), _ptr(b)) for a, b in self.outs))
        need = C.hstu_adamw_workspace_size(d, optimizer._table)
        self.ws = torch.zeros(need, device=dev, dtype=torch.uint8)
        self._run = Launch(dev, C.load().hstu_adamw_read, "hstu_adamw_read", d, self.ws.data_ptr(), need)
        with torch.cuda.device(dev):
            C.hstu_adamw_read_init(d, optimizer._table, table, _DTYPES[dtype], self.ws.data_ptr(), need,
                                   torch.cuda.current_stream().cuda_stream)

    def run(self, stream=None):
        self._run(stream)

    def device_error(self, stream=None) -> int:
        return device_error(self.optimizer.device, self.ws, stream)
