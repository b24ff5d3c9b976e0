"""Queries and keys before the attention: an RMS norm per head and a rotation
by position, in one pass, through hstu_qk_norm_rope_fwd / _bwd of
libhstu_attn.so.  Marshalling and checks of arguments only."""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as C
from .attention import _ptr


def rope_tables(max_position: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """cos and sin [max_position, rot_dim / 2] FP32 of the angles
    p base^(-2i / rot_dim), computed in 64 bits."""
    if rot_dim < 2 or rot_dim % 2 or max_position < 1:
        raise ValueError(f"rope_tables: rot_dim {rot_dim} and max_position {max_position}")
    i = torch.arange(rot_dim // 2, device=device, dtype=torch.float64)
    a = torch.arange(max_position, device=device, dtype=torch.float64)[:, None] * (base ** (-2.0 * i / rot_dim))
    return a.cos().float(), a.sin().float()


def jagged_positions(seq_offsets, num_targets=None, starts=None, total_tokens: Optional[int] = None):
    """Position of every packed token: its index in its sequence (plus
    starts[b]), a candidate's the one behind the history, as in the
    attention's position buckets.  (Rows over a cache that holds some of them
    already: cached_positions.)  int32 [T]."""
    T = int(seq_offsets[-1]) if total_tokens is None else total_tokens
    t = torch.arange(T, device=seq_offsets.device)
    b = torch.searchsorted(seq_offsets, t, right=True).sub_(1).clamp_(max=seq_offsets.numel() - 2)
    pos = t - seq_offsets[b]
    if num_targets is not None:
        pos = torch.minimum(pos, (seq_offsets[1:] - seq_offsets[:-1] - num_targets)[b])
    if starts is not None:
        pos = pos + starts[b]
    return pos.to(torch.int32)


def cached_positions(seq_offsets, cache_lens, num_targets=None, total_tokens: Optional[int] = None):
    """Position of every packed row of hstu_attention_cached: cache_lens[b]
    counts a sequence's new history rows already (they were appended), so
    those are the last positions below it, as in the cache, and a candidate
    has cache_lens[b].  The tables of the rotation need a row more than the
    longest cache.  int32 [T]."""
    history = seq_offsets[1:] - seq_offsets[:-1]
    if num_targets is not None:
        history = history - num_targets
    return jagged_positions(seq_offsets, num_targets, cache_lens - history, total_tokens)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _same_device(device, **tensors):
    for name, t in tensors.items():
        _need(t is None or t.device == device, f"{name} is on {getattr(t, 'device', None)}, not on {device}")


def _strides(t):
    # (those of a tensor without elements lead nowhere and follow no rule)
    return (0, 0) if t is None or t.numel() == 0 else (t.stride(0), t.stride(1))


def _rows(t, name):
    """[T, H, d] with contiguous features and 16-byte steps, as the kernels
    take it; any other layout is copied."""
    per = 16 // t.element_size()
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, H, d], got {tuple(t.shape)}")
    if t.numel() and (t.stride(2) != 1 or t.stride(0) % per or t.stride(1) % per or t.data_ptr() % 16 or
                      t.stride(0) < 0 or t.stride(1) < 0):
        return t.contiguous()
    return t


def _fills(t):
    """Whether no two of an output's elements share their place."""
    dims = sorted((t.stride(i), t.shape[i]) for i in range(3) if t.shape[i] > 1)
    reach = 1
    for stride, size in dims:
        if stride < reach:
            return False
        reach = stride * (size - 1) + reach
    return True


class QKProblem:
    """q [T, Hq, d] and k [T, Hk, d] (either may be None), the tables and the
    outputs, with the C argument structs filled once; forward() fills q_out,
    k_out, backward() dq, dk, d_q_gain, d_k_gain from dq_out, dk_out.

    q and k are used in place where their features are contiguous and heads
    and tokens lie multiples of 16 bytes apart (parts of one projection's
    output, say), else copied once, here.  The outputs are allocated unless
    given; inplace=True writes over q and k (not with the backward of a norm,
    which needs them)."""

    def __init__(self, q, k, positions=None, cos=None, sin=None, *, rot_dim: Optional[int] = None,
                 interleaved: bool = False, norm: bool = True, eps: float = 1e-6, q_gain=None, k_gain=None,
                 num_tokens=None, dq_out=None, dk_out=None, q_out=None, k_out=None, inplace: bool = False,
                 want_gain_grads: bool = True, workspace=None):
        ref = q if q is not None else k
        _need(ref is not None, "QKProblem needs q or k")
        _need(ref.dtype in (torch.bfloat16, torch.float32), f"q, k must be BF16 or FP32, got {ref.dtype}")
        dev = ref.device
        self.device = dev
        _same_device(dev, q=q, k=k, positions=positions, cos=cos, sin=sin, q_gain=q_gain, k_gain=k_gain,
                     num_tokens=num_tokens, dq_out=dq_out, dk_out=dk_out, q_out=q_out, k_out=k_out, workspace=workspace)
        if rot_dim is None:
            rot_dim = 0 if cos is None else 2 * cos.shape[1]
        T, d = ref.shape[0], ref.shape[2]
        for name, t in (("q", q), ("k", k), ("dq_out", dq_out), ("dk_out", dk_out), ("q_out", q_out), ("k_out", k_out)):
            if t is None:
                continue
            src = q if name in ("q", "dq_out", "q_out") else k
            _need(src is not None and t.dim() == 3 and t.shape == src.shape and t.dtype == ref.dtype and
                  t.shape[0] == T and t.shape[2] == d, f"{name} does not match q, k in shape or type")
        if rot_dim:
            _need(positions is not None and positions.dtype == torch.int32 and positions.shape == (T,) and
                  positions.is_contiguous(), "positions must be int32 [T]")
            _need(cos is not None and sin is not None and cos.shape == sin.shape and cos.dim() == 2 and
                  cos.shape[1] == rot_dim // 2 and cos.dtype == sin.dtype == torch.float32 and
                  cos.is_contiguous() and sin.is_contiguous(), "cos, sin must be FP32 [max_position, rot_dim / 2]")
        for name, g in (("q_gain", q_gain), ("k_gain", k_gain)):
            _need(g is None or (norm and g.shape == (d,) and g.dtype == torch.float32 and g.is_contiguous()),
                  f"{name} must be FP32 [d], with norm")
        _need(num_tokens is None or (num_tokens.dtype == torch.int64 and num_tokens.numel() == 1),
              "num_tokens must be one int64 on the device")
        self.q, self.k = (None if t is None else _rows(t, n) for t, n in ((q, "q"), (k, "k")))
        _need(not inplace or (self.q is q and self.k is k), "in place needs 16-byte steps and contiguous features")
        new = lambda t: None if t is None else torch.empty(t.shape, device=dev, dtype=t.dtype)  # noqa: E731
        self.q_out = q_out if q_out is not None else (q if inplace else new(q))
        self.k_out = k_out if k_out is not None else (k if inplace else new(k))
        for name, t in (("q_out", self.q_out), ("k_out", self.k_out)):
            _need(t is None or (_rows(t, name) is t and _fills(t)), f"{name} needs places of its own, 16 bytes apart")
        self.dq_out, self.dk_out = (None if t is None else _rows(t, n) for t, n in ((dq_out, "dq_out"), (dk_out, "dk_out")))
        self.positions, self.cos, self.sin, self.q_gain, self.k_gain = positions, cos, sin, q_gain, k_gain
        self.num_tokens = num_tokens
        backward = dq_out is not None or dk_out is not None
        _need(not backward or ((dq_out is None) == (q is None) and (dk_out is None) == (k is None)),
              "the backward needs the gradients of both outputs")
        for x, out in ((self.q, self.q_out), (self.k, self.k_out)):
            _need(not (backward and norm) or x is None or x.numel() == 0 or x.data_ptr() != out.data_ptr(),
                  "the norm's backward needs the inputs, which a forward in place overwrites")
        self.dq, self.dk = (new(q), new(k)) if backward else (None, None)
        gain = lambda t, g: torch.empty(d, device=dev, dtype=torch.float32) \
            if backward and norm and want_gain_grads and t is not None and g is not None else None  # noqa: E731
        self.d_q_gain, self.d_k_gain = gain(q, q_gain), gain(k, k_gain)
        D = C.hstu_qk_desc()
        D.struct_size = C.ctypes.sizeof(D)
        D.dtype = C.HSTU_BF16 if ref.dtype == torch.bfloat16 else C.HSTU_FP32
        D.Hq, D.Hk, D.d = 0 if q is None else q.shape[1], 0 if k is None else k.shape[1], d
        D.rot_dim, D.interleaved, D.norm, D.eps = rot_dim, int(interleaved), int(norm), eps
        D.total_tokens, D.max_position = T, cos.shape[0] if rot_dim else 0
        D.q_strides, D.k_strides = _strides(self.q), _strides(self.k)
        D.q_out_strides, D.k_out_strides = _strides(self.q_out), _strides(self.k_out)
        self.desc = D
        fwd_b, bwd_b = C.hstu_qk_workspace_size(D)
        need = max(fwd_b, bwd_b if backward else 0)
        if workspace is None:
            workspace = torch.zeros(need, device=dev, dtype=torch.uint8)
        _need(workspace.dtype == torch.uint8 and workspace.is_contiguous(), "workspace must be contiguous uint8")
        self.ws, self.ws_bytes = workspace, workspace.numel()
        common = (_ptr(num_tokens), _ptr(positions), _ptr(cos), _ptr(sin), _ptr(q_gain), _ptr(k_gain), _ptr(self.q),
                  _ptr(self.k))
        self.fwd_args = C.hstu_qk_fwd_args(*common, _ptr(self.q_out), _ptr(self.k_out))
        if backward:
            B = C.hstu_qk_desc.from_buffer_copy(D)
            B.q_out_strides, B.k_out_strides = _strides(self.dq_out), _strides(self.dk_out)
            B.dq_strides, B.dk_strides = _strides(self.dq), _strides(self.dk)
            self.bwd_desc = B
            self.bwd_args = C.hstu_qk_bwd_args(*common, _ptr(self.dq_out), _ptr(self.dk_out), _ptr(self.dq), _ptr(self.dk),
                                               _ptr(self.d_q_gain), _ptr(self.d_k_gain))

        lib, w = C.load(), (self.ws.data_ptr(), self.ws_bytes)
        self._forward = Launch(dev, lib.hstu_qk_norm_rope_fwd, "hstu_qk_norm_rope_fwd", self.desc, self.fwd_args, *w)
        if backward:
            self._backward = Launch(dev, lib.hstu_qk_norm_rope_bwd, "hstu_qk_norm_rope_bwd", self.bwd_desc, self.bwd_args, *w)

    def forward(self, stream=None):
        self._forward(stream)

    def backward(self, stream=None):
        self._backward(stream)

    def device_error(self, stream=None) -> int:
        return device_error(self.device, self.ws, stream)


class Launch:
    """One C call with its arguments put together once: calling it launches on
    the given stream, or on the current one of the tensors' device.

    What a problem makes for itself (a zeroed workspace, copies of tensors in
    other layouts) is queued on the stream that is current then; the first call
    on another stream waits for that one.  The caller's own tensors are the
    caller's to wait for.  A call that is being captured waits for nothing: make
    the problem before the capture begins (torch.cuda.graph synchronises)."""

    __slots__ = ("index", "fn", "name", "args", "keep", "made", "known")

    def __init__(self, device, fn, name, *args):
        _need(device.type == "cuda", f"{name} needs tensors on a CUDA device, not on {device}")
        self.index = device.index if device.index is not None else torch.cuda.current_device()
        self.fn, self.name, self.keep = fn, name, args
        self.args = tuple(C.ctypes.byref(a) if isinstance(a, C.ctypes.Structure) else a for a in args)
        self.made = torch.cuda.current_stream(self.index)
        self.known = {self.made.cuda_stream}    # streams that have waited

    def __call__(self, stream=None):
        if torch._C._cuda_getDevice() != self.index:    # the launches go to the current device
            with torch.cuda.device(self.index):
                return self(stream)
        s = torch._C._cuda_getCurrentRawStream(self.index) if stream is None else stream.cuda_stream
        if s not in self.known:
            self._wait(stream if stream is not None else torch.cuda.current_stream(self.index))
        status = self.fn(*self.args, s)
        if status:
            raise C.HSTUError(status, self.name)

    def _wait(self, stream):
        for s in (stream, self.made):
            with torch.cuda.stream(s):
                if torch.cuda.is_current_stream_capturing():
                    return
        stream.wait_stream(self.made)
        self.known.add(stream.cuda_stream)


def device_error(device, workspace, stream=None) -> int:
    """The first error that a call with this workspace found on the device (0:
    none), kept until the header, its first 256 bytes, is zeroed.  Waits for
    the stream (default: the current one)."""
    with torch.cuda.device(device):
        s = stream if stream is not None else torch.cuda.current_stream()
        return C.hstu_get_device_error(workspace.data_ptr(), s.cuda_stream)


class QKNormRopeFunction(torch.autograd.Function):
    """(q', k') of q, k; gradients for q, k and the gains."""

    @staticmethod
    def forward(ctx, q, k, q_gain, k_gain, positions, cos, sin, num_tokens, rot_dim, interleaved, norm, eps, workspace):
        pr = QKProblem(q.detach() if q is not None else None, k.detach() if k is not None else None, positions, cos, sin,
                       rot_dim=rot_dim, interleaved=interleaved, norm=norm, eps=eps, q_gain=q_gain, k_gain=k_gain,
                       num_tokens=num_tokens, workspace=workspace)
        if num_tokens is not None:   # rows behind the batch are written by nobody
            for t in (pr.q_out, pr.k_out):
                if t is not None:
                    t.zero_()
        pr.forward()
        ctx.save_for_backward(q, k, q_gain, k_gain, positions, cos, sin, num_tokens)
        ctx.how = (rot_dim, interleaved, norm, eps)
        return pr.q_out, pr.k_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_gain, k_gain, positions, cos, sin, num_tokens = ctx.saved_tensors
        rot_dim, interleaved, norm, eps = ctx.how
        full = lambda g, t: None if t is None else (torch.zeros_like(t) if g is None else g.to(t.dtype))  # noqa: E731
        pr = QKProblem(q, k, positions, cos, sin, rot_dim=rot_dim, interleaved=interleaved, norm=norm, eps=eps,
                       q_gain=q_gain, k_gain=k_gain, num_tokens=num_tokens, dq_out=full(dq_out, q), dk_out=full(dk_out, k))
        if num_tokens is not None:
            for t in (pr.dq, pr.dk):
                if t is not None:
                    t.zero_()
        pr.backward()
        return (pr.dq, pr.dk, pr.d_q_gain, pr.d_k_gain) + (None,) * 9


def hstu_qk_norm_rope(q, k, positions=None, cos=None, sin=None, *, q_gain=None, k_gain=None, norm: bool = True,
                      eps: float = 1e-6, rot_dim: Optional[int] = None, interleaved: bool = False, num_tokens=None,
                      workspace=None):
    """Differentiable norm and rotation of q [T, Hq, d] and k [T, Hk, d]
    (either may be None): returns (q', k') for hstu_attention.  cos, sin:
    rope_tables; positions: jagged_positions, cached_positions, or any int32
    [T] below max_position.  num_tokens: one int64 on the device, tokens in use of a
    padded batch (rows behind it come back as zeros).  A position outside the
    tables raises nothing here: the device records it in the forward's
    workspace.  Give one to look (256 zeroed bytes, uint8, 256-byte aligned;
    device_error(device, workspace) != 0), or use QKProblem, which keeps its
    own.  There is no second derivative.  Into a CUDA graph goes QKProblem's
    forward and backward, rather than autograd's."""
    if rot_dim is None:
        rot_dim = 0 if cos is None else 2 * cos.shape[1]
    return QKNormRopeFunction.apply(q, k, q_gain, k_gain, positions, cos, sin, num_tokens, int(rot_dim), bool(interleaved),
                                    bool(norm), float(eps), workspace)
