"""A paged cache of keys and values in 4 bits: appending to it, reading it
back, and the HSTU attention of new rows over it, through hstu_cache_append,
hstu_cache_read and hstu_attn_fwd_cached of libhstu_attn.so.  Marshalling and
checks of arguments only."""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as C
from .attention import _ptr
from .qk import Launch, _need, _rows, _same_device, _strides, device_error


class PagedCache:
    """Pages of one layer's keys and values (see the cache section of
    hstu_attn.h): pages uint8 [num_pages, H, bytes], timestamps int64
    [num_pages, page_size] or None.  Allocated here (zeroed, on the current
    stream) unless given.
    Which page belongs to whom is the caller's book-keeping (block tables)."""

    def __init__(self, num_pages: Optional[int] = None, *, H: int, d: int, page_size: int = 64, k_exp: int = 0, v_exp: int = 0,
                 timestamps=True, pages=None, device="cuda"):
        if pages is not None:
            _need(pages.dtype == torch.uint8 and pages.is_contiguous() and pages.dim() == 3 and pages.shape[1] == H,
                  "pages must be contiguous uint8 [num_pages, H, bytes]")
            _need(num_pages is None or num_pages == pages.shape[0], "num_pages does not match pages")
            num_pages, device = pages.shape[0], pages.device
        _need(num_pages is not None, "PagedCache needs num_pages or pages")
        D = C.hstu_cache_desc()
        D.struct_size = C.ctypes.sizeof(D)
        D.H, D.d, D.page_size, D.num_pages, D.k_exp, D.v_exp, D.max_pages = H, d, page_size, num_pages, k_exp, v_exp, 1
        page_bytes, _ = C.hstu_cache_bytes(D)
        if pages is None:
            pages = torch.zeros(num_pages, H, page_bytes // H, device=device, dtype=torch.uint8)
        _need(pages.shape[2] * H == page_bytes, f"a page of a head has {page_bytes // H} bytes, not {pages.shape[2]}")
        if timestamps is True:
            timestamps = torch.zeros(num_pages, page_size, device=pages.device, dtype=torch.int64)
        elif timestamps is False:
            timestamps = None
        _need(timestamps is None or (timestamps.dtype == torch.int64 and timestamps.is_contiguous() and
                                     timestamps.shape == (num_pages, page_size) and timestamps.device == pages.device),
              "timestamps must be contiguous int64 [num_pages, page_size]")
        self.pages, self.timestamps, self.device = pages, timestamps, pages.device
        self.H, self.d, self.page_size, self.num_pages = H, d, page_size, num_pages
        D.pages, D.timestamps = _ptr(pages), _ptr(timestamps)
        self._desc = D

    def desc(self, max_pages: int) -> C.hstu_cache_desc:
        d = C.hstu_cache_desc.from_buffer_copy(self._desc)
        d.max_pages = max_pages
        return d


def _check_batch(cache, seq_offsets, block_table, lens, B, what):
    dev = cache.device
    _need(seq_offsets.dtype == torch.int64 and seq_offsets.is_contiguous() and seq_offsets.dim() == 1 and B >= 0,
          "seq_offsets must be contiguous int64 [B+1]")
    _need(block_table.dtype == torch.int32 and block_table.is_contiguous() and block_table.dim() == 2 and
          block_table.shape[0] == B and block_table.shape[1] >= 1, "block_table must be contiguous int32 [B, max_pages]")
    _need(lens is None or (lens.dtype == torch.int32 and lens.is_contiguous() and lens.shape == (B,)),
          f"{what} must be contiguous int32 [B]")
    _same_device(dev, seq_offsets=seq_offsets, block_table=block_table, **{what: lens})


class _Call:
    def _workspace(self, bytes_, workspace):
        if workspace is None:
            workspace = torch.zeros(bytes_, device=self.device, dtype=torch.uint8)
        _need(workspace.device == self.device and workspace.dtype == torch.uint8 and workspace.is_contiguous(),
              "workspace must be contiguous uint8 on the cache's device")
        self.ws, self.ws_bytes = workspace, workspace.numel()

    def _prepare(self, name, *args):
        self._launch = Launch(self.device, getattr(C.load(), name), name, *args, self.ws.data_ptr(), self.ws_bytes)

    def device_error(self, stream=None) -> int:
        return device_error(self.device, self.ws, stream)


class AppendProblem(_Call):
    """k, v [T, H, d] BF16 of the batch's new tokens on their way into the
    cache: run() writes them at the last positions of each sequence
    (cache_lens counts them already), keys through norm and rotation.  k, v are
    read in place where their features are contiguous and heads and tokens lie
    multiples of 16 bytes apart, else copied once, here."""

    def __init__(self, cache: PagedCache, k, v, seq_offsets, cache_lens, block_table, *, timestamps=None, cos=None, sin=None,
                 rot_dim: Optional[int] = None, interleaved: bool = False, norm: bool = False, eps: float = 1e-6, k_gain=None,
                 workspace=None):
        self.device, B = cache.device, seq_offsets.numel() - 1
        _check_batch(cache, seq_offsets, block_table, cache_lens, B, "cache_lens")
        _same_device(self.device, k=k, v=v, timestamps=timestamps, cos=cos, sin=sin, k_gain=k_gain)
        if rot_dim is None:
            rot_dim = 0 if cos is None else 2 * cos.shape[1]
        T = k.shape[0]
        for name, t in (("k", k), ("v", v)):
            _need(t.dtype == torch.bfloat16 and t.shape == (T, cache.H, cache.d), f"{name} must be BF16 [T, H, d] of the cache")
        _need((timestamps is None) == (cache.timestamps is None), "the cache keeps timestamps iff tokens have them")
        _need(timestamps is None or (timestamps.dtype == torch.int64 and timestamps.shape == (T,) and timestamps.is_contiguous()),
              "timestamps must be int64 [T]")
        if rot_dim:
            _need(cos is not None and sin is not None and cos.shape == sin.shape and cos.dim() == 2 and
                  cos.shape[1] == rot_dim // 2 and cos.dtype == sin.dtype == torch.float32 and cos.is_contiguous() and
                  sin.is_contiguous(), "cos, sin must be FP32 [max_position, rot_dim / 2]")
        _need(k_gain is None or (norm and k_gain.shape == (cache.d,) and k_gain.dtype == torch.float32 and k_gain.is_contiguous()),
              "k_gain must be FP32 [d], with norm")
        self.k, self.v = _rows(k, "k"), _rows(v, "v")
        self.keep = (cache, seq_offsets, cache_lens, block_table, timestamps, cos, sin, k_gain)
        self._workspace(256, workspace)
        self.desc = cache.desc(block_table.shape[1])
        a = C.hstu_cache_append_args()
        a.B, a.rot_dim, a.interleaved, a.norm, a.eps = B, rot_dim, int(interleaved), int(norm), eps
        a.total_tokens, a.max_position = T, cos.shape[0] if rot_dim else 0
        a.k_strides, a.v_strides = _strides(self.k), _strides(self.v)
        a.seq_offsets, a.cache_lens, a.block_table = _ptr(seq_offsets), _ptr(cache_lens), _ptr(block_table)
        a.token_times, a.cos, a.sin, a.k_gain, a.k, a.v = (_ptr(t) for t in (timestamps, cos, sin, k_gain, self.k, self.v))
        self.args = a
        self._prepare("hstu_cache_append", self.desc, self.args)

    def run(self, stream=None):
        self._launch(stream)


class ReadProblem(_Call):
    """Tokens of the cache as values: run() fills k, v [T, H, d] BF16 (and
    timestamps [T]) with positions [starts[b], starts[b] + n_b) of each
    sequence, packed by seq_offsets: what hstu_attn_fwd_delta takes as its
    packed cache."""

    def __init__(self, cache: PagedCache, seq_offsets, starts, block_table, *, total_tokens: Optional[int] = None, workspace=None):
        self.device, B = cache.device, seq_offsets.numel() - 1
        _check_batch(cache, seq_offsets, block_table, starts, B, "starts")
        T = int(seq_offsets[-1]) if total_tokens is None else total_tokens
        new = lambda *s, dt=torch.bfloat16: torch.empty(*s, device=self.device, dtype=dt)  # noqa: E731
        self.k, self.v = new(T, cache.H, cache.d), new(T, cache.H, cache.d)
        self.timestamps = new(T, dt=torch.int64) if cache.timestamps is not None else None
        self.keep = (cache, seq_offsets, starts, block_table)
        self._workspace(256, workspace)
        self.desc = cache.desc(block_table.shape[1])
        a = C.hstu_cache_read_args()
        a.B, a.total_tokens = B, T
        a.seq_offsets, a.starts, a.block_table = _ptr(seq_offsets), _ptr(starts), _ptr(block_table)
        a.k, a.v, a.token_times = _ptr(self.k), _ptr(self.v), _ptr(self.timestamps)
        self.args = a
        self._prepare("hstu_cache_read", self.desc, self.args)

    def run(self, stream=None):
        self._launch(stream)


class CachedProblem(_Call):
    """New rows over the cache: forward() fills o [T, H, d] and y [T, H*d]
    BF16.  The last num_targets[b] rows of a sequence are candidates (their own
    k, v are read), those before them its newest history tokens, already
    appended.  q, k, v, u that are not contiguous are copied once, here."""

    def __init__(self, cache: PagedCache, q, k, v, u, seq_offsets, cache_lens, block_table, *, max_rows: int, max_seq_len: int,
                 alpha: float, num_targets=None, timestamps=None, rab_pos=None, rab_time=None, norm: str = "layernorm",
                 eps: float = 1e-5, workspace=None):
        self.device, B = cache.device, seq_offsets.numel() - 1
        _check_batch(cache, seq_offsets, block_table, cache_lens, B, "cache_lens")
        _same_device(self.device, q=q, k=k, v=v, u=u, num_targets=num_targets, timestamps=timestamps, rab_pos=rab_pos,
                     rab_time=rab_time)
        T, H, d = q.shape
        _need((H, d) == (cache.H, cache.d), f"q is {H} x {d}, the cache {cache.H} x {cache.d}")
        for name, t, shape in (("q", q, (T, H, d)), ("k", k, (T, H, d)), ("v", v, (T, H, d)), ("u", u, (T, H * d))):
            _need(t is None or (t.dtype == torch.bfloat16 and t.shape == shape), f"{name} must be BF16 {shape}")
        _need(num_targets is None or (num_targets.dtype == torch.int32 and num_targets.shape == (B,) and
                                      num_targets.is_contiguous()), "num_targets must be int32 [B]")
        _need(num_targets is None or (k is not None and v is not None), "candidates need their own k and v")
        _need(timestamps is None or (timestamps.dtype == torch.int64 and timestamps.shape == (T,) and
                                     timestamps.is_contiguous()), "timestamps must be int64 [T]")
        _need(timestamps is None or cache.timestamps is not None, "row timestamps need the cache's")
        for name, t in (("rab_pos", rab_pos), ("rab_time", rab_time)):
            _need(t is None or (t.dtype == torch.float32 and t.dim() == 2 and t.shape[0] == H and t.is_contiguous()),
                  f"{name} must be FP32 [H, buckets]")
        self.q, self.k, self.v, self.u = (None if t is None else t.contiguous() for t in (q, k, v, u))
        self.o = torch.empty(T, H, d, device=self.device, dtype=torch.bfloat16)
        self.y = torch.empty(T, H * d, device=self.device, dtype=torch.bfloat16)
        self.desc = C.make_desc(dtype="bf16", out_dtype="bf16", B=B, H=H, d_qk=d, d_v=d, total_tokens=T,
                                max_seq_len=max_seq_len, alpha=alpha,
                                num_pos_buckets=rab_pos.shape[1] if rab_pos is not None else 128,
                                num_time_buckets=rab_time.shape[1] if rab_time is not None else 64, norm=norm, ln_eps=eps)
        self.cache_desc = cache.desc(block_table.shape[1])
        self.keep = (cache, seq_offsets, cache_lens, block_table, num_targets, timestamps, rab_pos, rab_time)
        self._workspace(C.hstu_attn_cached_workspace_size(self.desc, self.cache_desc, max_rows), workspace)
        a = C.hstu_attn_cached_args()
        a.max_rows = max_rows
        a.seq_offsets, a.cache_lens, a.num_targets, a.block_table = (_ptr(t) for t in (seq_offsets, cache_lens, num_targets,
                                                                                      block_table))
        a.row_times, a.rab_pos, a.rab_time = _ptr(timestamps), _ptr(rab_pos), _ptr(rab_time)
        a.q, a.k, a.v, a.u, a.o, a.y = (_ptr(t) for t in (self.q, self.k, self.v, self.u, self.o, self.y))
        self.args = a
        self._prepare("hstu_attn_fwd_cached", self.desc, self.cache_desc, self.args)

    def forward(self, stream=None):
        self._launch(stream)


# What the device finds wrong with offsets, lengths or page numbers raises nothing
# in the calls below, which drop the workspace that they make: a token without a
# place is left out, the rows of a refused batch hold nothing.  To look, hold a
# problem and ask its device_error(), or pass workspace= (zeroed uint8, 256 bytes
# but for the attention) and ask qk.device_error(device, workspace).

def hstu_cache_append(cache: PagedCache, k, v, seq_offsets, cache_lens, block_table, **kw) -> None:
    """Append once (AppendProblem's arguments).  Device errors: only with a
    workspace of the caller's (above)."""
    AppendProblem(cache, k, v, seq_offsets, cache_lens, block_table, **kw).run()


def hstu_cache_read(cache: PagedCache, seq_offsets, starts, block_table, **kw):
    """(k, v, timestamps) of the asked positions (ReadProblem's arguments; rows
    behind the last sequence hold nothing).  Device errors as in hstu_cache_append."""
    pr = ReadProblem(cache, seq_offsets, starts, block_table, **kw)
    pr.run()
    return pr.k, pr.v, pr.timestamps


def hstu_attention_cached(cache: PagedCache, q, k, v, u, seq_offsets, cache_lens, block_table, **kw):
    """(o, y) of new rows over the cache (CachedProblem's arguments; rows behind
    the last sequence hold nothing).  Device errors as in hstu_cache_append."""
    pr = CachedProblem(cache, q, k, v, u, seq_offsets, cache_lens, block_table, **kw)
    pr.forward()
    return pr.o, pr.y
