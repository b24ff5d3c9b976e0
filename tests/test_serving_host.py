"""What the query/key norm, the 4-bit cache and the attention over it refuse on
the host: the C entries (they return before any CUDA call) and the Python
classes' checks of their tensors."""
import ctypes

import pytest

from hstu_jagged_attention_02_gb300 import binding as C

BAD, NOT, WS = C.HSTU_ERR_INVALID_ARG, C.HSTU_ERR_UNSUPPORTED, C.HSTU_ERR_WORKSPACE
PTR = 1 << 20          # stands for a device address: nothing is read before the checks are through


def _status(fn, *args):
    try:
        fn(*args)
    except C.HSTUError as e:
        return e.status
    return 0


def _set(x, kw):
    for name, value in kw.items():
        if isinstance(value, tuple):
            value = type(getattr(x, name))(*value)
        setattr(x, name, value)
    return x


def _qk(**kw):
    d = C.hstu_qk_desc()
    d.struct_size = ctypes.sizeof(d)
    d.dtype, d.Hq, d.Hk, d.d, d.rot_dim, d.norm, d.eps = C.HSTU_BF16, 4, 2, 64, 32, 1, 1e-6
    d.total_tokens, d.max_position = 10, 100
    for name, H in (("q", 4), ("k", 2), ("q_out", 4), ("k_out", 2), ("dq", 4), ("dk", 2)):
        _set(d, {(name + "_strides"): (H * 64, 64)})
    return _set(d, kw)


def _qk_args(cls, **kw):
    a = cls()
    for name, _ in cls._fields_:
        setattr(a, name, PTR)
    return _set(a, kw)


@pytest.mark.parametrize("kw,status", [
    (dict(struct_size=8), BAD), (dict(dtype=7), BAD), (dict(Hq=-1), BAD), (dict(Hq=0, Hk=0), BAD),
    (dict(total_tokens=-1), BAD), (dict(reserved=1), BAD), (dict(interleaved=2), BAD), (dict(norm=-1), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(rot_dim=-8), BAD), (dict(rot_dim=72), BAD),
    (dict(max_position=0), BAD), (dict(d=48), NOT), (dict(rot_dim=20), NOT), (dict(Hq=5000), NOT),
    (dict(total_tokens=1 << 28), NOT), (dict(q_strides=(256, 4)), BAD), (dict(k_out_strides=(130, 64)), BAD),
])
def test_qk_descriptions(kw, status):
    d = _qk(**kw)
    assert _status(C.hstu_qk_workspace_size, d) == status
    assert _status(C.hstu_qk_norm_rope_fwd, d, _qk_args(C.hstu_qk_fwd_args), PTR, 1 << 20, 0) == status


@pytest.mark.parametrize("bwd,desc,kw,ws,status", [
    (0, {}, dict(q=None), (PTR, 256), BAD), (0, {}, dict(k_out=None), (PTR, 256), BAD),
    (0, {}, dict(positions=None), (PTR, 256), BAD), (0, {}, dict(sin=None), (PTR, 256), BAD),
    (0, {}, dict(q=PTR + 8), (PTR, 256), BAD), (0, {}, dict(k_out=PTR + 2), (PTR, 256), BAD),
    (0, {}, dict(cos=PTR + 4), (PTR, 256), BAD), (0, dict(norm=0), {}, (PTR, 256), BAD),
    (0, {}, {}, (0, 256), WS), (0, {}, {}, (PTR + 16, 1024), WS), (0, {}, {}, (PTR, 255), WS),
    (1, {}, dict(dq=None), (PTR, 1 << 20), BAD), (1, {}, dict(dk_out=None), (PTR, 1 << 20), BAD),
    (1, {}, dict(q=None), (PTR, 1 << 20), BAD), (1, {}, dict(dk=PTR + 4), (PTR, 1 << 20), BAD),
    (1, dict(dq_strides=(256, 68)), {}, (PTR, 1 << 20), BAD),
    (1, dict(norm=0), dict(q_gain=None, k_gain=None), (PTR, 1 << 20), BAD),     # gains' gradients without the norm
    (1, {}, {}, (PTR, 256), WS),
])
def test_qk_calls(bwd, desc, kw, ws, status):
    fn, cls = (C.hstu_qk_norm_rope_bwd, C.hstu_qk_bwd_args) if bwd else (C.hstu_qk_norm_rope_fwd, C.hstu_qk_fwd_args)
    assert _status(fn, _qk(**desc), _qk_args(cls, **kw), *ws, 0) == status


def _cache(**kw):
    c = C.hstu_cache_desc()
    c.struct_size = ctypes.sizeof(c)
    c.H, c.d, c.page_size, c.num_pages, c.max_pages, c.pages, c.timestamps = 4, 64, 64, 10, 3, PTR, PTR
    return _set(c, kw)


@pytest.mark.parametrize("kw,status", [
    (dict(struct_size=4), BAD), (dict(H=0), BAD), (dict(num_pages=0), BAD), (dict(max_pages=0), BAD), (dict(k_exp=33), BAD),
    (dict(v_exp=-33), BAD), (dict(d=32), NOT), (dict(page_size=16), NOT), (dict(page_size=96), NOT), (dict(H=33), NOT),
    (dict(max_pages=(1 << 24) + 1), NOT),
])
def test_cache_descriptions(kw, status):
    c = _cache(**kw)
    assert _status(C.hstu_cache_bytes, c) == status
    assert _status(C.hstu_cache_append, c, _append(), PTR, 256, 0) == status
    assert _status(C.hstu_cache_read, c, _read(), PTR, 256, 0) == status
    assert _status(C.hstu_attn_fwd_cached, _attn(), c, _cached(), PTR, 1 << 30, 0) == status


def test_bytes_of_pages():
    assert C.hstu_cache_bytes(_cache()) == (4 * 64 * 2 * 36, 10 * 4 * 64 * 2 * 36)
    # a size that passes 32 bits
    assert C.hstu_cache_bytes(_cache(H=16, d=128, num_pages=1 << 20, page_size=128))[1] == (1 << 20) * 16 * 128 * 2 * 72


def _append(**kw):
    a = C.hstu_cache_append_args()
    for name in ("seq_offsets", "cache_lens", "block_table", "token_times", "cos", "sin", "k_gain", "k", "v"):
        setattr(a, name, PTR)
    a.B, a.rot_dim, a.norm, a.eps, a.total_tokens, a.max_position = 2, 64, 1, 1e-6, 10, 1000
    _set(a, dict(k_strides=(256, 64), v_strides=(256, 64)))
    return _set(a, kw)


def _read(**kw):
    a = C.hstu_cache_read_args()
    for name in ("seq_offsets", "starts", "block_table", "k", "v", "token_times"):
        setattr(a, name, PTR)
    a.B, a.total_tokens = 2, 10
    return _set(a, kw)


@pytest.mark.parametrize("cache,kw,ws,status", [
    ({}, dict(B=-1), (PTR, 256), BAD), ({}, dict(total_tokens=-1), (PTR, 256), BAD), ({}, dict(reserved=1), (PTR, 256), BAD),
    ({}, dict(interleaved=2), (PTR, 256), BAD), ({}, dict(norm=3), (PTR, 256), BAD), ({}, dict(eps=-1.0), (PTR, 256), BAD),
    ({}, dict(norm=0), (PTR, 256), BAD), ({}, dict(rot_dim=72), (PTR, 256), BAD), ({}, dict(rot_dim=12), (PTR, 256), NOT),
    ({}, dict(max_position=0), (PTR, 256), BAD), ({}, dict(total_tokens=(1 << 30) + 1), (PTR, 256), NOT),
    ({}, dict(seq_offsets=None), (PTR, 256), BAD), ({}, dict(cache_lens=None), (PTR, 256), BAD),
    ({}, dict(block_table=None), (PTR, 256), BAD), ({}, dict(k=None), (PTR, 256), BAD), ({}, dict(v=None), (PTR, 256), BAD),
    ({}, dict(cos=None), (PTR, 256), BAD), ({}, dict(token_times=None), (PTR, 256), BAD),
    (dict(timestamps=None), {}, (PTR, 256), BAD), (dict(pages=None), {}, (PTR, 256), BAD),
    (dict(pages=PTR + 8), {}, (PTR, 256), BAD), (dict(timestamps=PTR + 8), {}, (PTR, 256), BAD),
    ({}, dict(k=PTR + 8), (PTR, 256), BAD), ({}, dict(k_gain=PTR + 4), (PTR, 256), BAD),
    ({}, dict(k_strides=(256, 4)), (PTR, 256), BAD), ({}, dict(v_strides=(-12, 64)), (PTR, 256), BAD),
    ({}, {}, (None, 256), WS), ({}, {}, (PTR + 128, 512), WS), ({}, {}, (PTR, 128), WS),
])
def test_append_calls(cache, kw, ws, status):
    assert _status(C.hstu_cache_append, _cache(**cache), _append(**kw), *ws, 0) == status


@pytest.mark.parametrize("cache,kw,ws,status", [
    ({}, dict(B=-1), (PTR, 256), BAD), ({}, dict(total_tokens=-1), (PTR, 256), BAD), ({}, dict(reserved=1), (PTR, 256), BAD),
    ({}, dict(total_tokens=(1 << 30) + 1), (PTR, 256), NOT), ({}, dict(seq_offsets=None), (PTR, 256), BAD),
    ({}, dict(block_table=None), (PTR, 256), BAD), (dict(timestamps=None), {}, (PTR, 256), BAD),
    ({}, dict(k=PTR + 8), (PTR, 256), BAD), ({}, dict(v=PTR + 2), (PTR, 256), BAD), (dict(pages=None), {}, (PTR, 256), BAD),
    ({}, {}, (None, 256), WS), ({}, {}, (PTR + 128, 512), WS), ({}, {}, (PTR, 128), WS),
])
def test_read_calls(cache, kw, ws, status):
    assert _status(C.hstu_cache_read, _cache(**cache), _read(**kw), *ws, 0) == status


def _attn(**kw):
    base = dict(dtype="bf16", out_dtype="bf16", B=3, H=4, d_qk=64, d_v=64, total_tokens=50, max_seq_len=300, alpha=0.1)
    return C.make_desc(**{**base, **kw})


def _cached(**kw):
    a = C.hstu_attn_cached_args()
    for name, _ in a._fields_:
        if name not in ("max_rows", "reserved"):
            setattr(a, name, PTR)
    a.max_rows = 20
    return _set(a, kw)


@pytest.mark.parametrize("attn,cache,kw,status", [
    (dict(dtype="fp16"), {}, {}, NOT), (dict(out_dtype="fp32"), {}, {}, NOT), (dict(dropout_p=0.1), {}, {}, NOT),
    (dict(H=2), {}, {}, BAD), (dict(d_qk=128, d_v=128), {}, {}, BAD), (dict(flags=C.HSTU_FLAG_FORCE_SIMT), {}, {}, BAD),
    (dict(B=-1), {}, {}, BAD), (dict(total_tokens=(1 << 30) + 1), {}, {}, NOT),
    (dict(total_tokens=1 << 29, max_seq_len=10000), {}, {}, NOT),       # more tiles than 32 bits count
    ({}, {}, dict(max_rows=0), BAD), ({}, {}, dict(reserved=1), BAD), ({}, {}, dict(seq_offsets=None), BAD),
    ({}, {}, dict(cache_lens=None), BAD), ({}, {}, dict(block_table=None), BAD), ({}, {}, dict(q=None), BAD),
    ({}, {}, dict(k=None), BAD), ({}, {}, dict(v=None), BAD), ({}, dict(timestamps=None), {}, BAD),
    ({}, dict(pages=None), {}, BAD), ({}, {}, dict(q=PTR + 8), BAD), ({}, {}, dict(u=PTR + 8), BAD), ({}, {}, dict(y=PTR + 8), BAD),
])
def test_attention_calls(attn, cache, kw, status):
    assert _status(C.hstu_attn_fwd_cached, _attn(**attn), _cache(**cache), _cached(**kw), PTR, 1 << 40, 0) == status


def test_attention_workspaces():
    need = C.hstu_attn_cached_workspace_size(_attn(), _cache(), 20)
    assert need > 256
    for at, size in ((None, need), (PTR + 64, need + 256), (PTR, need - 1)):
        assert _status(C.hstu_attn_fwd_cached, _attn(), _cache(), _cached(), at, size, 0) == WS
    # wider blocks hold no less; no rows at all need little and do nothing
    sizes = [C.hstu_attn_cached_workspace_size(_attn(), _cache(), n) for n in (8, 32, 64, 128, 1000)]
    assert sizes == sorted(sizes)
    none = _attn(total_tokens=0)
    assert _status(C.hstu_attn_fwd_cached, none, _cache(), _cached(), PTR, need, 0) == 0
    assert C.hstu_last_launch_count() == 0


# ------------------------------------------------------------------ Python
torch = pytest.importorskip("torch")

from hstu_jagged_attention_02_gb300.cache import AppendProblem, CachedProblem, PagedCache, ReadProblem  # noqa: E402
from hstu_jagged_attention_02_gb300.qk import QKProblem, jagged_positions, rope_tables  # noqa: E402

i32, i64, bf16 = torch.int32, torch.int64, torch.bfloat16


def _host(**kw):
    return PagedCache(6, **{**dict(H=2, d=64, device="cpu"), **kw})


def test_paged_cache():
    c = _host()
    assert c.pages.shape == (6, 2, 64 * 2 * 36) and c.timestamps.shape == (6, 64)
    assert PagedCache(H=2, d=64, pages=c.pages).num_pages == 6
    assert _host(timestamps=False).timestamps is None
    for kw in (dict(pages=c.pages, num_pages=5), dict(pages=c.pages.float()), dict(pages=c.pages[:, :1]),
               dict(pages=c.pages, page_size=32), dict(), dict(pages=c.pages, timestamps=torch.zeros(6, 32, dtype=i64))):
        with pytest.raises(ValueError):
            PagedCache(**{**dict(H=2, d=64), **kw})


def _batch():
    return dict(k=torch.zeros(3, 2, 64, dtype=bf16), v=torch.zeros(3, 2, 64, dtype=bf16),
                seq_offsets=torch.tensor([0, 1, 3]), cache_lens=torch.tensor([5, 2], dtype=i32),
                block_table=torch.zeros(2, 1, dtype=i32), timestamps=torch.zeros(3, dtype=i64))


@pytest.mark.parametrize("kw", [
    dict(k=torch.zeros(3, 2, 64)), dict(v=torch.zeros(2, 2, 64, dtype=bf16)), dict(k=torch.zeros(3, 1, 64, dtype=bf16)),
    dict(seq_offsets=torch.tensor([0, 1, 3], dtype=i32)), dict(cache_lens=torch.tensor([5, 2])),
    dict(cache_lens=torch.tensor([5], dtype=i32)), dict(block_table=torch.zeros(2, 0, dtype=i32)),
    dict(block_table=torch.zeros(1, 2, dtype=i32)), dict(block_table=torch.zeros(4, 2, dtype=i32)[::2, :1]),
    dict(timestamps=None), dict(timestamps=torch.zeros(4, dtype=i64)), dict(cos=torch.zeros(9, 16)),
    dict(cos=torch.zeros(9, 16), sin=torch.zeros(9, 8)), dict(k_gain=torch.ones(64)), dict(norm=True, k_gain=torch.ones(32)),
    dict(workspace=torch.zeros(256)), dict(workspace=torch.zeros(1, dtype=torch.uint8).expand(256)),
    {},                                                                # all in order, but on the host
])
def test_append_tensors(kw):
    with pytest.raises(ValueError):
        AppendProblem(_host(), **{**_batch(), **kw})


def test_read_tensors():
    b = _batch()
    for off, starts, table in ((b["seq_offsets"].int(), None, b["block_table"]), (b["seq_offsets"], b["cache_lens"].long(), b["block_table"]),
                               (b["seq_offsets"], None, b["block_table"].long()), (b["seq_offsets"], None, b["block_table"])):
        with pytest.raises(ValueError):
            ReadProblem(_host(), off, starts, table)


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(3, 2, 64)), dict(q=torch.zeros(3, 4, 64, dtype=bf16)), dict(u=torch.zeros(3, 64, dtype=bf16)),
    dict(num_targets=torch.zeros(2)), dict(num_targets=torch.zeros(3, dtype=i32)),
    dict(num_targets=torch.zeros(2, dtype=i32), k=None), dict(timestamps=torch.zeros(2, dtype=i64)),
    dict(rab_pos=torch.zeros(1, 128)), dict(rab_time=torch.zeros(2, 64, dtype=torch.float64)), {},
])
def test_attention_tensors(kw):
    b = _batch()
    b.update(q=torch.zeros(3, 2, 64, dtype=bf16), u=None, max_rows=2, max_seq_len=100, alpha=0.1)
    with pytest.raises(ValueError):
        CachedProblem(_host(), **{**b, **kw})


def test_row_times_need_the_caches():
    b = _batch()
    b.update(q=torch.zeros(3, 2, 64, dtype=bf16), u=None, max_rows=2, max_seq_len=100, alpha=0.1)
    with pytest.raises(ValueError, match="need the cache's"):
        CachedProblem(_host(timestamps=False), **b)


@pytest.mark.parametrize("kw", [
    dict(q=None, k=None), dict(q=torch.zeros(5, 2, 64).half()), dict(k=torch.zeros(5, 2, 64, dtype=bf16)),
    dict(k=torch.zeros(4, 2, 64)), dict(positions=None), dict(positions=torch.zeros(5, dtype=i64)), dict(sin=torch.zeros(9, 8)),
    dict(q_gain=torch.ones(32)), dict(norm=False, q_gain=torch.ones(64)), dict(num_tokens=torch.zeros(1, dtype=i32)),
    dict(q_out=torch.zeros(5, 1, 64).expand(5, 2, 64)), dict(dq_out=torch.zeros(5, 2, 64)),
    dict(workspace=torch.zeros(1 << 20)), {},
])
def test_qk_tensors(kw):
    base = dict(q=torch.zeros(5, 2, 64), k=torch.zeros(5, 2, 64), positions=torch.zeros(5, dtype=i32), cos=torch.zeros(9, 16),
                sin=torch.zeros(9, 16))
    with pytest.raises(ValueError):
        QKProblem(**{**base, **kw})


def test_tables_and_positions():
    cos, sin = rope_tables(5, 8, device="cpu")
    ang = torch.arange(5, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(4, dtype=torch.float64) / 4)
    assert torch.equal(cos, ang.cos().float()) and torch.equal(sin, ang.sin().float())
    for bad in ((0, 8), (5, 7), (5, 0)):
        with pytest.raises(ValueError):
            rope_tables(*bad, device="cpu")
    off = torch.tensor([0, 4, 4, 7])
    assert jagged_positions(off).tolist() == [0, 1, 2, 3, 0, 1, 2]
    assert jagged_positions(off, torch.tensor([2, 0, 3])).tolist() == [0, 1, 2, 2, 0, 0, 0]
    assert jagged_positions(off, None, torch.tensor([10, 5, 20])).tolist() == [10, 11, 12, 13, 20, 21, 22]
