"""The attention over the paged 4-bit cache against the plain 64-bit form on
the values that the cache holds.  The bounds (tests/serving_ref.py) are worst
cases: one FP16 rounding of each score, FP32 sums, one last rounding to BF16."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from hstu_jagged_attention_02_gb300 import binding as C  # noqa: E402
from tests import serving_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu

P, TB = 128, 64


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


class Serve:
    """hist newest tokens (already appended) and cand candidates of each
    sequence over cached tokens (the newest among them)."""

    def __init__(self, cached, hist, cand, H, d, page, seed, *, times="own", P=P, TB=TB, exps=(0, 0), wide=False,
                 bias=0.3, max_pages=None):
        from hstu_jagged_attention_02_gb300.cache import PagedCache, hstu_cache_append, hstu_cache_read
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.cached, self.hist, self.cand, self.H, self.d = cached, hist, cand, H, d
        B, total = len(cached), sum(cached)
        need = [-(-n // page) for n in cached]
        order = torch.randperm(sum(need) + 2, generator=g).int()
        table, at = torch.full((B, max_pages or max(max(need), 1)), -3, dtype=torch.int32), 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table.cuda()
        self.cache = PagedCache(sum(need) + 2, H=H, d=d, page_size=page, k_exp=exps[0], v_exp=exps[1], timestamps=times is not None)
        # pages and places of nobody hold NaN scales
        self.cache.pages.fill_(0x7F)
        self.lens = torch.tensor(cached, dtype=torch.int32).cuda()
        coff = torch.tensor([0] + cached).cumsum(0).cuda()
        k, v = (rnd(total, H, d).mul_(2.0 ** e).bfloat16().cuda() for e in exps)
        gaps = torch.randint(0, 1200, (total,), generator=g)
        if wide:
            gaps = gaps * 3_000_000
        when = (1_700_000_000 + gaps.cumsum(0)).cuda()
        hstu_cache_append(self.cache, k, v, coff, self.lens, self.table, timestamps=when if times is not None else None)
        kc, vc, _ = hstu_cache_read(self.cache, coff, None, self.table)
        self.kc, self.vc, self.tc, self.coff = _f64(kc), _f64(vc), when.cpu().numpy(), coff.tolist()
        n = [a + b for a, b in zip(hist, cand)]
        self.T, self.n = sum(n), n
        self.off = torch.tensor([0] + n).cumsum(0).cuda()
        self.q, self.k, self.v = (rnd(self.T, H, d).bfloat16().cuda() for _ in range(3))
        self.u = rnd(self.T, H * d).bfloat16().cuda()
        self.nt = torch.tensor(cand, dtype=torch.int32).cuda()
        self.rab_pos, self.rab_time = (bias * rnd(H, P)).cuda(), (bias * rnd(H, TB)).cuda()
        rows = []
        for b in range(B):
            t = self.tc[self.coff[b]:self.coff[b + 1]]
            last = int(t[-1]) if len(t) else 1_700_000_000
            rows += [int(x) for x in t[len(t) - hist[b]:]] if hist[b] else []
            extra = torch.randint(0, 10 ** 5, (cand[b],), generator=g).tolist() if times == "own" else [777] * cand[b]
            rows += [last + e for e in extra]
        self.times = torch.tensor(rows, dtype=torch.int64).cuda() if times is not None else None
        self.N = max(max(a + b for a, b in zip(cached, cand)), 1)

    def problem(self, **kw):
        from hstu_jagged_attention_02_gb300.cache import CachedProblem
        a = dict(max_rows=max(max(self.n), 1), max_seq_len=self.N, alpha=self.d ** -0.5, num_targets=self.nt,
                 timestamps=self.times, rab_pos=self.rab_pos, rab_time=self.rab_time)
        a.update(kw)
        return CachedProblem(self.cache, self.q, self.k, self.v, a.pop("u", self.u), self.off, self.lens, self.table, **a)

    def check(self, pr, u="same", rab_pos="same", rab_time="same", norm="layernorm", N=None, alpha=None):
        pick = lambda x, y: y if isinstance(x, str) else x  # noqa: E731
        u, rp, rt = _f64(pick(u, self.u)), _f64(pick(rab_pos, self.rab_pos)), _f64(pick(rab_time, self.rab_time))
        off, o, y = self.off.tolist(), _f64(pr.o), _f64(pr.y)
        t = None if self.times is None else self.times.cpu().numpy()
        for b in range(len(self.cached)):
            r, c = slice(off[b], off[b + 1]), slice(self.coff[b], self.coff[b + 1])
            if r.start == r.stop:
                continue
            wo, wy, bo, by = R.attention(
                _f64(self.q[r]), _f64(self.k[r]), _f64(self.v[r]), None if u is None else u[r], self.kc[c], self.vc[c],
                None if t is None else t[r], self.tc[c], self.cand[b], float(np.float32(alpha or self.d ** -0.5)), rp, rt,
                N or self.N, norm == "layernorm", float(np.float32(1e-5)))
            for name, got, want, bound in (("o", o[r], wo, bo), ("y", y[r], wy, by)):
                off_by = np.abs(got - want)
                assert np.all(off_by <= bound), f"{name} of {b}: {np.max(off_by / bound):.3g} of what it may be off"


CASES = [
    # cached, hist, cand, H, d, page, times
    ([1], [1], [0], 1, 128, 64, "own"),
    ([300], [1], [0], 4, 128, 64, "own"),
    ([0], [0], [1], 2, 64, 32, "own"),
    ([0, 3], [0, 0], [5, 2], 2, 128, 32, "request"),
    ([128, 129, 127, 0, 700], [1, 1, 1, 0, 1], [0, 0, 0, 0, 0], 2, 128, 32, "own"),
    ([500, 0, 131, 64], [0, 0, 0, 0], [17, 3, 0, 128], 2, 128, 64, "request"),
    ([260, 700], [0, 0], [150, 300], 2, 64, 128, "own"),
    ([90, 333, 12], [9, 0, 12], [5, 23, 0], 3, 64, 32, "request"),
    ([200, 45], [200, 45], [0, 0], 2, 128, 64, "own"),
    ([390, 10], [390, 10], [20, 0], 1, 64, 32, "own"),
    ([1000, 513], [40, 33], [30, 31], 2, 128, 128, "own"),
    ([5000], [2], [1], 1, 128, 64, "own"),
    ([63, 64, 65], [1, 2, 3], [1, 1, 1], 2, 64, 64, None),
]


@pytest.mark.parametrize("cached,hist,cand,H,d,page,times", CASES)
def test_rows_against_the_definition(cached, hist, cand, H, d, page, times):
    s = Serve(cached, hist, cand, H, d, page, seed=sum(cached) + d, times=times)
    pr = s.problem()
    pr.o.fill_(float("nan"))
    pr.y.fill_(float("nan"))
    pr.forward()
    assert pr.device_error() == 0
    s.check(pr)


def test_wide_time_gaps_and_other_tables():
    s = Serve([700, 260], [5, 0], [4, 60], 2, 128, 64, seed=31, wide=True, P=17, TB=9, bias=2.0, exps=(-2, 3))
    pr = s.problem()
    pr.forward()
    assert pr.device_error() == 0
    s.check(pr)


@pytest.mark.parametrize("drop", ["u", "rab_pos", "rab_time", "norm"])
def test_parts_left_out(drop):
    s = Serve([150, 20], [3, 0], [10, 6], 2, 64, 32, seed=32)
    kw = {"norm": "none"} if drop == "norm" else {drop: None}
    pr = s.problem(**kw)
    pr.forward()
    assert pr.device_error() == 0
    s.check(pr, **kw)


def test_biases_that_mute():
    # the type's lowest value and minus infinity leave pairs out; scores far below zero count as almost nothing
    s = Serve([200], [0], [20], 2, 64, 32, seed=33, times="request")
    s.rab_pos[:, 40:] = torch.finfo(torch.float32).min
    pr = s.problem(rab_time=None)
    pr.forward()
    s.check(pr, rab_time=None)
    s.rab_pos[:, 40:] = float("-inf")
    inf = s.problem(rab_time=None)
    inf.forward()
    assert torch.equal(inf.o, pr.o) and torch.equal(inf.y, pr.y)
    s.rab_pos[:, 40:] = -9.0
    pr = s.problem(rab_time=None)
    pr.forward()
    s.check(pr, rab_time=None)


def test_a_row_that_sees_nothing_and_one_key():
    # no cache and no candidate of its own leaves nothing: a history row always sees itself, a candidate itself
    s = Serve([1, 0], [1, 0], [0, 1], 2, 128, 32, seed=34)
    pr = s.problem()
    pr.forward()
    s.check(pr)


def test_padded_batch_equal_bits_and_graph():
    s = Serve([300, 40], [2, 0], [7, 3], 2, 128, 64, seed=35)
    pr = s.problem()
    pr.forward()
    o, y = pr.o.clone(), pr.y.clone()
    pad = lambda t: torch.cat([t, t.new_zeros(6, *t.shape[1:])])  # noqa: E731
    for n in ("q", "k", "v", "u", "times"):
        setattr(s, n, pad(getattr(s, n)))
    pp = s.problem()
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            pp.forward()
    for _ in range(2):
        pp.o.fill_(5.0)
        pp.y.fill_(6.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pp.o[:s.T], o) and torch.equal(pp.y[:s.T], y)
        assert bool((pp.o[s.T:] == 5.0).all()) and bool((pp.y[s.T:] == 6.0).all())
    assert pp.device_error() == 0


def test_wider_tiles_than_needed_and_two_streams():
    # max_rows only bounds the rows: a larger one gives the definition too; calls on two streams keep to themselves
    s, t = Serve([400, 90], [1, 1], [0, 4], 2, 128, 64, seed=36), Serve([77], [0], [33], 2, 64, 32, seed=37)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a = [s.problem(max_rows=r) for r in (5, 20, 40, 100, 1000)]
    b = t.problem()
    torch.cuda.synchronize()
    for pr in a:
        pr.forward(s1)
        b.forward(s2)
    torch.cuda.synchronize()
    for pr in a:
        s.check(pr)
    t.check(b)


@pytest.mark.parametrize("what", ["page", "lens", "targets", "rows", "length", "offsets"])
def test_batches_that_do_not_fit_are_reported(what):
    s = Serve([100, 200], [3, 0], [5, 9], 2, 64, 32, seed=38)
    kw = {}
    if what == "page":
        s.table[1, 3] = 10 ** 6
    elif what == "lens":
        s.lens[0] = 2                    # fewer cached tokens than new rows
    elif what == "targets":
        s.nt[1] = 10                     # more candidates than rows
    elif what == "rows":
        kw["max_rows"] = 8
    elif what == "length":
        kw["max_seq_len"] = 208
    elif what == "offsets":
        s.off[2] = 18
    pr = s.problem(**kw)
    pr.forward()
    assert pr.device_error() == C.HSTU_ERR_DEVICE_CHECK
    torch.cuda.synchronize()


def test_from_projection_to_scores():
    """The whole serving step: norm and rotate q, append k and v, attend; the
    same numbers as the plain forms one after the other, and as the BF16 delta
    forward on what the cache gives back."""
    from hstu_jagged_attention_02_gb300.cache import PagedCache, hstu_attention_cached, hstu_cache_append, hstu_cache_read
    from hstu_jagged_attention_02_gb300.qk import hstu_qk_norm_rope, jagged_positions, rope_tables
    g = torch.Generator().manual_seed(40)
    H, d, page = 2, 128, 64
    cached, cand = [400, 210], [70, 90]
    N = 500
    cos, sin = rope_tables(600, d)
    gq, gk = ((1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    cache = PagedCache(12, H=H, d=d, page_size=page)
    table = torch.tensor([[3, 1, 4, 11, 5, 9, 2], [6, 0, 8, 7, 10, 0, 0]], dtype=torch.int32).cuda()
    coff, off = (torch.tensor([0] + x).cumsum(0).cuda() for x in (cached, cand))
    lens = torch.tensor(cached, dtype=torch.int32).cuda()
    kv = torch.randn(610, 2 * H, d, generator=g).bfloat16().cuda()
    when = (1_700_000_000 + torch.randint(0, 900, (610,), generator=g).cumsum(0)).cuda()
    # in two steps: all but 10 tokens of each, then those
    first = [a - 10 for a in cached]
    keep = torch.cat([torch.arange(a) + s for a, s in zip(first, coff.tolist())]).cuda()
    rest = torch.cat([torch.arange(10) + s + a for a, s in zip(first, coff.tolist())]).cuda()
    for rows, n, length in ((keep, first, first), (rest, [10, 10], cached)):
        hstu_cache_append(cache, kv[rows][:, :H], kv[rows][:, H:], torch.tensor([0] + n).cumsum(0).cuda(),
                          torch.tensor(length, dtype=torch.int32).cuda(), table, timestamps=when[rows], cos=cos, sin=sin,
                          norm=True, k_gain=gk)
    T = 160
    x = torch.randn(T, 3 * H, d, generator=g).bfloat16().cuda()
    u = torch.randn(T, H * d, generator=g).bfloat16().cuda()
    nt = torch.tensor(cand, dtype=torch.int32).cuda()
    pos = jagged_positions(off, nt, starts=lens)
    assert pos.tolist() == [400] * 70 + [210] * 90
    q, k = hstu_qk_norm_rope(x[:, :H], x[:, H:2 * H], pos, cos, sin, q_gain=gq, k_gain=gk)
    v = x[:, 2 * H:].contiguous()
    t_rows = torch.cat([when[399].repeat(70) + 60, when[609].repeat(90) + 60])
    rp, rt = (0.1 * torch.randn(H, n, generator=g).cuda() for n in (P, TB))
    o, y = hstu_attention_cached(cache, q, k, v, u, off, lens, table, max_rows=90, max_seq_len=N, alpha=d ** -0.5,
                                 num_targets=nt, timestamps=t_rows, rab_pos=rp, rab_time=rt)
    kc, vc, tc = hstu_cache_read(cache, coff, None, table)
    assert torch.equal(tc, when)
    c, s = (z.cpu().numpy()[np.concatenate([np.arange(a) for a in cached])] for z in (cos, sin))
    want_k = R.qk_forward(_f64(kv[:, :H]), _f64(gk), c, s, False, True, float(np.float32(1e-6)))
    np.testing.assert_array_equal(_f64(kc), R.four_bit(want_k))
    for b in range(2):
        r, cc = slice(off[b], off[b + 1]), slice(coff[b], coff[b + 1])
        wo, wy, bo, by = R.attention(_f64(q[r]), _f64(k[r]), _f64(v[r]), _f64(u[r]), _f64(kc[cc]), _f64(vc[cc]),
                                     t_rows[r].cpu().numpy(), tc[cc].cpu().numpy(), cand[b], float(np.float32(d ** -0.5)),
                                     _f64(rp), _f64(rt), N, True, float(np.float32(1e-5)))
        assert np.all(np.abs(_f64(o[r]) - wo) <= bo) and np.all(np.abs(_f64(y[r]) - wy) <= by)
    # the delta forward on the packed values (its own bar: 1e-2 of the output's RMS, plus this one's BF16 rounding)
    desc = C.make_desc(dtype="bf16", out_dtype="fp32", B=2, H=H, d_qk=d, d_v=d, total_tokens=T, max_seq_len=N, alpha=d ** -0.5)
    ws = torch.empty(C.hstu_attn_workspace_size(desc)[0], dtype=torch.uint8, device="cuda")
    do, dy = torch.empty(T, H, d, device="cuda"), torch.empty(T, H * d, device="cuda")
    args = C.hstu_attn_delta_args(*[z.data_ptr() if torch.is_tensor(z) else z for z in (
        off, coff, 610, t_rows, tc, rp, rt, q, k, v, u, kc, vc, do, dy)], None, None)
    C.hstu_attn_fwd_delta(desc, args, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    for a, b in ((o, do), (y, dy)):
        a, b = _f64(a), _f64(b)
        assert np.max(np.abs(a - b) - 2.0 ** -8 * np.abs(b)) <= 2e-2 * np.sqrt(np.mean(b * b))
