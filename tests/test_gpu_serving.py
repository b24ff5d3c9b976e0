"""The attention over the paged 4-bit cache at its corners: each kernel with
each page size, more sequences than a block has threads, wide rows, pages that
lie beyond 32-bit offsets or belong to two sequences, captured calls side by
side.  The bounds are those of tests/serving_ref.py."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_cached import Serve, _f64  # noqa: E402

pytestmark = pytest.mark.gpu


def _run(s, **kw):
    pr = s.problem(**kw)
    pr.o.fill_(float("nan"))
    pr.y.fill_(float("nan"))
    pr.forward()
    assert pr.device_error() == 0
    return pr


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_every_kernel_with_every_page(page, d):
    s = Serve([300, 0, 70, 513], [2, 0, 0, 5], [3, 4, 0, 2], 3, d, page, seed=page + d)
    for rows in (8, 32, 64, 128):
        s.check(_run(s, max_rows=rows))


@pytest.mark.parametrize("rows", [4, 20])
def test_more_sequences_than_threads(rows):
    g = torch.Generator().manual_seed(50)
    n = 2000
    cached = torch.randint(0, 90, (n,), generator=g).tolist()
    hist = [min(c, int(h)) for c, h in zip(cached, torch.randint(0, 3, (n,), generator=g))]
    cand = torch.randint(0, 3, (n,), generator=g).tolist()
    cached[1000:1040] = hist[1000:1040] = cand[1000:1040] = [0] * 40        # some with nothing at all
    s = Serve(cached, hist, cand, 2, 64, 32, seed=51)
    s.check(_run(s, max_rows=rows))


@pytest.mark.parametrize("H,d,cached,hist,cand", [
    (16, 128, [150], [1], [0]), (16, 128, [150, 30], [0, 2], [120, 100]), (12, 128, [260], [0], [3]), (32, 64, [200], [2], [1]),
    (9, 128, [140, 20], [3, 20], [170, 0]), (1, 64, [40], [0], [2]),
])
def test_narrow_and_wide_rows(H, d, cached, hist, cand):
    s = Serve(cached, hist, cand, H, d, 32, seed=H + d)
    s.check(_run(s))


def test_one_long_sequence_of_many_pieces():
    s = Serve([20011], [3], [4], 2, 64, 128, seed=52)
    for rows in (7, 30):
        s.check(_run(s, max_rows=rows))


def test_pages_beyond_32_bits():
    """The same tokens in pages whose bytes and times lie beyond 2^32 and in
    pages at the cache's start: the same bits."""
    from hstu_jagged_attention_02_gb300.cache import CachedProblem, PagedCache, hstu_cache_append, hstu_cache_read
    H, d, page = 16, 128, 128
    far = (1 << 32) // (H * page * 2 * 72) + 50
    cache = PagedCache(far + 8, H=H, d=d, page_size=page)
    g = torch.Generator().manual_seed(53)
    rnd = lambda *z: torch.randn(*z, generator=g).bfloat16().cuda()  # noqa: E731
    L, rows = 300, 40
    k, v, q, kr, vr = rnd(L, H, d), rnd(L, H, d), rnd(rows, H, d), rnd(rows, H, d), rnd(rows, H, d)
    off, roff = torch.tensor([0, L]).cuda(), torch.tensor([0, rows]).cuda()
    lens, nt = torch.tensor([L], dtype=torch.int32).cuda(), torch.tensor([rows], dtype=torch.int32).cuda()
    when = torch.arange(L).cuda() * 37 + 10 ** 9
    got = []
    for first in (0, far):
        table = (torch.tensor([[2, 0, 1]], dtype=torch.int32) + first).cuda()
        hstu_cache_append(cache, k, v, off, lens, table, timestamps=when)
        back = hstu_cache_read(cache, off, None, table)
        assert torch.equal(back[2], when)
        outs = []
        for n in (8, rows):
            pr = CachedProblem(cache, q[:n], kr[:n], vr[:n], None, roff.clamp(max=n), lens, table, max_rows=n, max_seq_len=400,
                               alpha=0.1, num_targets=nt.clamp(max=n), timestamps=when[-1:].repeat(n),
                               rab_time=torch.linspace(-1, 1, H * 64).view(H, 64).cuda())
            pr.forward()
            assert pr.device_error() == 0
            outs += [pr.o, pr.y]
        got.append([back[0], back[1]] + outs)
    for a, b in zip(*got):
        assert torch.equal(a, b) and bool(torch.isfinite(a.float()).all())


def test_sequences_that_share_pages():
    s = Serve([200, 200], [0, 0], [6, 6], 2, 128, 64, seed=54, times="request")
    half = s.T // 2
    s.table[1] = s.table[0]
    for name in ("q", "k", "v", "u", "times"):
        x = getattr(s, name)
        x[half:] = x[:half]
    pr = _run(s)
    assert torch.equal(pr.o[:half], pr.o[half:]) and torch.equal(pr.y[:half], pr.y[half:])
    s.kc[200:], s.vc[200:], s.tc[200:] = s.kc[:200], s.vc[:200], s.tc[:200]
    s.check(pr)


def test_captured_step_beside_another():
    """A captured step (norm and rotation, append, read, attention) replayed on
    one stream while another problem with a workspace of its own runs on a
    second: the bits of the eager calls."""
    from hstu_jagged_attention_02_gb300.cache import AppendProblem, ReadProblem
    from hstu_jagged_attention_02_gb300.qk import QKProblem, rope_tables
    s, other = Serve([500, 90], [1, 1], [3, 0], 2, 128, 64, seed=55), Serve([260], [0], [100], 2, 64, 32, seed=56)
    cos, sin = rope_tables(600, 128)
    pos = torch.arange(s.T, dtype=torch.int32).cuda() * 20
    coff = torch.tensor(s.coff).cuda()
    g = torch.Generator().manual_seed(57)
    new = torch.randn(2, 2, 2, 128, generator=g).bfloat16().cuda()          # [k or v, tokens, H, d]
    one = torch.tensor([0, 1, 2]).cuda()
    qk = QKProblem(s.q, s.k, pos, cos, sin)
    ap = AppendProblem(s.cache, new[0], new[1], one, s.lens, s.table, timestamps=s.times[[0, 4]].contiguous(), cos=cos, sin=sin,
                       norm=True)
    rd = ReadProblem(s.cache, coff, None, s.table)
    s.q, s.k = qk.q_out, qk.k_out
    at, beside = s.problem(), other.problem()

    def step():
        qk.forward()
        ap.run()
        rd.run()
        at.forward()
    step()
    beside.forward()
    torch.cuda.synchronize()
    outs = lambda: [x.clone() for x in (qk.q_out, qk.k_out, rd.k, rd.v, rd.timestamps, at.o, at.y)]  # noqa: E731
    want, want_beside = outs(), beside.y.clone()
    graph, s1, s2 = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        with torch.cuda.graph(graph, stream=s1):
            step()
    for _ in range(3):
        for x in (qk.q_out, qk.k_out, rd.k, rd.v, at.o, at.y, beside.y):
            x.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            with torch.cuda.stream(s1):
                graph.replay()
            beside.forward(s2)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs(), want)) and torch.equal(beside.y, want_beside)
    s.kc, s.vc = _f64(rd.k), _f64(rd.v)
    s.tc = rd.timestamps.cpu().numpy()
    s.check(at)


def test_no_second_derivative():
    from hstu_jagged_attention_02_gb300.qk import hstu_qk_norm_rope
    q = torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(58)).cuda().requires_grad_()
    out, _ = hstu_qk_norm_rope(q, None)
    (g,) = torch.autograd.grad(out.square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
