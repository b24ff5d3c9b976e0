"""Products of ragged groups (hstu_group_*) against a plain 64-bit form.

Tolerances: operands are BF16, whose products are exact; the tensor core adds
16 of them and the sum so far at a time, in FP32 where at worst each term loses
what lies below 2^-22 of the largest, so n summands cost (n / 16 + 16) 2^-22 of
the sum of their sizes (a split gradient adds its pieces in FP32, within the same).
y and dx are rounded once more to their type."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import training_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _loss(n):
    return (n / 16 + 16) * 2.0 ** -22


def _inputs(sizes, K, N, seed, behind=0):
    g = torch.Generator().manual_seed(seed)
    T = sum(sizes) + behind
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    off = torch.tensor([0] + list(sizes), dtype=torch.int64).cumsum(0).cuda()
    return rnd(T, K), rnd(len(sizes), K, N), off, rnd(T, N)


def _check(name, got, want, bound):
    got = _f64(got)
    assert got.shape == want.shape, name
    off = np.abs(got - want)
    assert np.all(off <= bound), f"{name}: off by {np.max(off / np.maximum(bound, 1e-300)):.3g} of what it may be"


def _check_all(pr, x, w, off, dy, yt, dxt):
    x, w, dy, o = _f64(x), _f64(w), _f64(dy), off.tolist()
    n, K, N = o[-1], w.shape[1], w.shape[2]
    y, size = R.groups_forward(x, w, o)
    _check("y", pr.y[:n], y[:n], (HALF[yt] * np.abs(y) + _loss(K) * size)[:n])
    (dx, sx), (dw, sw) = R.groups_backward(x, w, o, dy)
    _check("dx", pr.dx[:n], dx[:n], (HALF[dxt] * np.abs(dx) + _loss(N) * sx)[:n])
    _check("dw", pr.dw, dw, _loss(max(b - a for a, b in zip(o, o[1:]))) * sw)


CASES = [
    # sizes, K, N, y, dx
    ((1,), 8, 8, "bf16", "bf16"), ((1, 0, 1), 64, 128, "fp32", "fp32"), ((0, 0), 64, 64, "bf16", "bf16"),
    ((15, 16, 17, 1, 0, 33), 64, 128, "bf16", "fp32"), ((5, 64, 63, 65, 2), 72, 136, "fp32", "bf16"),
    ((127, 128, 129), 128, 256, "bf16", "bf16"), ((255, 1, 256, 257), 200, 264, "bf16", "bf16"),
    ((8, 8, 7, 9, 6, 10, 8, 8), 512, 2048, "bf16", "bf16"), ((700, 3, 0, 41), 264, 520, "fp32", "fp32"),
    ((300,), 512, 512, "bf16", "fp32"), ((31, 900, 12, 2, 1500, 0, 64), 128, 384, "bf16", "bf16"),
    ((5000, 10), 128, 256, "fp32", "bf16"), ((2, 3000, 4100, 77), 256, 512, "bf16", "bf16"),
    ((40,) * 30, 1032, 72, "bf16", "bf16"), (tuple(range(70)), 40, 24, "bf16", "fp32"),
]


@pytest.mark.parametrize("sizes,K,N,yt,dxt", CASES)
def test_forward_and_backward(sizes, K, N, yt, dxt):
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    x, w, off, dy = _inputs(sizes, K, N, seed=K + N + len(sizes))
    pr = GroupProblem(x, w, off, out_dtype=TYPES[yt], dy=dy, dx_dtype=TYPES[dxt])
    for t in (pr.y, pr.dx, pr.dw):
        t.fill_(float("nan"))
    pr.forward()
    pr.backward()
    assert pr.device_error() == 0
    _check_all(pr, x, w, off, dy, yt, dxt)


@pytest.mark.parametrize("sizes,K,N,yt,dxt", [
    ((1, 0, 20_000, 300, 37, 9_999, 64, 65, 9_000), 512, 512, "bf16", "bf16"),    # rows stay in shared memory (K), stream (N)
    ((30_011, 2), 264, 1032, "fp32", "fp32"), ((12_345, 23_456), 1096, 640, "bf16", "fp32"),
    ((700,) * 40, 320, 2048, "bf16", "bf16"), ((40_000,), 64, 768, "fp32", "bf16"),
    (tuple(200 + 37 * i for i in range(60)), 520, 264, "bf16", "bf16"),
    ((1, 0, 20_000, 300, 37, 9_999, 64, 65, 9_000), 512, 2048, "fp32", "bf16"), ((40_001,), 512, 1024, "bf16", "bf16"),
])
def test_large_batches(sizes, K, N, yt, dxt):
    """CTAs in pairs, groups cut into pieces; compared on the GPU in 64 bits."""
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    x, w, off, dy = _inputs(sizes, K, N, seed=K + N + len(sizes))
    pr = GroupProblem(x, w, off, out_dtype=TYPES[yt], dy=dy, dx_dtype=TYPES[dxt])
    for t in (pr.y, pr.dx, pr.dw):
        t.fill_(float("nan"))
    pr.forward()
    pr.backward()
    assert pr.device_error() == 0
    near = lambda got, want, size, half, n: bool(((got.double() - want).abs() <= half * want.abs() + _loss(n) * size).all())  # noqa: E731
    o = off.tolist()
    for g, (a, b) in enumerate(zip(o, o[1:])):
        xs, ws, gs = x[a:b].double(), w[g].double(), dy[a:b].double()
        assert near(pr.y[a:b], xs @ ws, xs.abs() @ ws.abs(), HALF[yt], K), (g, "y")
        assert near(pr.dx[a:b], gs @ ws.T, gs.abs() @ ws.abs().T, HALF[dxt], N), (g, "dx")
        assert near(pr.dw[g], xs.T @ gs, xs.abs().T @ gs.abs(), 2.0 ** -24, b - a), (g, "dw")
    first = [t.clone() for t in (pr.y, pr.dx, pr.dw)]
    for _ in range(3):
        pr.forward()
        pr.backward()
    assert all(torch.equal(t, f) for t, f in zip((pr.y, pr.dx, pr.dw), first))


def test_many_groups():
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    rng = np.random.default_rng(1)
    for E in (321, 4096):
        sizes = rng.integers(0, 4, E).tolist()
        x, w, off, dy = _inputs(sizes, 16, 24, seed=E)
        pr = GroupProblem(x, w, off, dy=dy)
        pr.dw.fill_(float("nan"))
        pr.forward()
        pr.backward()
        assert pr.device_error() == 0
        _check_all(pr, x, w, off, dy, "bf16", "bf16")


def test_neighbours_and_rows_behind():
    """Infinities and NaN in other groups' rows and weights, and behind the last group, reach nothing."""
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    sizes, K, N = (37, 70, 5, 130), 72, 136
    x, w, off, dy = _inputs(sizes, K, N, seed=5, behind=40)
    ref = GroupProblem(x, w, off, dy=dy)
    ref.forward()
    ref.backward()
    x2, w2, dy2 = x.clone(), w.clone(), dy.clone()
    x2[37:107], dy2[37:107] = float("nan"), float("inf")
    x2[242:], dy2[242:] = float("inf"), float("nan")
    w2[1] = float("nan")
    pr = GroupProblem(x2, w2, off, dy=dy2)
    for t in (pr.y, pr.dx):
        t.fill_(7.0)
    pr.forward()
    pr.backward()
    assert pr.device_error() == 0
    keep = torch.tensor([i for i in range(242) if not 37 <= i < 107], device="cuda")
    assert torch.equal(pr.y[keep], ref.y[keep]) and torch.equal(pr.dx[keep], ref.dx[keep])
    assert bool((pr.y[242:] == 7).all()) and bool((pr.dx[242:] == 7).all())
    for g in (0, 2, 3):
        assert torch.equal(pr.dw[g], ref.dw[g])


def test_strides_and_copies():
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    sizes, K, N = (50, 0, 33), 72, 48
    x, w, off, dy = _inputs(sizes, K, N, seed=6)
    ref = GroupProblem(x, w, off, dy=dy)
    ref.forward()
    ref.backward()
    wide = lambda t, pad, at: torch.full((83, t.shape[1] + pad), 3.0, dtype=t.dtype, device="cuda")[:, at:at + t.shape[1]].copy_(t)  # noqa: E731
    xs, gs, ys, ds = wide(x, 24, 8), wide(dy, 8, 0), wide(dy, 16, 16), wide(x, 40, 32)
    pr = GroupProblem(xs, w, off, dy=gs, y=ys, dx=ds)
    assert pr.x is xs and pr.dy is gs
    pr.forward()
    pr.backward()
    assert torch.equal(ys, ref.y) and torch.equal(ds, ref.dx) and torch.equal(pr.dw, ref.dw)
    assert bool((ys._base[:, :16] == 3).all()) and bool((ds._base[:, :32] == 3).all()) and bool((ds._base[:, 104:] == 3).all())
    # rows that are not 16 bytes apart, or not aligned, are copied
    odd = GroupProblem(wide(x, 3, 1), w, off, dy=wide(dy, 5, 2))
    odd.forward()
    odd.backward()
    assert torch.equal(odd.y, ref.y) and torch.equal(odd.dx, ref.dx) and torch.equal(odd.dw, ref.dw)
    # one gradient alone
    a, b = GroupProblem(x, w, off, dy=dy, want_dw=False), GroupProblem(x, w, off, dy=dy, want_dx=False)
    a.backward()
    b.backward()
    assert a.dw is None and b.dx is None and torch.equal(a.dx, ref.dx) and torch.equal(b.dw, ref.dw)


def test_offsets_out_of_order_are_reported():
    from hstu_jagged_attention_02_gb300 import binding as C
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    x, w, _, dy = _inputs((30, 30, 4), 64, 64, seed=7)
    for bad in ([0, 40, 30, 64], [1, 30, 60, 64], [0, 30, 60, 65], [-1, 0, 3, 4], [0, 1 << 40, 60, 64], [0, 30, 60, -4]):
        pr = GroupProblem(x, w, torch.tensor(bad, device="cuda"), dy=dy)
        for t in (pr.y, pr.dx, pr.dw):
            t.fill_(7.0)
        pr.forward()
        assert pr.device_error() == C.HSTU_ERR_DEVICE_CHECK, bad
        pr.ws[:256].zero_()
        pr.backward()
        assert pr.device_error() == C.HSTU_ERR_DEVICE_CHECK, bad
        assert all(bool((t == 7).all()) for t in (pr.y, pr.dx, pr.dw))


def test_batches_of_no_rows():
    from hstu_jagged_attention_02_gb300.groups import GroupProblem, hstu_group_linear
    x, w, off, dy = _inputs((0, 0, 0), 64, 72, seed=8)
    pr = GroupProblem(x, w, off, dy=dy)
    pr.dw.fill_(3.0)
    pr.forward()
    pr.backward()
    assert pr.y.shape == (0, 72) and pr.dx.shape == (0, 64) and not pr.dw.any()
    assert hstu_group_linear(x, w, off).shape == (0, 72)


def test_same_bits_and_graphs():
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    x, w, off, dy = _inputs((900, 4000, 30, 2500), 256, 512, seed=9)
    pr = GroupProblem(x, w, off, dy=dy)
    pr.forward()
    pr.backward()
    outs = (pr.y, pr.dx, pr.dw)
    first = [t.clone() for t in outs]
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            pr.forward()
            pr.backward()
    for t in outs:
        t.fill_(float("nan"))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, first))
    # other sizes on the same buffers: the graph reads the offsets
    off.copy_(torch.tensor([0, 2000, 2000, 5000, 7400]))
    graph.replay()
    torch.cuda.synchronize()
    assert pr.device_error() == 0
    _check_all(pr, x, w, off, dy, "bf16", "bf16")


def test_autograd_with_rows_in_any_order():
    from hstu_jagged_attention_02_gb300.groups import GroupProblem, group_rows, hstu_group_linear
    g = torch.Generator().manual_seed(10)
    kind = torch.randint(0, 5, (400,), generator=g).cuda()
    x, w, _, dy = _inputs((400, 0, 0, 0, 0), 64, 128, seed=11)
    order, off = group_rows(kind, 5)
    assert off.tolist() == [0] + torch.bincount(kind, minlength=5).cumsum(0).tolist()
    xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
    y = hstu_group_linear(xl[order], wl, off, out_dtype=torch.float32)
    back = torch.empty_like(y).index_copy(0, order, y)
    back.backward(dy.float())
    pr = GroupProblem(x[order], w, off, out_dtype=torch.float32, dy=dy[order])
    pr.forward()
    pr.backward()
    assert torch.equal(y, pr.y) and torch.equal(xl.grad[order], pr.dx) and torch.equal(wl.grad, pr.dw.bfloat16())
    for e in range(5):
        want = x[kind == e].double() @ w[e].double()
        assert torch.allclose(back[kind == e].double(), want, rtol=0, atol=1e-3)


def test_a_wait_that_runs_out_ends_the_call():
    from hstu_jagged_attention_02_gb300 import binding as C
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    x, w, off, _ = _inputs((100, 30), 128, 256, seed=12)
    pr = GroupProblem(x, w, off, flags=C.HSTU_FLAG_TEST_TIMEOUT)
    pr.forward()
    assert pr.device_error() == C.HSTU_ERR_TIMEOUT
    again = GroupProblem(x, w, off)
    again.forward()
    assert again.device_error() == 0
    want = torch.cat([x[:100].double() @ w[0].double(), x[100:].double() @ w[1].double()])
    assert torch.allclose(again.y.double(), want, rtol=2.0 ** -8, atol=1e-3)


@pytest.mark.parametrize("sizes,K,N", [
    ((257, 0, 12_000, 63), 1024, 1096), ((4_000, 9_000), 1032, 1024), ((6_000, 6_100, 1), 960, 1088),   # pairs
    ((257, 0, 6_000, 63), 256, 264), ((9_000, 1), 264, 256),
    ((200, 7, 64), 192, 72), ((200, 7, 64), 72, 192), ((1, 90, 33), 64, 320),
])
def test_columns_of_wider_tensors(sizes, K, N):
    """Operands and results with other data (NaN) beside their columns; widths that come in one copy and that do not."""
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    x0, w, off, dy0 = _inputs(sizes, K, N, seed=K + 3 * N)
    T = x0.shape[0]
    wide = lambda n, at, dt=torch.bfloat16: torch.full((T, n + 200), float("nan"), device="cuda", dtype=dt)[:, at:at + n]  # noqa: E731
    x, dy, y, dx = wide(K, 64), wide(N, 8), wide(N, 128), wide(K, 16, torch.float32)
    x.copy_(x0)
    dy.copy_(dy0)
    pr = GroupProblem(x, w, off, dy=dy, y=y, dx=dx)
    assert pr.x is x and pr.dy is dy and pr.y is y and pr.dx is dx
    pr.forward()
    pr.backward()
    assert pr.device_error() == 0
    ref = GroupProblem(x0, w, off, dy=dy0, dx_dtype=torch.float32)
    ref.forward()
    ref.backward()
    assert torch.equal(y, ref.y) and torch.equal(dx, ref.dx) and torch.equal(pr.dw, ref.dw)
    assert bool(torch.isnan(y._base[:, :128]).all()) and bool(torch.isnan(dx._base[:, K + 16:]).all())
    _check_all(ref, x0, w, off, dy0, "bf16", "fp32")
