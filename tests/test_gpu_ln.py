"""Layer norm with weight and bias (hstu_ln_*) against a plain 64-bit form.

Tolerances: an output is rounded once (half a step of its type) from FP32
arithmetic.  Sums over a row are at most 32 additions a lane, 5 shuffles and 16
warps, and a product with 1 / D: below 64 roundings of 2^-24, so 2^-18 of the
terms' size; the square root halves it and adds 2^-22, the products 2^-22: 2^-17
in all.  The weight's and the bias's gradients are sums over the rows of a warp
(at most rows / 8 / CTAs), 8 warps, and 304 / 8 + 8 CTAs: at these sizes below
128 roundings, 2^-17 of the sum of their terms' sizes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import training_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
EPS = 1e-5


def _f64(t):
    return t.detach().double().cpu().numpy()


def _inputs(T, D, x, y, seed, weight=True, bias=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    size = 0.1 + 3 * torch.rand(T, 1, generator=g)
    t = (rnd(T, D) * size + rnd(T, 1)).to(TYPES[x]).cuda()
    w, b = (1 + 0.3 * rnd(D)).cuda() if weight else None, (0.2 * rnd(D)).cuda() if bias else None
    return t, w, b, rnd(T, D).to(TYPES[y]).cuda(), rnd(T, D).to(TYPES[x]).cuda()


def _check(name, got, want, bound):
    got = _f64(got)
    assert got.shape == want.shape, name
    off = np.abs(got - want)
    assert np.all(off <= bound), f"{name}: off by {np.max(off / np.maximum(bound, 1e-300)):.3g} of what it may be"


def _check_all(pr, x, w, b, dy, dres, xt, yt):
    x64, w64, b64 = _f64(x), None if w is None else _f64(w), None if b is None else _f64(b)
    y, mean, rstd, size = R.ln_forward(x64, w64, b64, EPS)
    _check("y", pr.y, y, HALF[yt] * np.abs(y) + 2.0 ** -17 * size)
    _check("mean", pr.mean, mean, 2.0 ** -17 * np.abs(x64).mean(-1))
    _check("rstd", pr.rstd, rstd, 2.0 ** -17 * rstd)
    (dx, sx), (dw, sw), (db, sb) = R.ln_backward(x64, w64, _f64(pr.mean), _f64(pr.rstd), _f64(dy))
    if dres is not None:
        dx, sx = dx + _f64(dres), sx + np.abs(_f64(dres))
    _check("dx", pr.dx, dx, HALF[xt] * np.abs(dx) + 2.0 ** -17 * sx)
    if pr.d_weight is not None:
        _check("dw", pr.d_weight, dw, 2.0 ** -17 * sw)
    if pr.d_bias is not None:
        _check("db", pr.d_bias, db, 2.0 ** -17 * sb)


CASES = [
    # rows, D, x, y, weight, bias, dres
    (1, 512, "bf16", "bf16", True, True, False), (1, 1, "fp32", "fp32", True, True, False),
    (3, 2, "bf16", "fp32", True, True, True), (64, 512, "fp32", "bf16", True, True, True),
    (7, 8, "bf16", "bf16", True, True, False), (65, 256, "fp32", "fp32", True, False, False),
    (37, 264, "bf16", "fp32", False, True, True), (33, 301, "fp32", "fp32", True, True, True),
    (50, 130, "bf16", "bf16", True, True, False), (41, 127, "fp32", "bf16", False, False, False),
    (19, 1024, "bf16", "bf16", True, True, True), (20, 1000, "fp32", "fp32", True, True, False),
    (21, 1023, "bf16", "fp32", True, True, True), (9, 1032, "fp32", "bf16", True, True, True),
    (5, 2048, "bf16", "bf16", True, True, False), (6, 2056, "fp32", "fp32", True, True, True),
    (4, 2049, "bf16", "bf16", True, True, True), (3, 5001, "fp32", "fp32", True, True, False),
    (3, 8192, "bf16", "fp32", True, True, True), (4, 8200, "fp32", "bf16", True, True, False),
    (2, 16384, "bf16", "bf16", True, True, True), (2, 16383, "fp32", "fp32", True, True, True),
    (5000, 512, "bf16", "bf16", True, True, False), (5003, 96, "fp32", "bf16", True, True, True),
    (700, 1500, "bf16", "fp32", True, True, False),
]


@pytest.mark.parametrize("T,D,xt,yt,weight,bias,res", CASES)
def test_forward_and_backward(T, D, xt, yt, weight, bias, res):
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    x, w, b, dy, dres = _inputs(T, D, xt, yt, T + D, weight, bias)
    pr = LNProblem(x, w, b, eps=EPS, out_dtype=TYPES[yt], dy=dy, dres=dres if res else None, want_weight_grad=True,
                   want_bias_grad=True)
    for t in (pr.y, pr.mean, pr.rstd, pr.dx, pr.d_weight, pr.d_bias):
        t.fill_(float("nan"))
    pr.forward()
    pr.backward()
    assert pr.device_error() == 0
    _check_all(pr, x, w, b, dy, dres if res else None, xt, yt)


def test_gradients_against_differences():
    rng = np.random.default_rng(4)
    x, w, b, dy = rng.normal(size=(6, 40)), 1 + 0.3 * rng.normal(size=40), rng.normal(size=40), rng.normal(size=(6, 40))
    f = lambda x, w, b: (R.ln_forward(x, w, b, EPS)[0] * dy).sum()  # noqa: E731
    _, mean, rstd, _ = R.ln_forward(x, w, b, EPS)
    grads = [g for g, _ in R.ln_backward(x, w, mean, rstd, dy)]
    for k, (arg, g) in enumerate(zip((x, w, b), grads)):
        for at in list(np.ndindex(arg.shape))[::17]:
            e = np.zeros_like(arg)
            e[at] = 1e-6
            args = [[x, w, b], [x, w, b]]
            args[0][k], args[1][k] = arg + e, arg - e
            assert abs((f(*args[0]) - f(*args[1])) / 2e-6 - g[at]) < 1e-6 * max(1, abs(g[at]))


def test_strides_offsets_and_in_place():
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    x, w, b, dy, dres = _inputs(90, 200, "bf16", "bf16", 8)
    whole = LNProblem(x, w, b, dy=dy, dres=dres)
    whole.forward()
    whole.backward()
    # parts of wider rows, aligned and not (the narrow loads sum in another order)
    for pad, at in ((56, 8), (3, 1), (8, 4)):
        cut = lambda t: torch.full((90, 200 + pad), 9.0, dtype=t.dtype, device="cuda")[:, at:at + 200].copy_(t)  # noqa: E731
        xs, ys, gs, rs, ds = (cut(t) for t in (x, x, dy, dres, x))
        pr = LNProblem(xs, w, b, dy=gs, dres=rs, y=ys, dx=ds)
        assert pr.x is xs and pr.dy is gs
        pr.forward()
        pr.backward()
        _check_all(pr, x, w, b, dy, dres, "bf16", "bf16")
        for t in (ys, ds):
            rows = t._base
            assert bool((rows[:, :at] == 9).all()) and bool((rows[:, at + 200:] == 9).all())
    # features that are not contiguous are copied
    pr = LNProblem(x.t().contiguous().t(), w, b)
    pr.forward()
    assert torch.equal(pr.y, whole.y)
    # in place: y over x, dx over dy
    z, g = x.clone(), dy.clone()
    pr = LNProblem(z, w, b, y=z)
    pr.forward()
    assert torch.equal(z, whole.y)
    pr = LNProblem(x, w, b, dy=g, dx=g, dres=dres, mean=whole.mean, rstd=whole.rstd)
    pr.backward()
    assert torch.equal(g, whole.dx) and torch.equal(pr.d_weight, whole.d_weight)


@pytest.mark.parametrize("D", [64, 301, 1500])
def test_padded_batches(D):
    from hstu_jagged_attention_02_gb300 import binding as C
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    x, w, b, dy, _ = _inputs(90, D, "fp32", "bf16", 12)
    x[53:] = float("nan")
    dy[53:] = float("inf")
    for n in (53, 0, 1):
        pr = LNProblem(x, w, b, dy=dy, num_rows=torch.tensor([n], device="cuda"))
        first = LNProblem(x[:n], w, b, dy=dy[:n])
        for t in (pr.y, pr.dx, pr.mean, pr.rstd):
            t.fill_(7.0)
        for q in (pr, first):
            q.forward()
            q.backward()
        assert pr.device_error() == 0
        for t, f in ((pr.y, first.y), (pr.dx, first.dx), (pr.mean, first.mean), (pr.rstd, first.rstd)):
            assert torch.equal(t[:n], f) and bool((t[n:] == 7).all())
        assert torch.allclose(pr.d_weight, first.d_weight, rtol=1e-5, atol=1e-4)
        assert torch.allclose(pr.d_bias, first.d_bias, rtol=1e-5, atol=1e-4)
        if n == 0:
            assert not pr.d_weight.any() and not pr.d_bias.any()
    for bad in (91, -1):
        pr = LNProblem(x, w, b, dy=dy, num_rows=torch.tensor([bad], device="cuda"))
        pr.y.fill_(7.0)
        pr.forward()
        assert pr.device_error() == C.HSTU_ERR_DEVICE_CHECK and bool((pr.y == 7).all())


def test_rows_keep_to_themselves():
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    x, w, b, dy, _ = _inputs(40, 512, "fp32", "fp32", 13)
    pr = LNProblem(x, w, b)
    pr.forward()
    want = pr.y.clone()
    x[3], x[17, 5], x[20] = float("nan"), float("inf"), 5.0
    pr.forward()
    keep = [i for i in range(40) if i not in (3, 17, 20)]
    assert torch.equal(pr.y[keep], want[keep]) and bool(pr.y[3].isnan().all()) and bool(pr.y[17].isnan().any())
    # a row of equal values has no variance: its output is the bias
    assert torch.equal(pr.y[20], b)


def test_same_bits_and_graphs():
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    x, w, b, dy, _ = _inputs(4000, 512, "bf16", "bf16", 14)
    pr = LNProblem(x, w, b, dy=dy)
    pr.forward()
    pr.backward()
    outs = (pr.y, pr.mean, pr.rstd, pr.dx, pr.d_weight, pr.d_bias)
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
    assert all(torch.equal(a, c) for a, c in zip(outs, first))


def test_autograd_and_broadcast_gradients():
    from hstu_jagged_attention_02_gb300.norm import LNProblem, hstu_ln
    x, w, b, _, _ = _inputs(70, 128, "bf16", "bf16", 15)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    y = hstu_ln(*leaves, out_dtype=torch.float32)
    y.sum().backward()                       # the gradient of y is one number, broadcast
    pr = LNProblem(x, w, b, out_dtype=torch.float32, dy=torch.ones(70, 128, device="cuda"))
    pr.forward()
    pr.backward()
    assert torch.equal(y, pr.y)
    for leaf, g in zip(leaves, (pr.dx, pr.d_weight, pr.d_bias)):
        assert torch.equal(leaf.grad, g)
    y = hstu_ln(leaves[0].detach()[:0], w, b)
    assert y.shape == (0, 128)


@pytest.mark.parametrize("D", [256, 376, 384, 392, 512, 760, 768, 1024, 1528, 1536, 2048, 2152, 3056, 4096, 8192])
def test_sums_of_a_cta_fill_its_shared_memory(D):
    """The backward's sums of the rows a CTA has at a time are 48 KB at 384, 768, 1,536 features: what a launch gets unasked."""
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    x, w, b, dy, dres = _inputs(77, D, "bf16", "bf16", 77 + D)
    pr = LNProblem(x, w, b, eps=EPS, dy=dy, dres=dres)
    pr.forward()
    pr.backward()
    _check_all(pr, x, w, b, dy, dres, "bf16", "bf16")


def test_gradients_in_place():
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    for D in (72, 301, 1500):
        x, w, b, dy, dres = _inputs(50, D, "fp32", "fp32", D)
        ref = LNProblem(x, w, b, eps=EPS, dy=dy, dres=dres)
        ref.forward()
        ref.backward()
        for name in ("dy", "dres"):
            t = dict(dy=dy.clone(), dres=dres.clone())
            pr = LNProblem(x, w, b, eps=EPS, dx=t[name], mean=ref.mean, rstd=ref.rstd, **t)
            pr.backward()
            assert torch.equal(t[name], ref.dx) and torch.equal(pr.d_weight, ref.d_weight) and torch.equal(pr.d_bias, ref.d_bias)
