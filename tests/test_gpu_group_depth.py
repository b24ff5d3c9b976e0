"""Products of groups over long depths.

Operands are positive, so that what the tensor core's sums lose (always towards
zero) adds up and a result is as large as its terms together.  The kernel reads
an accumulator after 1,024 of the depth and adds in FP32: a run of 1,024 takes
64 additions of 16 exact products and one for each of 16 of them, of which each
loses at worst 2^-22 of the run's sum, and n / 1,024 runs are added with half a
step each: (64 + 16) 2^-22 + ceil(n / 1,024) 2^-24 of the result.  One
accumulator for a depth of 65,536 loses some 2,048 x 2^-24 on average, more than
four times that."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _loss(n):
    return 80 * 2.0 ** -22 + -(-n // 1024) * 2.0 ** -24


def _positive(g, *shape):
    return (0.5 + torch.rand(*shape, generator=g)).bfloat16().cuda()


@pytest.mark.parametrize("sizes,K,N,yt,dxt", [
    ((3, 40, 0, 17), 65536, 64, "fp32", "fp32"), ((3, 40, 0, 17), 64, 65536, "fp32", "fp32"),
    ((1,), 16384, 8, "fp32", "bf16"), ((130, 5), 136, 24_000, "bf16", "fp32"), ((2, 300), 8_200, 264, "bf16", "bf16"),
    ((33, 64, 255), 1032, 2056, "fp32", "fp32"), ((31, 97), 1096, 1088, "bf16", "bf16"),
    ((6000, 1, 9_001), 2048, 4096, "fp32", "bf16"), ((257, 12_000), 4168, 1544, "bf16", "fp32"),
])
def test_long_depths(sizes, K, N, yt, dxt):
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    g = torch.Generator().manual_seed(K + N)
    T = sum(sizes)
    x, w, dy = _positive(g, T, K), _positive(g, len(sizes), K, N), _positive(g, T, N)
    off = torch.tensor([0] + list(sizes), dtype=torch.int64).cumsum(0).cuda()
    pr = GroupProblem(x, w, off, out_dtype=TYPES[yt], dy=dy, dx_dtype=TYPES[dxt], want_dw=False)
    pr.y.fill_(float("nan"))
    pr.dx.fill_(float("nan"))
    pr.forward()
    pr.backward()
    assert pr.device_error() == 0
    o = off.tolist()
    for e, (a, b) in enumerate(zip(o, o[1:])):
        if a == b:
            continue
        y, dx = x[a:b].double() @ w[e].double(), dy[a:b].double() @ w[e].double().T
        for name, got, want, n, half in (("y", pr.y[a:b], y, K, HALF[yt]), ("dx", pr.dx[a:b], dx, N, HALF[dxt])):
            worst = float(((got.double() - want).abs() / want).max())
            assert worst <= half + _loss(n), (e, name, worst)
    first = [pr.y.clone(), pr.dx.clone()]
    pr.forward()
    pr.backward()
    assert torch.equal(pr.y, first[0]) and torch.equal(pr.dx, first[1])


def test_signs_and_infinities():
    """Sums of both signs, and an infinity in one run of the depth, which reaches its own row alone."""
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    g = torch.Generator().manual_seed(1)
    K, N, sizes = 5000, 136, (70, 35)
    x, w = (torch.randn(105, K, generator=g).bfloat16().cuda(), torch.randn(2, K, N, generator=g).bfloat16().cuda())
    off = torch.tensor([0, 70, 105], device="cuda")
    ref = GroupProblem(x, w, off, out_dtype=torch.float32)
    ref.forward()
    for e, (a, b) in enumerate(((0, 70), (70, 105))):
        want, size = x[a:b].double() @ w[e].double(), x[a:b].double().abs() @ w[e].double().abs()
        assert bool(((ref.y[a:b].double() - want).abs() <= _loss(K) * size).all()), e
    x2 = x.clone()
    x2[33, 3000] = float("inf")
    pr = GroupProblem(x2, w, off, out_dtype=torch.float32)
    pr.forward()
    keep = torch.arange(105, device="cuda") != 33
    assert torch.equal(pr.y[keep], ref.y[keep]) and not bool(pr.y[33].isfinite().any())
    assert pr.device_error() == 0
