"""Layer norm's backward where rows lie far from zero, from given statistics.

The kernel takes x - mean, then times rstd (two roundings of h), or x rstd - mean
rstd with the second product in two parts (a rounding of h and one of a part of
2^-24 |mean| rstd, which is no larger than |h| unless that is zero): at most
three roundings, |h' - h| <= 3 x 2^-24 |h|.  With both uses of it, e = dy weight (one),
the two means (a lane's 32 sums, 5 shuffles, 16 warps and 1 / D: fewer than 56),
and the last six, dx is off by less than 72 x 2^-24 of
rstd (|e| + mean|e| + |h| mean|e h|); the sums over the rows of d_weight are
fewer than 128 roundings (rows of a team, 64 teams, 160 CTAs by 16), those of h among
them: 131 x 2^-24 of sum |dy h|.  Nothing goes by |mean| rstd."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _f64(t):
    return t.detach().double().cpu().numpy()


# widths of every shape of the kernel: teams of 8 to 512 lanes, wide loads and single ones, rows computed twice
@pytest.mark.parametrize("D", [24, 64, 128, 256, 301, 512, 1000, 1024, 1501, 2048, 4096, 5001, 8192, 16384])
@pytest.mark.parametrize("xt,yt", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32")])
def test_rows_far_from_zero(D, xt, yt):
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    g = torch.Generator().manual_seed(D)
    T = 300 if D < 2000 else 40
    at = 10.0 ** (6 * torch.rand(T, 1, generator=g) - 1)
    x = (torch.randn(T, D, generator=g) + at * torch.sign(torch.randn(T, 1, generator=g))).to(TYPES[xt]).cuda()
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()
    dy = torch.randn(T, D, generator=g).to(TYPES[yt]).cuda()
    mean = x.double().mean(-1).float()
    rstd = (x.double().var(-1, unbiased=False) + 1e-5).rsqrt().float()
    pr = LNProblem(x, w, torch.zeros_like(w), dy=dy, mean=mean, rstd=rstd)
    pr.backward()
    assert pr.device_error() == 0
    x, w, dy, mean, r = _f64(x), _f64(w), _f64(dy), _f64(mean)[:, None], _f64(rstd)[:, None]
    h, e = (x - mean) * r, dy * w
    dx = r * (e - e.mean(-1, keepdims=True) - h * (e * h).mean(-1, keepdims=True))
    size = r * (np.abs(e) + np.abs(e).mean(-1, keepdims=True) + np.abs(h) * np.abs(e * h).mean(-1, keepdims=True))
    assert np.all(np.abs(_f64(pr.dx) - dx) <= HALF[xt] * np.abs(dx) + 72 * 2.0 ** -24 * size)
    assert np.all(np.abs(_f64(pr.d_weight) - (dy * h).sum(0)) <= 131 * 2.0 ** -24 * np.abs(dy * h).sum(0))


@pytest.mark.parametrize("D", [24, 301, 512, 2048, 8192])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_constant_rows(D, dtype):
    """h is zero there, and d_weight with it."""
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    T = 50
    value = torch.linspace(-3000, 1000, T)[:, None].to(dtype).cuda()
    x = value.expand(T, D).contiguous()
    g = torch.Generator().manual_seed(D)
    dy = torch.randn(T, D, generator=g).to(dtype).cuda()
    rstd = torch.full((T,), float(np.float32(1e-5) ** -0.5), device="cuda")
    pr = LNProblem(x, torch.ones(D, device="cuda"), dy=dy, mean=value[:, 0].float(), rstd=rstd, want_weight_grad=True)
    pr.backward()
    assert pr.device_error() == 0 and not bool(pr.d_weight.any())
