"""What the backward of the differentiable calls allocates: its results, not
the forward's output once more."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def _rise(run):
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    run()
    torch.cuda.synchronize()
    return torch.cuda.max_memory_allocated() - before


def test_products_of_groups():
    from hstu_jagged_attention_02_gb300 import binding as C
    from hstu_jagged_attention_02_gb300.groups import GroupProblem, hstu_group_linear
    T, K, N = 20_000, 64, 4096
    x = torch.randn(T, K, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(2, K, N, device="cuda").bfloat16().requires_grad_()
    off = torch.tensor([0, 9_000, T], device="cuda")
    y, dy = hstu_group_linear(x, w, off), torch.randn(T, N, device="cuda").bfloat16()
    ws = C.hstu_group_workspace_size(GroupProblem(x.detach(), w.detach(), off).desc)[1]
    results = 2 * T * K + 6 * 2 * K * N      # dx, dw in FP32 and in w's type
    assert _rise(lambda: y.backward(dy)) < results + ws + (8 << 20) < 2 * T * N


def test_layer_norm():
    from hstu_jagged_attention_02_gb300.norm import LNProblem, hstu_ln
    T, D = 20_000, 2048
    x = torch.randn(T, D, device="cuda").requires_grad_()
    w = torch.ones(D, device="cuda").requires_grad_()
    y, dy = hstu_ln(x, w), torch.randn(T, D, device="cuda")
    assert _rise(lambda: y.backward(dy)) < 4 * T * D + (16 << 20)
    # a problem of the backward alone
    stats = x.detach().mean(-1), (x.detach().var(-1, unbiased=False) + 1e-5).rsqrt()
    pr = LNProblem(x.detach(), w.detach(), dy=dy, mean=stats[0], rstd=stats[1], want_y=False)
    pr.backward()
    assert pr.y is None and pr.device_error() == 0
    with pytest.raises(ValueError, match="no forward"):
        pr.forward()
    for kw in (dict(dy=dy), dict(mean=stats[0], rstd=stats[1])):
        with pytest.raises(ValueError, match="backward alone"):
            LNProblem(x.detach(), w.detach(), want_y=False, **kw)
