"""AdamW where the second moment is subnormal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import training_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_subnormal_second_moments(bits):
    """A step whose v is subnormal, with a beta2 near one, so that 1 / (1 - beta2^t) brings its root back among the
    numbers that count.  The square root of a v that has k bits left of its 24 (v itself is rounded, which the 64-bit
    form takes as it is): what the parameters move by is off by 2^-19 of it, as for any v."""
    from hstu_jagged_attention_02_gb300.optim import AdamW, zero_moments
    n, lr, b1, b2, eps = 512, 1.0, 0.9, 1 - 1e-9, 1e-12
    m0 = torch.zeros(n, device="cuda")
    v0 = 10.0 ** torch.linspace(-42, -38, n)
    p, g = torch.zeros(n, device="cuda"), torch.full((n,), 1e-16, device="cuda")
    if bits == 32:
        opt = AdamW([p], [g], lr=lr, betas=(b1, b2), eps=eps, moments=[(m0, v0.cuda())])
    else:
        mom = zero_moments(p, 8)
        mom.v.copy_(torch.arange(n).remainder(240).to(torch.uint8))
        opt = AdamW([p], [g], lr=lr, betas=(b1, b2), eps=eps, moments=[mom])
        v0 = opt.read_moments()[0][1].cpu()
    opt.step()
    m, v = R.moments(np.zeros(n, np.float32), v0.numpy(), g.cpu().numpy(), b1, b2)
    want, moved = R.adamw(np.zeros(n), m.astype(np.float64), v.astype(np.float64), 1, lr, b1, b2, eps, 0.0)
    assert np.any((v > 0) & (v < 2.0 ** -126)) and opt.device_error() == 0
    assert np.all(np.abs(p.double().cpu().numpy() - want) <= 2.0 ** -19 * moved)
