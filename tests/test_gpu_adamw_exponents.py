"""AdamW from moments in 8 bits whose exponent bytes lie below the least one."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("byte", [0, 3, 6, 7, 14, 15, 16])
def test_exponent_bytes_below_the_least(byte):
    """Moments restored from zeros: a byte below 16 counts as 16."""
    from hstu_jagged_attention_02_gb300.optim import AdamW, Moments8
    n = 700
    g = torch.Generator().manual_seed(byte)

    def start(e, codes):
        make = lambda: torch.full((3,), e, dtype=torch.uint8, device="cuda")  # noqa: E731
        return Moments8(codes[0].clone(), codes[1].clone(), make(), make())

    grad = torch.randn(n, generator=g).cuda()
    grad[5] = 0.0
    some = [torch.randint(0, 100, (n,), generator=g).to(torch.uint8).cuda() for _ in range(2)]
    for codes in ([torch.zeros(n, dtype=torch.uint8, device="cuda")] * 2, some):
        runs = []
        for e in (byte, 16):
            p, mom = torch.ones(n, device="cuda"), start(e, codes)
            opt = AdamW([p], [grad], lr=1e-3, moments=[mom], seed=4)
            read = opt.read_moments()[0]
            opt.step()
            assert opt.device_error() == 0
            runs.append([p, *mom, *read])
        assert all(torch.equal(a, b) for a, b in zip(*runs))
        assert all(bool(t.isfinite().all()) for t in runs[0] if t.is_floating_point())
