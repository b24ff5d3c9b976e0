"""The time buckets of the attention over the paged cache for gaps beyond 63
bits: a bucket is the number of binary digits of the gap, whatever the signs
and sizes of the two times."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_cached import Serve  # noqa: E402

pytestmark = pytest.mark.gpu

FAR = 6 * 10 ** 18      # two of them apart pass 2^63


@pytest.mark.parametrize("rows", [6, 20, 100])
@pytest.mark.parametrize("early,late", [(-FAR, FAR), (-(1 << 63), (1 << 63) - 1)])
def test_gaps_beyond_63_bits(rows, early, late):
    # cached tokens near the earliest row: among them the 32-bit gaps of most rows, and rows further than int64 holds
    s = Serve([300, 40], [3, 0], [rows - 3, rows], 2, 64, 32, seed=80 + rows)
    first = int(s.tc.min())
    s.cache.timestamps.sub_(first).add_(early + 5)
    s.tc = s.tc.astype(object) - first + early + 5          # Python integers: no gap wraps
    g = torch.Generator().manual_seed(81)
    t = torch.randint(0, 1 << 20, (s.T,), generator=g) + early
    t[torch.rand(s.T, generator=g) < 0.5] = late
    t[0], t[-1] = early, late
    s.times = t.cuda()
    pr = s.problem()
    pr.forward()
    assert pr.device_error() == 0
    s.check(pr)
    # the other way round: the tokens late, some rows early
    s.cache.timestamps.fill_(late)
    s.tc = s.tc * 0 + late
    pr.forward()
    assert pr.device_error() == 0
    s.check(pr)
