"""A wait of the cached attention that runs out, without a hang: in the test
mode CTA 0 prepares none of its work, so its warps' waits end after a
millisecond.  The call reports HSTU_ERR_TIMEOUT, the finishing kernel follows
none of the records that were not written (they hold what the workspace held),
and the next call on the same workspace is right."""
import pytest

torch = pytest.importorskip("torch")

from hstu_jagged_attention_02_gb300 import binding as C  # noqa: E402
from tests.test_gpu_cached import Serve  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fill", [0x00, 0x7f, 0xff, "random"])
@pytest.mark.parametrize("d,cand,rows", [(128, [4, 0, 2], 8), (64, [4, 0, 2], 8), (128, [20, 3, 0], 30), (64, [50, 3, 0], 64),
                                         (128, [150, 3, 0], 153), (128, None, 4)])
def test_waits_that_run_out(d, cand, rows, fill):
    s = Serve([700, 90, 260], [3, 1, 2], cand or [0, 0, 0], 2, d, 64, seed=90 + rows)
    kw = {}
    if cand is None:        # no candidates: no keys and values of rows to read either
        kw = dict(num_targets=None)
        s.k = s.v = None
    need = s.problem(max_rows=rows, **kw).ws.numel()
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    if fill == "random":
        ws[256:] = torch.randint(0, 256, (need - 256,), generator=torch.Generator().manual_seed(rows), dtype=torch.uint8).cuda()
    else:
        ws[256:] = fill
    pr = s.problem(max_rows=rows, workspace=ws, **kw)
    pr.o.fill_(7.0)
    pr.y.fill_(7.0)
    pr.desc.flags |= C.HSTU_FLAG_TEST_TIMEOUT
    pr.forward()
    assert pr.device_error() == C.HSTU_ERR_TIMEOUT
    assert bool((pr.o == 7.0).all()) and bool((pr.y == 7.0).all())
    # an earlier error in the header hides no later timeout from the finishing kernel
    ws[0] = C.HSTU_ERR_DEVICE_CHECK
    pr.forward()
    torch.cuda.synchronize()
    assert bool((pr.o == 7.0).all()) and bool((pr.y == 7.0).all())
    pr.desc.flags &= ~C.HSTU_FLAG_TEST_TIMEOUT
    ws[:256] = 0
    pr.forward()
    assert pr.device_error() == 0
    if cand is None:
        s.k, s.v = torch.zeros_like(s.q), torch.zeros_like(s.q)     # (the check's; no row is a candidate)
    s.check(pr)
