"""A wait that runs out in a pair of CTAs (the test mode withholds the first
load of the first pair): the call ends, says so, and leaves the GPU as it was."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_groups import _inputs  # noqa: E402

pytestmark = pytest.mark.gpu


# sizes at which CTAs work in pairs: rows that stay in shared memory, rows that stream, depths of several accumulators
@pytest.mark.parametrize("sizes,K,N", [((1500,) * 4, 512, 2048), ((6000, 1, 9001), 1024, 2048), ((6000, 1, 9001), 2048, 4096)])
def test_pairs(sizes, K, N):
    from hstu_jagged_attention_02_gb300 import binding as C
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    x, w, off, _ = _inputs(sizes, K, N, seed=K)
    want = GroupProblem(x, w, off)
    want.forward()
    pr = GroupProblem(x, w, off, flags=C.HSTU_FLAG_TEST_TIMEOUT)
    pr.forward()
    assert pr.device_error() == C.HSTU_ERR_TIMEOUT
    again = GroupProblem(x, w, off)
    for _ in range(3):
        again.forward()
    assert again.device_error() == 0 and torch.equal(again.y, want.y)
    pr.ws[:256].zero_()      # the same workspace serves again
    other = GroupProblem(x, w, off, workspace=pr.ws)
    other.forward()
    assert other.device_error() == 0 and torch.equal(other.y, want.y)
