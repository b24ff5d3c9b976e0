"""What the training block's handles refuse about tensors that share memory, or
that have moved (checked on the host, before anything is launched)."""
import pytest

torch = pytest.importorskip("torch")

from hstu_jagged_attention_02_gb300.groups import GroupProblem  # noqa: E402
from hstu_jagged_attention_02_gb300.norm import LNProblem  # noqa: E402
from hstu_jagged_attention_02_gb300.optim import AdamW, _apart  # noqa: E402


def test_inputs_that_an_output_overwrites():
    x = torch.zeros(10, 64)
    with pytest.raises(ValueError, match="forward in place"):
        LNProblem(x, y=x, dy=torch.zeros(10, 64))
    a, w, off = torch.zeros(10, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    dy = torch.zeros(10, 64, dtype=torch.bfloat16)
    for kw in (dict(y=a), dict(dy=dy, dx=dy), dict(dy=dy, dx=a)):
        with pytest.raises(ValueError, match="lie apart"):
            GroupProblem(a, w, off, **kw)


def test_gradients_that_a_step_overwrites():
    buf = torch.zeros(400)
    p, m, v = buf[:100], buf[100:200], buf[200:300]
    for g in (p, v, buf[52:152], buf[48:148], buf[252:352]):
        with pytest.raises(ValueError, match="gradient 0 overlaps"):
            AdamW([p], [g], moments=[(m, v)])
    with pytest.raises(ValueError, match="CUDA"):   # apart: goes on to the device, which is missing here
        AdamW([p], [buf[300:]], moments=[(m, v)])


@pytest.mark.parametrize("lo,hi,want", [(0, 4, True), (0, 5, False), (4, 8, False), (5, 6, False), (8, 12, True), (6, 14, False),
                                        (20, 24, True), (0, 24, False), (6, 6, True)])
def test_spans(lo, hi, want):
    t = torch.zeros(24, dtype=torch.uint8)
    at = t.data_ptr()
    assert _apart([(at + 4, at + 8), (at + 12, at + 20)], t[lo:hi]) == want
