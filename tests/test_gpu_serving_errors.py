"""What the device finds wrong in the one-call functions of the serving path is
in the workspace that the caller gave."""
import pytest

torch = pytest.importorskip("torch")

from hstu_jagged_attention_02_gb300 import binding as C  # noqa: E402
from tests.test_gpu_cached import Serve  # noqa: E402
from tests.test_gpu_qk import _inputs  # noqa: E402

pytestmark = pytest.mark.gpu


def test_errors_of_one_call_functions():
    from hstu_jagged_attention_02_gb300.cache import hstu_attention_cached, hstu_cache_append, hstu_cache_read
    from hstu_jagged_attention_02_gb300.qk import device_error, hstu_qk_norm_rope
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    q, k, pos, cos, sin, gains, _ = _inputs(20, 2, 2, 64, 64, "bf16", True, seed=120)
    q, gain = q.detach().requires_grad_(), gains[0].requires_grad_()
    want = hstu_qk_norm_rope(q, k, pos, cos, sin, q_gain=gain)
    got = hstu_qk_norm_rope(q, k, pos, cos, sin, q_gain=gain, workspace=ws)
    assert device_error(q.device, ws) == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got[0].float().square().sum().backward()
    assert q.grad is not None and gain.grad is not None
    bad = pos.clone()
    bad[3] = cos.shape[0]
    hstu_qk_norm_rope(q, k, bad, cos, sin, workspace=ws)
    assert device_error(q.device, ws) == C.HSTU_ERR_DEVICE_CHECK

    s = Serve([100, 70], [2, 0], [3, 9], 2, 64, 32, seed=121)
    off = torch.tensor([0, 2, 3]).cuda()
    new = torch.randn(3, 2, 64, device="cuda").bfloat16()
    when = torch.zeros(3, dtype=torch.int64, device="cuda")
    for broken in (False, True):
        if broken:
            s.table[0, 3] = 10 ** 6
        ws.zero_()
        hstu_cache_append(s.cache, new, new, off, s.lens, s.table, timestamps=when, workspace=ws)
        assert device_error(ws.device, ws) == (C.HSTU_ERR_DEVICE_CHECK if broken else 0)
        ws.zero_()
        hstu_cache_read(s.cache, off, s.lens - off.diff().int(), s.table, workspace=ws)
        assert device_error(ws.device, ws) == (C.HSTU_ERR_DEVICE_CHECK if broken else 0)
        big = torch.zeros_like(s.problem().ws)
        hstu_attention_cached(s.cache, s.q, s.k, s.v, s.u, s.off, s.lens, s.table, max_rows=9, max_seq_len=200, alpha=0.1,
                              num_targets=s.nt, workspace=big)
        assert device_error(ws.device, big) == (C.HSTU_ERR_DEVICE_CHECK if broken else 0)
