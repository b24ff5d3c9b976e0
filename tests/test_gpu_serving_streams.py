"""The serving operators' classes beside other work: batches of no tokens, and
streams other than the one on which a problem's buffers were made."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_cached import Serve  # noqa: E402
from tests.test_gpu_qk import _inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("odd", [False, True])
def test_batches_of_no_tokens(odd):
    # whatever strides a tensor without elements has (a cut of a padded row, say)
    from hstu_jagged_attention_02_gb300.cache import PagedCache, hstu_attention_cached, hstu_cache_append, hstu_cache_read
    from hstu_jagged_attention_02_gb300.qk import QKProblem, hstu_qk_norm_rope, rope_tables
    H, d = 2, 64
    width = d + 3 if odd else d
    some = lambda: torch.zeros(4, H, width, dtype=torch.bfloat16, device="cuda")[2:2, :, width - d:]  # noqa: E731
    cos, sin = rope_tables(10, d)
    pos, gain = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.ones(d, device="cuda")
    pr = QKProblem(some(), some(), pos, cos, sin, q_gain=gain, k_gain=gain, dq_out=some(), dk_out=some())
    pr.d_q_gain.fill_(3.0)
    pr.forward()
    pr.backward()
    assert pr.device_error() == 0 and not pr.d_q_gain.any() and pr.q_out.shape == (0, H, d)
    q = some().requires_grad_()
    hstu_qk_norm_rope(q, None, pos, cos, sin)[0].sum().backward()
    assert q.grad.shape == q.shape
    cache = PagedCache(3, H=H, d=d, page_size=32)
    off, lens = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    when = torch.zeros(0, dtype=torch.int64, device="cuda")
    hstu_cache_append(cache, some(), some(), off, lens, table, timestamps=when, cos=cos, sin=sin, norm=True)
    k, v, t = hstu_cache_read(cache, off, lens, table)
    assert k.shape == v.shape == (0, H, d) and t.shape == (0,) and not cache.pages.any()
    o, y = hstu_attention_cached(cache, some(), some(), some(), None, off, lens, table, max_rows=4, max_seq_len=20, alpha=0.1,
                                 num_targets=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert o.shape == (0, H, d) and y.shape == (0, H * d)
