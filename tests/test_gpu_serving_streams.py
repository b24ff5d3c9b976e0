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


def _dirty(n=64 << 20):
    """Leaves the allocator memory that holds no zeros."""
    x = torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
    y = [torch.full((1 << k,), 0x7f, dtype=torch.uint8, device="cuda") for k in range(9, 22) for _ in range(4)]
    torch.cuda.synchronize()
    del x, y


@pytest.mark.parametrize("how", ["argument", "current"])
def test_a_first_call_on_another_stream(how):
    """Problems made on a stream that is still busy, called on another one: their
    own buffers (a zeroed workspace, copies of tensors in other layouts) are
    there first.  The other stream waits for the inputs itself, as it must."""
    from hstu_jagged_attention_02_gb300.qk import QKProblem
    q, k, pos, cos, sin, gains, grads = _inputs(2000, 4, 2, 128, 128, "bf16", True, seed=110)
    odd = torch.zeros(2000, 4, 131, dtype=torch.bfloat16, device="cuda")[..., 1:129]
    odd.copy_(q)
    s = Serve([700, 90], [2, 1], [30, 4], 2, 128, 64, seed=111)
    s.q = torch.zeros(s.T, 2, 131, dtype=torch.bfloat16, device="cuda")[..., 1:129].copy_(s.q)
    args = dict(q_gain=gains[0], k_gain=gains[1], dq_out=grads[0], dk_out=grads[1])

    def run(pr, stream, name):
        if how == "argument":
            getattr(pr, name)(stream)
        else:
            with torch.cuda.stream(stream):
                getattr(pr, name)()

    want = None
    for late in (False, True):
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        _dirty()
        if late:
            torch.cuda._sleep(40_000_000)       # some 20 ms, before everything that the constructors queue
        at = s.problem()
        qk = QKProblem(odd, k, pos, cos, sin, **args)
        if not late:
            torch.cuda.synchronize()
        run(at, side, "forward")
        run(qk, side, "forward")
        run(qk, side, "backward")
        torch.cuda.synchronize()
        assert at.device_error() == 0 and qk.device_error() == 0
        got = [at.o, at.y, qk.q_out, qk.k_out, qk.dq, qk.dk, qk.d_q_gain, qk.d_k_gain]
        if want is None:
            want = [x.clone() for x in got]
            s.check(at)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_capture_on_another_stream():
    # nothing of another stream is waited for inside a capture
    s = Serve([300], [1], [6], 2, 64, 32, seed=112)
    pr = s.problem()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            pr.forward()
            pr.forward(side)
    graph.replay()
    torch.cuda.synchronize()
    assert pr.device_error() == 0
    s.check(pr)
    # after it as before
    pr.o.zero_()
    torch.cuda.synchronize()
    pr.forward(side)
    torch.cuda.synchronize()
    s.check(pr)
