"""The training block's operators beside other work: streams other than the
one on which a problem's buffers were made, calls at the same time, captures."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_adamw import _tensors  # noqa: E402
from tests.test_gpu_groups import _inputs as _group_inputs  # noqa: E402
from tests.test_gpu_ln import _inputs as _ln_inputs  # noqa: E402

pytestmark = pytest.mark.gpu


def _dirty(n=64 << 20):
    """Leaves the allocator memory that holds no zeros."""
    x = torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
    y = [torch.full((1 << k,), 0x7f, dtype=torch.uint8, device="cuda") for k in range(9, 26) for _ in range(4)]
    torch.cuda.synchronize()
    del x, y


def _problems():
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    from hstu_jagged_attention_02_gb300.optim import AdamW
    x, w, b, dy, _ = _ln_inputs(900, 300, "bf16", "bf16", 50)
    gx, gw, off, gdy = _group_inputs((600, 33, 5000), 264, 520, seed=51)
    odd = torch.zeros(gx.shape[0], 267, dtype=torch.bfloat16, device="cuda")[:, 1:265].copy_(gx)
    params, grads = _tensors([3000, 17], 52)
    return (x.t().contiguous().t(), w, b, dy), (odd, gw, off, gdy), (params, grads), (LNProblem, GroupProblem, AdamW)


def _run(ln, gp, opt, stream, how):
    calls = [ln.forward, ln.backward, gp.forward, gp.backward, opt.step]
    for call in calls:
        if how == "argument":
            call(stream)
        else:
            with torch.cuda.stream(stream):
                call()


@pytest.mark.parametrize("how", ["argument", "current"])
def test_a_first_call_on_another_stream(how):
    want = None
    for late in (False, True):
        a, b, (params, grads), (LN, Group, Adam) = _problems()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        _dirty()
        if late:
            torch.cuda._sleep(40_000_000)       # some 20 ms, before everything that the constructors queue
        ln, gp = LN(a[0], a[1], a[2], dy=a[3]), Group(*b[:3], dy=b[3])
        opt = Adam(params, grads, lr=1e-3, state_bits=8, seed=1)
        if not late:
            torch.cuda.synchronize()
        _run(ln, gp, opt, side, how)
        torch.cuda.synchronize()
        assert ln.device_error() == 0 and gp.device_error() == 0 and opt.device_error() == 0
        got = [ln.y, ln.dx, ln.d_weight, gp.y, gp.dx, gp.dw, *params, *opt.moments[0]]
        if want is None:
            want = [x.clone() for x in got]
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_calls_at_the_same_time():
    """Two of each, with workspaces of their own, on two streams at once."""
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    pairs = []
    for k in range(2):
        x, w, b, dy, _ = _ln_inputs(3000 + k, 512, "bf16", "bf16", 60 + k)
        gx, gw, off, gdy = _group_inputs((4000, 33 + k, 9000), 256, 512, seed=62 + k)
        pairs.append((LNProblem(x, w, b, dy=dy), GroupProblem(gx, gw, off, dy=gdy)))
    outs = lambda: [t for ln, gp in pairs for t in (ln.y, ln.dx, ln.d_weight, ln.d_bias, gp.y, gp.dx, gp.dw)]  # noqa: E731
    calls = lambda ln, gp: (ln.forward(), ln.backward(), gp.forward(), gp.backward())  # noqa: E731
    for ln, gp in pairs:
        calls(ln, gp)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs()]
    streams = [torch.cuda.Stream() for _ in pairs]
    for _ in range(5):
        for t in outs():
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            for s, (ln, gp) in zip(streams, pairs):
                with torch.cuda.stream(s):
                    calls(ln, gp)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs(), want))
    assert all(ln.device_error() == 0 and gp.device_error() == 0 for ln, gp in pairs)


def test_a_captured_step_beside_autograd():
    """A step of handles is captured while a graph of autograd over the same tensors is alive."""
    from hstu_jagged_attention_02_gb300.groups import GroupProblem, hstu_group_linear
    from hstu_jagged_attention_02_gb300.norm import LNProblem, hstu_ln
    x, w, b, _, _ = _ln_inputs(400, 64, "bf16", "bf16", 70)
    _, gw, off, gdy = _group_inputs((150, 0, 250), 64, 128, seed=71)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, gw)]
    y = hstu_group_linear(hstu_ln(leaves[0], leaves[1], leaves[2]), leaves[3], off)
    y.backward(gdy, retain_graph=True)
    eager = [t.grad.clone() for t in leaves]
    ln = LNProblem(x, w, b, out_dtype=torch.bfloat16, dy=torch.zeros(400, 64, device="cuda", dtype=torch.bfloat16))
    gp = GroupProblem(ln.y, gw, off, dy=gdy, dx=ln.dy)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            ln.forward()
            gp.forward()
            gp.backward()
            ln.backward()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(gp.y, y.detach()) and torch.equal(gp.dw.bfloat16(), eager[3])
    assert torch.equal(ln.dx, eager[0]) and torch.equal(ln.d_weight, eager[1]) and torch.equal(ln.d_bias, eager[2])
    for t in leaves:
        t.grad = None
    y.backward(gdy)                       # the eager graph as before
    assert all(torch.equal(t.grad, e) for t, e in zip(leaves, eager))
