"""A workspace that serves one call after the other, of other shapes and of
other operators: results are those of workspaces of their own, bit for bit."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_groups import _inputs  # noqa: E402
from tests.test_gpu_ln import _inputs as _ln_inputs  # noqa: E402

pytestmark = pytest.mark.gpu


def _same(pr, own):
    return torch.equal(pr.dx, own.dx) and torch.equal(pr.dw, own.dw) if pr.dx is not None else torch.equal(pr.dw, own.dw)


# (4 x 150 rows leave sums behind their counters where 4 x 10,000 rows have counters; 30,000 rows of one group and
# widths whose tiles are taken by pairs of CTAs; many groups of which few are cut)
SHAPES = [((150,) * 4, 512, 512), ((10_000,) * 4, 512, 512), ((30_000,), 264, 520), ((1, 5000, 7, 0, 9000), 512, 2048),
          ((3,) * 400 + (4000, 6000), 64, 128), ((900, 1000), 128, 256)]


@pytest.mark.parametrize("want_dx", [True, False])
def test_shapes_in_turn(want_dx):
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    data = [_inputs(*s, seed=80 + i) for i, s in enumerate(SHAPES)]
    own = []
    for x, w, off, dy in data:
        pr = GroupProblem(x, w, off, dy=dy, want_dx=want_dx)
        pr.backward()
        own.append(pr)
    ws = torch.zeros(max(pr.ws_bytes for pr in own), dtype=torch.uint8, device="cuda")
    shared = [GroupProblem(x, w, off, dy=dy, want_dx=want_dx, workspace=ws) for x, w, off, dy in data]
    n = len(SHAPES)
    for i in [*range(n), *reversed(range(n)), 0, 3, 0, 4, 2, 5]:
        shared[i].dw.fill_(float("nan"))
        shared[i].backward()
        assert _same(shared[i], own[i]), i
    assert all(pr.device_error() == 0 for pr in shared)


def test_another_operators_workspace():
    """The header alone has to be zero: the norm's backward leaves its sums behind it."""
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    x, w, off, dy = _inputs((10_000,) * 4, 512, 512, seed=90)
    own = GroupProblem(x, w, off, dy=dy)
    own.backward()
    a, g, b, da, _ = _ln_inputs(5000, 512, "bf16", "bf16", 91)
    alone = LNProblem(a, g, b, dy=da)
    ws = torch.full((max(own.ws_bytes, alone.ws_bytes),), 0x5A, dtype=torch.uint8, device="cuda")
    ws[:256].zero_()
    ln, pr = LNProblem(a, g, b, dy=da, workspace=ws), GroupProblem(x, w, off, dy=dy, workspace=ws)
    for k in range(3):
        for p in (alone, ln):
            p.forward()
            p.backward()
        pr.dw.fill_(float("nan"))
        pr.backward()
        assert _same(pr, own), k
        assert torch.equal(ln.dx, alone.dx) and torch.equal(ln.d_weight, alone.d_weight)
    assert pr.device_error() == 0 and ln.device_error() == 0
    # and in a graph, with the weight gradient alone
    only = GroupProblem(x, w, off, dy=dy, want_dx=False, workspace=ws)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            ln.forward()
            ln.backward()
            only.backward()
    for _ in range(2):
        only.dw.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(only.dw, own.dw)
