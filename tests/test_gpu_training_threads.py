"""Calls from several host threads at once: each with tensors, a workspace and
a stream of its own, of sizes that share a kernel but not the shared memory they
ask for."""
import threading

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_groups import _inputs  # noqa: E402
from tests.test_gpu_ln import _inputs as _ln_inputs  # noqa: E402

pytestmark = pytest.mark.gpu


def _groups(kind, sizes, K, N, seed):
    from hstu_jagged_attention_02_gb300.groups import GroupProblem
    x, w, off, dy = _inputs(sizes, K, N, seed=seed)
    pr = GroupProblem(x, w, off, dy=None if kind == "y" else dy, want_dx=kind == "dx", want_dw=kind == "dw")
    return (pr.forward if kind == "y" else pr.backward), pr, lambda: pr.y if kind == "y" else (pr.dx if kind == "dx" else pr.dw)


def _norm(D, seed):
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    x, w, b, dy, _ = _ln_inputs(40, D, "fp32", "fp32", seed)
    pr = LNProblem(x, w, b, dy=dy)
    pr.forward()
    return pr.backward, pr, lambda: pr.dx


PAIRS = {
    "y": lambda: [_groups("y", (5, 9), 64, 64, 1), _groups("y", (1, 2) * 1500, 64, 64, 2)],
    "dx": lambda: [_groups("dx", (5, 9), 64, 64, 3), _groups("dx", (1, 2) * 1500, 64, 64, 4)],
    "dw": lambda: [_groups("dw", (5, 9), 64, 64, 5), _groups("dw", (1,) * 2000, 64, 64, 6)],
    "norm": lambda: [_norm(288, 7), _norm(512, 8)],
}


@pytest.mark.parametrize("what", sorted(PAIRS))
def test_two_threads(what):
    pairs = PAIRS[what]()
    for call, _, _ in pairs:
        call()
    torch.cuda.synchronize()
    want = [out().clone() for _, _, out in pairs]
    failed, start = [], threading.Barrier(len(pairs))

    def work(call):
        s = torch.cuda.Stream()
        start.wait()
        try:
            for i in range(3000):
                call(s)
                if i % 200 == 199:
                    s.synchronize()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(call,)) for call, _, _ in pairs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert all(torch.equal(out(), w) and pr.device_error() == 0 for (_, pr, out), w in zip(pairs, want))
