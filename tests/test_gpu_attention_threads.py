"""Attention calls from two host threads at once, each with a batch, a workspace
and a stream of its own: batches and bias tables of sizes that share the kernels
but not the shared memory they ask for."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from hstu_jagged_attention_02_gb300 import synth  # noqa: E402
from hstu_jagged_attention_02_gb300.attention import Problem  # noqa: E402

pytestmark = pytest.mark.gpu


def _problem(dtype, d, B, P, Tb, seed):
    rng = np.random.default_rng(seed)
    b = synth.make_batch(rng.integers(1, 60, B), H=2, d_qk=d, d_v=d, dtype=dtype, num_targets=3, seed=seed)
    b.rab_pos, b.rab_time = (0.02 * rng.standard_normal((2, n)).astype(np.float32) for n in (P, Tb))
    return Problem(b)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 32)])
def test_two_threads(dtype, d):
    pairs = [_problem(dtype, d, 3, 128, 64, 1), _problem(dtype, d, 400, 900, 200, 2)]
    for pr in pairs:
        pr.forward()
        pr.backward()
    torch.cuda.synchronize()
    want = [(pr.o.clone(), pr.dvv.clone()) for pr in pairs]
    failed, start = [], threading.Barrier(len(pairs))

    def work(pr):
        s = torch.cuda.Stream()
        start.wait()
        try:
            for i in range(1500):
                pr.forward(s)
                pr.backward(s)
                if i % 50 == 49:
                    s.synchronize()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(pr,)) for pr in pairs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for pr, (o, dv) in zip(pairs, want):
        assert pr.device_error() == 0 and torch.equal(pr.o, o)
        assert torch.allclose(pr.dvv, dv, rtol=1e-5, atol=1e-6)
