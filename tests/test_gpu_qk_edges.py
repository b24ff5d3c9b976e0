"""Norm and rotation of queries and keys at their edges: gradients that are
not finite."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import serving_ref as R  # noqa: E402
from tests.test_gpu_qk import _f64, _inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 40, 3000])
def test_infinite_gradients_of_gains(T):
    # a gain's gradient is the sum of its terms, an infinity among them included; the other gains' stay what they are
    from hstu_jagged_attention_02_gb300.qk import QKProblem
    q, k, _, _, _, gains, grads = _inputs(T, 3, 2, 64, 0, "fp32", True, seed=70)
    grads[0][T // 2, 1, 5] = float("inf")
    grads[0][T // 3, 0, 9] = float("-inf")
    grads[1][T - 1, 1, 17] = float("nan")
    if T > 1:       # infinities of both signs have no sum
        x = _f64(q)[:, 0, 30]
        grads[0][0, 0, 30], grads[0][T - 1, 0, 30] = float("inf") * np.sign(x[0]), -float("inf") * np.sign(x[-1])
    pr = QKProblem(q, k, rot_dim=0, norm=True, q_gain=gains[0], k_gain=gains[1], dq_out=grads[0], dk_out=grads[1])
    pr.backward()
    assert pr.device_error() == 0
    none = np.zeros((T, 0))
    for x, gain, dout, dg, odd in ((q, gains[0], grads[0], pr.d_q_gain, (5, 9) + ((30,) if T > 1 else ())),
                                   (k, gains[1], grads[1], pr.d_k_gain, (17,))):
        with np.errstate(invalid="ignore"):
            _, want, _ = R.qk_backward(_f64(x), _f64(dout), _f64(gain), none, none, False, True, 1e-6)
            terms = np.abs(_f64(dout) * R.norm(_f64(x), None, 1e-6)[0]).sum((0, 1))
        got = _f64(dg)
        keep = np.ones(64, bool)
        keep[list(odd)] = False
        assert np.isfinite(want[keep]).all() and not np.isfinite(want[~keep]).any()
        np.testing.assert_array_equal(got[~keep], want[~keep])
        # FP32 sums, as in tests/test_gpu_qk.py
        assert np.all(np.abs(got[keep] - want[keep]) <= 2.0 ** -17 * terms[keep])
