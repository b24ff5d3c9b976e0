"""Calls of the serving operators' Python classes that are refused on the host
because their results would be wrong."""
import pytest

torch = pytest.importorskip("torch")

from hstu_jagged_attention_02_gb300.qk import QKProblem  # noqa: E402


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("norm", [True, False])
def test_a_forward_in_place_leaves_the_norms_backward_no_inputs(norm, given):
    q, k, g = torch.zeros(5, 2, 64), torch.zeros(5, 1, 64), torch.zeros(5, 2, 64)
    out = dict(k_out=k) if given else dict(inplace=True)
    with pytest.raises(ValueError) as e:
        QKProblem(q, k, norm=norm, dq_out=g, dk_out=g[:, :1], **out)
    # without the norm the gradient reads neither: refused only for being on the host
    assert ("overwrites" in str(e.value)) == norm
    with pytest.raises(ValueError, match="CUDA device"):
        QKProblem(q, k, norm=norm, **out)
