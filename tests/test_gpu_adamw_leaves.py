"""AdamW beside autograd: whose gradients a step takes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import training_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu


def test_gradients_at_the_copies_are_not_passed_over():
    """Mixed precision: the BF16 copies are the leaves.  A step without a list finds nothing at the masters."""
    from hstu_jagged_attention_02_gb300.optim import AdamW
    masters = [torch.randn(300, device="cuda"), torch.randn(64, device="cuda")]
    leaves = [m.bfloat16().requires_grad_() for m in masters]
    opt = AdamW(masters, copies=leaves, grad_dtype=torch.bfloat16)
    (leaves[0].float().square().sum() + leaves[1].float().sum()).backward()
    before = [m.clone() for m in masters]
    with pytest.raises(ValueError, match="parameter 0 lies at its copy"):
        opt.step()
    assert opt.steps() == 0 and all(torch.equal(a, b) for a, b in zip(masters, before))
    # with the list it steps, and the leaves follow
    opt = AdamW(masters, [t.grad for t in leaves], copies=[t.detach() for t in leaves])
    opt.step()
    assert opt.steps() == 1 and opt.device_error() == 0
    assert all(torch.equal(t.detach(), m.bfloat16()) and not torch.equal(m, b) for t, m, b in zip(leaves, masters, before))


def test_masters_as_leaves_with_copies():
    """The masters are the leaves, and the copies are cast from them: their gradients count, whatever the copies are."""
    from hstu_jagged_attention_02_gb300.optim import AdamW
    w = torch.randn(300, device="cuda").requires_grad_()
    copy = w.detach().bfloat16()
    opt = AdamW([w], copies=[copy])
    w.square().sum().backward()
    opt.step()
    assert opt.steps() == 1 and torch.equal(copy, w.detach().bfloat16())
    made = w.bfloat16()          # no leaf
    opt = AdamW([w], copies=[made])
    opt.step()
    w.grad = None
    opt.step()
    assert opt.steps() == 2 and torch.equal(made.detach(), w.detach().bfloat16())


@pytest.mark.parametrize("how", ["weight", "copy", "detached"])
def test_a_backward_behind_a_step_finds_out(how):
    """A graph that saved what a step has changed since raises, as behind any change in place."""
    from hstu_jagged_attention_02_gb300.groups import hstu_group_linear
    from hstu_jagged_attention_02_gb300.norm import hstu_ln
    from hstu_jagged_attention_02_gb300.optim import AdamW
    x = torch.randn(40, 64, device="cuda").requires_grad_()
    if how == "copy":
        master = torch.randn(1, 64, 64, device="cuda")
        leaf = master.bfloat16().requires_grad_()
        run = lambda: hstu_group_linear(x.bfloat16(), leaf, torch.tensor([0, 40], device="cuda"))  # noqa: E731
        opt = AdamW([master], [torch.ones_like(leaf)], copies=[leaf])
    else:
        leaf = torch.randn(64, device="cuda").requires_grad_()
        run = lambda: hstu_ln(x, leaf)  # noqa: E731
        opt = AdamW([leaf if how == "weight" else leaf.detach()], [torch.ones_like(leaf)])
    run().float().sum().backward()
    y = run()
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()
    run().float().sum().backward()


def test_one_count_for_all():
    """A parameter without a gradient for two steps takes the third with the corrections of t = 3."""
    from hstu_jagged_attention_02_gb300.optim import AdamW
    first, late = (torch.zeros(256, device="cuda").requires_grad_() for _ in range(2))
    opt = AdamW([first, late], grad_dtype=torch.float32, lr=1e-3)
    for t in range(1, 4):
        first.grad = torch.ones_like(first)
        late.grad = torch.ones_like(late) if t == 3 else None
        opt.step()
        assert t == 3 or not bool(late.detach().any())
    zero, one = np.zeros(256, np.float32), np.ones(256, np.float32)
    m, v = R.moments(zero, zero, one, 0.9, 0.999)
    want, moved = R.adamw(zero.astype(np.float64), m.astype(np.float64), v.astype(np.float64), 3, 1e-3, 0.9, 0.999, 1e-8, 0.0)
    # the bound of any step: 2^-19 of what it moves by
    assert np.all(np.abs(late.detach().double().cpu().numpy() - want) <= 2.0 ** -19 * moved)
    assert opt.steps() == 3 and opt.device_error() == 0
