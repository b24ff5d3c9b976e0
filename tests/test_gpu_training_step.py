"""Layer norm, the products of groups and AdamW together, as a training step
uses them: around the attention, in a block of products by kind of token, and
behind the layer's own backward."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import training_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().double().cpu().numpy()


def _rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


def test_a_block_of_products_by_kind():
    """x + (SiLU(LN(x) W1[kind])) W2[kind], its gradients and three AdamW steps
    against the same in 64 bits.  Roundings to BF16 on the way (the norm's output, both
    products' outputs, the activation, the gradients between them): each half a step, 2^-8
    of its value; a gradient passes through seven of them and sums of random signs do not add them
    all up, so 7 x 2^-8 of a tensor's RMS bounds the RMS of what is off."""
    from hstu_jagged_attention_02_gb300.groups import group_rows, hstu_group_linear
    from hstu_jagged_attention_02_gb300.norm import hstu_ln
    from hstu_jagged_attention_02_gb300.optim import AdamW
    g = torch.Generator().manual_seed(1)
    T, D, F, E = 700, 128, 256, 3
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    kind = torch.randint(0, E, (T,), generator=g).cuda()
    order, off = group_rows(kind, E)
    x, dout = rnd(T, D)[order].contiguous(), rnd(T, D)
    masters = [1 + 0.1 * rnd(D), 0.1 * rnd(D), rnd(E, D, F) * D ** -0.5, rnd(E, F, D) * F ** -0.5]
    copies = [None, None, masters[2].bfloat16(), masters[3].bfloat16()]
    w, b, w1, w2 = masters[0], masters[1], copies[2], copies[3]
    for t in (w, b, w1, w2):
        t.requires_grad_()
    grads = [torch.zeros_like(t) for t in masters]
    hyper = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8)
    opt = AdamW([t.detach() for t in masters], grads, copies=[None, None] + [t.detach() for t in copies[2:]], weight_decay=0.05,
                **hyper)
    state = [(np.zeros(t.shape, np.float32).reshape(-1),) * 2 for t in masters]
    bounds = off.tolist()
    for step in range(1, 4):
        xl = x.clone().requires_grad_()
        h = hstu_ln(xl, w, b, out_dtype=torch.bfloat16)
        a = torch.nn.functional.silu(hstu_group_linear(h, w1, off))
        y = xl + hstu_group_linear(a, w2, off)
        y.backward(dout)
        # the same in 64 bits, on the same (rounded) weights
        leaves = [t.detach().double().requires_grad_() for t in (xl, w, b, w1, w2)]
        x6, w6, b6, v1, v2 = leaves
        var, mean = torch.var_mean(x6, -1, unbiased=False, keepdim=True)
        h6 = (x6 - mean) / (var + 1e-5).sqrt() * w6 + b6
        rows = [slice(bounds[e], bounds[e + 1]) for e in range(E)]
        z6 = torch.cat([h6[r] @ v1[e] for e, r in enumerate(rows)])
        a6 = z6 / (1 + torch.exp(-z6))
        y6 = x6 + torch.cat([a6[r] @ v2[e] for e, r in enumerate(rows)])
        want = torch.autograd.grad(y6, leaves, dout.double())
        got = [xl.grad, w.grad, b.grad, w1.grad, w2.grad]
        for name, p, q in zip(("x", "w", "b", "w1", "w2"), got, want):
            p, q = _f64(p), _f64(q)
            assert _rms(p - q) <= 7 * 2.0 ** -8 * _rms(q), (step, name)
        assert _rms(_f64(y) - _f64(y6)) <= 7 * 2.0 ** -8 * _rms(_f64(y6))
        before = [_f64(t).reshape(-1) for t in masters]
        for dst, src in zip(grads, got[1:]):
            dst.copy_(src.float())
        opt.step()
        for i, t in enumerate(masters):
            m, v = R.moments(*state[i], grads[i].cpu().numpy().reshape(-1), 0.9, 0.999)
            state[i] = (m, v)
            now, moved = R.adamw(before[i], m.astype(np.float64), v.astype(np.float64), step, 1e-3, 0.9, 0.999, 1e-8, 0.05)
            assert np.all(np.abs(_f64(t).reshape(-1) - now) <= 2.0 ** -22 * np.abs(now) + 2.0 ** -19 * moved)
        for t, c in zip(masters[2:], (w1, w2)):
            assert torch.equal(c.detach(), t.bfloat16())
        for t in (w, b, w1, w2):
            t.grad = None
    assert opt.steps() == 3


def test_around_the_attention():
    """LN, projections by kind into q, k, v, u, the attention, and back: the
    gradients are those of the operators' own handles."""
    from hstu_jagged_attention_02_gb300.attention import hstu_attention
    from hstu_jagged_attention_02_gb300.groups import GroupProblem, group_rows, hstu_group_linear
    from hstu_jagged_attention_02_gb300.norm import LNProblem, hstu_ln
    g = torch.Generator().manual_seed(2)
    lens, H, d = [150, 0, 210], 2, 128
    T, D = sum(lens), H * d
    off = torch.tensor([0, 150, 150, 360], device="cuda")
    nt = torch.tensor([20, 0, 30], dtype=torch.int32, device="cuda")
    # candidates take another projection than the history
    kind = torch.zeros(T, dtype=torch.int64)
    kind[130:150], kind[330:360] = 1, 1
    order, goff = group_rows(kind.cuda(), 2)
    back = torch.empty_like(order)
    back[order] = torch.arange(T, device="cuda")
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, w, b = rnd(T, D).bfloat16().requires_grad_(), (1 + 0.1 * rnd(D)).requires_grad_(), (0.1 * rnd(D)).requires_grad_()
    proj = (rnd(2, D, 4 * D) * D ** -0.5).bfloat16().requires_grad_()
    dy = rnd(T, D)
    h = hstu_ln(x, w, b)
    h.retain_grad()
    hs = h[order]
    z = hstu_group_linear(hs, proj, goff)
    z.retain_grad()
    u, v, q, k = z[back].split(D, 1)
    y = hstu_attention(q.reshape(T, H, d), k.reshape(T, H, d), v.reshape(T, H, d), u, off, 210, d ** -0.5, num_targets=nt)
    y.backward(dy)
    gp = GroupProblem(h.detach()[order], proj.detach(), goff, dy=z.grad)
    gp.forward()
    gp.backward()
    assert torch.equal(gp.y, z.detach()) and torch.equal(proj.grad, gp.dw.bfloat16())
    assert torch.equal(h.grad[order], gp.dx)
    ln = LNProblem(x.detach(), w.detach(), b.detach(), dy=h.grad)
    ln.forward()
    ln.backward()
    assert torch.equal(ln.y, h.detach()) and torch.equal(x.grad, ln.dx)
    assert torch.equal(w.grad, ln.d_weight) and torch.equal(b.grad, ln.d_bias)
    assert bool(x.grad.isfinite().all()) and float(x.grad.float().abs().sum()) > 0


@pytest.mark.parametrize("bits", [32, 8])
def test_the_layer_is_stepped(bits):
    """LayerProblem.optimizer: the layer's operands follow its FP32 masters, by its own gradients,
    launched one by one and from a graph."""
    from hstu_jagged_attention_02_gb300 import synth
    from hstu_jagged_attention_02_gb300.layer import LayerProblem
    b = synth.layer(5, n_lo=100, n_hi=300, B=3)
    pr, twin = LayerProblem(b), LayerProblem(b)
    opt = pr.optimizer(lr=1e-3, weight_decay=0.1, state_bits=bits, seed=3)
    second = twin.optimizer(lr=1e-3, weight_decay=0.1, state_bits=bits, seed=3)

    def step(p, o):
        p.forward()
        p.backward()
        o.step()

    w1, tables = pr.w1.clone(), pr.rab_pos.clone()
    first = opt.params[0].clone()
    step(pr, opt)
    assert pr.device_error() == 0 and opt.device_error() == 0
    # a first step moves every weight with a gradient by about lr
    moved = opt.params[0] - first * (1 - 1e-3 * 0.1)
    big = pr.dw1.abs() > 1e-5        # (beside eps)
    assert bool(big.any()) and torch.allclose(moved[big], -1e-3 * torch.sign(pr.dw1[big]), rtol=0.01, atol=1e-7)
    assert torch.equal(pr.w1, opt.params[0].bfloat16()) and torch.equal(pr.w2, opt.params[1].bfloat16())
    assert not torch.equal(pr.w1, w1) and not torch.equal(pr.rab_pos, tables)
    step(twin, second)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step(twin, second)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert second.steps() == 3 and twin.device_error() == 0
    # (the layer's weight gradients are sums in no fixed order: near, not equal)
    step(pr, opt)
    step(pr, opt)
    assert opt.steps() == 3
    assert torch.allclose(twin.out, pr.out, rtol=0.05, atol=0.05 * float(pr.out.std()))
