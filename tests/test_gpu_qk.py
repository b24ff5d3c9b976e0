"""Norm and rotation of queries and keys (hstu_qk_norm_rope_*) against a plain
64-bit form and, for the gradients, against differences of it.

Tolerances: an output is rounded once (half a step of its type) from FP32
arithmetic whose error is below 2^-20 of the turned feature's two terms
(sum of squares, root, two products and the turn: eight roundings of 2^-24
at most on each).  The gradients add a mean over the row (2^-18 of the terms'
sizes); a gain's gradient is a sum in FP32 over at most a few hundred rows a
lane and FP64 above: 2^-17 of the sum of its terms' sizes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import serving_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _inputs(T, Hq, Hk, d, rot, dtype, norm, seed, max_pos=300, side_by_side=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    both = rnd(T, Hq + Hk, d).to(TYPES[dtype]).cuda()
    q, k = both[:, :Hq], both[:, Hq:]
    if not side_by_side:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(0, max_pos, (T,), generator=g, dtype=torch.int32).cuda()
    cos, sin = (torch.from_numpy(x).cuda() for x in R.rope_tables(max_pos, rot)) if rot else (None, None)
    gains = [(1 + 0.3 * rnd(d)).cuda() if norm else None for _ in range(2)]
    grads = [rnd(T, H, d).to(TYPES[dtype]).cuda() for H in (Hq, Hk)]
    return q if Hq else None, k if Hk else None, pos, cos, sin, gains, [x if x.shape[1] else None for x in grads]


def _angles(pos, cos, sin, T):
    if cos is None:
        return np.ones((T, 0)), np.zeros((T, 0))
    p = pos.cpu().numpy()
    return cos.cpu().numpy()[p], sin.cpu().numpy()[p]


def _check(name, got, want, bound):
    got = _f64(got)
    assert got.shape == want.shape, name
    off = np.abs(got - want)
    assert np.all(off <= bound), f"{name}: off by {np.max(off / np.maximum(bound, 1e-300)):.3g} of what it may be"


CASES = [
    # T, Hq, Hk, d, rot, interleaved, norm, dtype
    (1, 1, 1, 128, 128, False, True, "bf16"),
    (1, 4, 4, 128, 128, False, True, "fp32"),
    (37, 4, 4, 128, 128, False, True, "bf16"),
    (333, 4, 1, 128, 64, False, True, "bf16"),
    (65, 3, 2, 128, 8, False, True, "fp32"),
    (129, 4, 2, 64, 64, False, True, "bf16"),
    (50, 5, 3, 64, 16, False, True, "fp32"),
    (77, 7, 1, 32, 32, False, True, "bf16"),
    (31, 9, 2, 32, 8, False, True, "fp32"),
    (40, 4, 4, 128, 128, True, True, "bf16"),
    (41, 2, 2, 64, 32, True, True, "fp32"),
    (42, 3, 3, 32, 8, True, True, "bf16"),
    (100, 4, 4, 128, 0, False, True, "bf16"),
    (100, 4, 4, 128, 128, False, False, "bf16"),
    (64, 2, 2, 64, 64, True, False, "fp32"),
    (19, 4, 0, 128, 128, False, True, "bf16"),
    (19, 0, 3, 64, 64, False, True, "fp32"),
    (2500, 4, 4, 128, 128, False, True, "bf16"),
    (3001, 6, 2, 64, 32, True, True, "fp32"),
]


@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter,norm,dtype", CASES)
def test_forward_and_backward(T, Hq, Hk, d, rot, inter, norm, dtype):
    from hstu_jagged_attention_02_gb300.qk import QKProblem
    q, k, pos, cos, sin, gains, grads = _inputs(T, Hq, Hk, d, rot, dtype, norm, seed=T + d)
    pr = QKProblem(q, k, pos, cos, sin, rot_dim=rot, interleaved=inter, norm=norm, eps=1e-6, q_gain=gains[0],
                   k_gain=gains[1], dq_out=grads[0], dk_out=grads[1])
    for t in (pr.q_out, pr.k_out, pr.dq, pr.dk, pr.d_q_gain, pr.d_k_gain):
        if t is not None:
            t.fill_(float("nan"))
    pr.forward()
    pr.backward()
    assert pr.device_error() == 0
    c, s = _angles(pos, cos, sin, T)
    for n, x, gain, dout, out, dx, dg in (("q", q, gains[0], grads[0], pr.q_out, pr.dq, pr.d_q_gain),
                                          ("k", k, gains[1], grads[1], pr.k_out, pr.dk, pr.d_k_gain)):
        if x is None:
            continue
        x64, g64 = _f64(x), None if gain is None else _f64(gain)
        want = R.qk_forward(x64, g64, c, s, inter, norm, 1e-6)
        w = R.norm(x64, g64, 1e-6)[0] if norm else x64
        _check(n + "'", out, want, HALF[dtype] * np.abs(want) + 2.0 ** -20 * R.spread(w, rot, inter))
        want, want_g, size = R.qk_backward(x64, _f64(dout), g64, c, s, inter, norm, 1e-6)
        _check("d" + n, dx, want, HALF[dtype] * np.abs(want) + 2.0 ** -18 * size)
        if norm:
            terms = (R.spread(_f64(dout), rot, inter) * np.abs(R.norm(x64, None, 1e-6)[0])).sum((0, 1))
            _check("dg" + n, dg, want_g, 2.0 ** -17 * terms)


def test_gradients_against_differences():
    # the formula's own gradient: central differences of the 64-bit form
    rng = np.random.default_rng(3)
    x, gain, dout = rng.normal(size=(5, 2, 64)), 1 + 0.3 * rng.normal(size=64), rng.normal(size=(5, 2, 64))
    c, s = (t[rng.integers(0, 40, 5)] for t in R.rope_tables(40, 32))
    f = lambda a, g: (R.qk_forward(a, g, c, s, True, True, 1e-6) * dout).sum()  # noqa: E731
    dx, dg, _ = R.qk_backward(x, dout, gain, c, s, True, True, 1e-6)
    for at in ((0, 0, 0), (2, 1, 31), (4, 0, 63), (1, 1, 32)):
        e = np.zeros_like(x)
        e[at] = 1e-6
        assert abs((f(x + e, gain) - f(x - e, gain)) / 2e-6 - dx[at]) < 1e-6 * max(1, abs(dx[at]))
    for i in (0, 7, 40):
        e = np.zeros_like(gain)
        e[i] = 1e-6
        assert abs((f(x, gain + e) - f(x, gain - e)) / 2e-6 - dg[i]) < 1e-6 * max(1, abs(dg[i]))


def test_autograd_runs_into_the_attention():
    """q, k of a projection, norm and rotation, then the attention, and back:
    the gradients are the handles' own."""
    from hstu_jagged_attention_02_gb300.attention import hstu_attention
    from hstu_jagged_attention_02_gb300.qk import QKProblem, hstu_qk_norm_rope, jagged_positions, rope_tables
    off = torch.tensor([0, 130, 130, 300], dtype=torch.int64, device="cuda")
    nt = torch.tensor([7, 0, 20], dtype=torch.int32, device="cuda")
    T, H, d = 300, 2, 128
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, 3 * H, d, generator=g).bfloat16().cuda().requires_grad_()
    gq, gk = ((1 + 0.2 * torch.randn(d, generator=g)).cuda().requires_grad_() for _ in range(2))
    u, dy = torch.randn(T, H * d, generator=g).bfloat16().cuda(), torch.randn(T, H * d, generator=g).cuda()
    pos = jagged_positions(off, nt)
    assert pos.tolist() == [min(i, 123) for i in range(130)] + [min(i, 150) for i in range(170)]
    cos, sin = rope_tables(300, d)
    q2, k2 = hstu_qk_norm_rope(x[:, :H], x[:, H:2 * H], pos, cos, sin, q_gain=gq, k_gain=gk)
    q2.retain_grad()
    k2.retain_grad()
    y = hstu_attention(q2, k2, x[:, 2 * H:], u, off, 170, d ** -0.5, num_targets=nt)
    y.backward(dy)
    pr = QKProblem(x.detach()[:, :H], x.detach()[:, H:2 * H], pos, cos, sin, q_gain=gq.detach(), k_gain=gk.detach(),
                   dq_out=q2.grad, dk_out=k2.grad)
    pr.forward()
    pr.backward()
    assert torch.equal(pr.q_out, q2.detach()) and torch.equal(pr.k_out, k2.detach())
    assert torch.equal(x.grad[:, :H], pr.dq) and torch.equal(x.grad[:, H:2 * H], pr.dk)
    assert torch.equal(gq.grad, pr.d_q_gain) and torch.equal(gk.grad, pr.d_k_gain)


def test_strides_in_place_and_padding():
    from hstu_jagged_attention_02_gb300.qk import QKProblem
    q, k, pos, cos, sin, gains, grads = _inputs(90, 3, 2, 64, 64, "bf16", True, seed=9)
    whole = QKProblem(q, k, pos, cos, sin, q_gain=gains[0], k_gain=gains[1], dq_out=grads[0], dk_out=grads[1])
    whole.forward()
    whole.backward()
    # [H, T, d] order, odd features (copied), in place
    qt = q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    odd = torch.zeros(90, 2, 67, dtype=torch.bfloat16, device="cuda")[..., 1:65]
    odd.copy_(k)
    a = QKProblem(qt, odd, pos, cos, sin, q_gain=gains[0], k_gain=gains[1])
    assert a.q is qt and a.k is not odd
    a.forward()
    assert torch.equal(a.q_out, whole.q_out) and torch.equal(a.k_out, whole.k_out)
    both = torch.cat([q, k], 1)
    b = QKProblem(both[:, :3], both[:, 3:], pos, cos, sin, q_gain=gains[0], k_gain=gains[1], inplace=True)
    b.forward()
    assert torch.equal(both, torch.cat([whole.q_out, whole.k_out], 1))
    # rows behind num_tokens are left as they are, and do not count
    n = torch.tensor([53], device="cuda")
    c = QKProblem(q, k, pos, cos, sin, q_gain=gains[0], k_gain=gains[1], dq_out=grads[0], dk_out=grads[1], num_tokens=n)
    first = QKProblem(q[:53], k[:53], pos[:53], cos, sin, q_gain=gains[0], k_gain=gains[1], dq_out=grads[0][:53],
                      dk_out=grads[1][:53])
    for t in (c.q_out, c.k_out, c.dq, c.dk):
        t.fill_(7.0)
    for pr in (c, first):
        pr.forward()
        pr.backward()
    for t, f in ((c.q_out, first.q_out), (c.k_out, first.k_out), (c.dq, first.dq), (c.dk, first.dk)):
        assert torch.equal(t[:53], f) and bool((t[53:] == 7.0).all())
    for t, f in ((c.d_q_gain, first.d_q_gain), (c.d_k_gain, first.d_k_gain)):
        assert torch.allclose(t, f, rtol=2e-6, atol=1e-5)
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    z = QKProblem(q, k, pos, cos, sin, q_gain=gains[0], k_gain=gains[1], dq_out=grads[0], dk_out=grads[1], num_tokens=zero)
    z.backward()
    assert not z.d_q_gain.any() and not z.d_k_gain.any()


def test_same_bits_every_time_and_in_a_graph():
    from hstu_jagged_attention_02_gb300.qk import QKProblem
    q, k, pos, cos, sin, gains, grads = _inputs(4000, 4, 4, 128, 128, "bf16", True, seed=11)
    pr = QKProblem(q, k, pos, cos, sin, q_gain=gains[0], k_gain=gains[1], dq_out=grads[0], dk_out=grads[1])

    def step():
        pr.forward()
        pr.backward()

    step()
    outs = (pr.q_out, pr.k_out, pr.dq, pr.dk, pr.d_q_gain, pr.d_k_gain)
    first = [t.clone() for t in outs]
    for _ in range(3):
        step()
        assert all(torch.equal(a, b) for a, b in zip(outs, first))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step()
    for t in outs:
        t.fill_(float("nan"))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, first))
    assert pr.device_error() == 0


def test_a_position_outside_the_tables_is_reported():
    from hstu_jagged_attention_02_gb300 import binding as C
    from hstu_jagged_attention_02_gb300.qk import QKProblem
    q, k, pos, cos, sin, gains, _ = _inputs(20, 2, 2, 64, 64, "bf16", True, seed=12)
    good = QKProblem(q, k, pos, cos, sin)
    good.forward()
    for bad in (300, -1):
        p2 = pos.clone()
        p2[13] = bad
        pr = QKProblem(q, k, p2, cos, sin)
        pr.forward()
        assert pr.device_error() == C.HSTU_ERR_DEVICE_CHECK
        keep = torch.arange(20, device="cuda") != 13
        assert torch.equal(pr.q_out[keep], good.q_out[keep])
    assert good.device_error() == 0
