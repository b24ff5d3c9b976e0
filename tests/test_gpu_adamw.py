"""AdamW over many tensors (hstu_adamw_*) against plain forms.

The moments are FP32 products and sums one by one, so NumPy's FP32 numbers are
the same bits; so are the 8-bit codes, whose rounding goes by given random
words.  Parameters: three roundings on p (2^-22 of it), and on what it moves by
an approximate square root and quotient and five products: 2^-19 of it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import training_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu

HYPER = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8)


def _tensors(sizes, seed, grad=torch.float32):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda n: torch.randn(n, generator=g)  # noqa: E731
    params = [(0.05 * rnd(n)).cuda() for n in sizes]
    grads = [(rnd(n) * torch.exp(2 * rnd(n))).to(grad).cuda() for n in sizes]
    return params, grads


def _np(t):
    return t.detach().float().cpu().numpy()


def _check_step(before, grads, opt, t, wd, scale=None, copies=None):
    """One step from the kept copies before = [(p, m, v)] FP32."""
    b1, b2 = HYPER["betas"]
    for i, ((p, m, v), g) in enumerate(zip(before, grads)):
        m2, v2 = R.moments(m, v, _np(g), b1, b2, scale)
        want, moved = R.adamw(p.astype(np.float64), m2.astype(np.float64), v2.astype(np.float64), t, HYPER["lr"], b1, b2,
                              HYPER["eps"], wd[i])
        got = _np(opt.params[i])
        assert np.all(np.abs(got - want) <= 2.0 ** -22 * np.abs(want) + 2.0 ** -19 * moved), i
        if copies is not None and copies[i] is not None:
            assert torch.equal(copies[i], opt.params[i].bfloat16())
        yield i, m2, v2


SIZES = [1, 7, 255, 256, 257, 2048, 2049, 5000, 4, 0, 70_001]


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [32, 8])
def test_steps(bits, grad):
    from hstu_jagged_attention_02_gb300.optim import AdamW
    params, grads = _tensors(SIZES, 1, grad)
    copies = [p.bfloat16() if i % 3 else None for i, p in enumerate(params)]
    wd = [0.1 if i % 2 else 0.0 for i in range(len(SIZES))]
    seed = 0xABCDEF0123456789
    opt = AdamW(params, grads, weight_decay=wd, copies=copies, state_bits=bits, seed=seed, **HYPER)
    g = torch.Generator().manual_seed(2)
    for t in range(1, 5):
        if bits == 32:
            before = [(_np(p), _np(m[0]), _np(m[1])) for p, m in zip(params, opt.moments)]
        else:
            dec = lambda c, e, k: R.decode(c.cpu().numpy(), e.cpu().numpy(), k).astype(np.float32)  # noqa: E731
            before = [(_np(p), dec(m.m, m.m_exp, "m"), dec(m.v, m.v_exp, "v")) for p, m in zip(params, opt.moments)]
        opt.step()
        block = 0
        for i, m2, v2 in _check_step(before, grads, opt, t, wd, copies=copies):
            now = opt.moments[i]
            if bits == 32:
                assert np.array_equal(_np(now[0]), m2) and np.array_equal(_np(now[1]), v2), i
            else:
                word = R.words(block, m2.size, t, seed)
                for x, codes, exps, kind in ((m2, now.m, now.m_exp, "m"), (v2, now.v, now.v_exp, "v")):
                    want, e = R.encode(x, word, kind)
                    assert np.array_equal(exps.cpu().numpy(), e), (i, kind)
                    assert np.array_equal(codes.cpu().numpy(), want), (i, kind)
            block += (m2.size + 255) // 256
        for x in grads:
            x.copy_(torch.randn(x.shape, generator=g).to(x.dtype))
    assert opt.steps() == 4 and opt.device_error() == 0


@pytest.mark.parametrize("sizes", [(8_000_003, 300_000), (1000, 33_000_001, 5)])
def test_long_lists(sizes):
    """Chunks of several blocks: codes, moments and parameters of some blocks of every tensor."""
    from hstu_jagged_attention_02_gb300.optim import AdamW
    for bits in (8, 32):
        params, grads = _tensors(sizes, 11)
        before = [p.clone() for p in params]
        opt = AdamW(params, grads, state_bits=bits, seed=77, **HYPER)
        opt.step()
        assert opt.device_error() == 0
        block, rng = 0, np.random.default_rng(1)
        for p, q, g, mom in zip(params, before, grads, opt.moments):
            blocks = (p.numel() + 255) // 256
            for k in sorted({0, blocks - 1, *rng.integers(0, blocks, 60).tolist()}):
                at = slice(k * 256, min(p.numel(), k * 256 + 256))
                zero = np.zeros(at.stop - at.start, np.float32)
                m, v = R.moments(zero, zero, _np(g[at]), 0.9, 0.999)
                want, moved = R.adamw(_np(q[at]).astype(np.float64), m.astype(np.float64), v.astype(np.float64), 1, 1e-3, 0.9,
                                      0.999, 1e-8, 0.0)
                assert np.all(np.abs(_np(p[at]) - want) <= 2.0 ** -22 * np.abs(want) + 2.0 ** -19 * moved)
                if bits == 32:
                    assert np.array_equal(_np(mom[0][at]), m) and np.array_equal(_np(mom[1][at]), v)
                    continue
                word = R.words(block + k, m.size, 1, 77)
                for x, codes, exps, kind in ((m, mom.m, mom.m_exp, "m"), (v, mom.v, mom.v_exp, "v")):
                    code, e = R.encode(x, word, kind)
                    assert np.array_equal(codes[at].cpu().numpy(), code) and int(exps[k]) == int(e[0])
            block += blocks


def test_8_bit_moments_keep_their_means():
    """Without gradients v decays by a thousandth a step, far below half a step of its format.  A
    value's rounding moves it by at most an eighth of itself with variance at most (1/16)^2 of it a step:
    over 200 steps and 65,536 elements the mean is off by less than 6 sqrt(200 / 65536) / 16 of itself."""
    from hstu_jagged_attention_02_gb300.optim import AdamW, zero_moments
    n, steps = 65_536, 200
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    gen = torch.Generator().manual_seed(3)
    mom = zero_moments(p, 8)
    mom.v.copy_(torch.randint(128, 240, (n,), generator=gen).to(torch.uint8))
    mom.m.copy_((torch.randint(60, 120, (n,), generator=gen)).to(torch.uint8))
    opt = AdamW([p], [g], lr=0.0, betas=(0.999, 0.999), moments=[mom], seed=5)
    before = [x.double().mean() for x in opt.read_moments()[0]]
    for _ in range(steps):
        opt.step()
    after = [x.double().mean() for x in opt.read_moments()[0]]
    for a, b in zip(after, before):
        assert abs(float(a / b) / 0.999 ** steps - 1) < 6 * (steps / n) ** 0.5 / 16


def test_values_read_back():
    from hstu_jagged_attention_02_gb300.optim import AdamW, zero_moments
    params = [torch.zeros(n, device="cuda") for n in (256, 300, 5000)]
    g = torch.Generator().manual_seed(4)
    moments = []
    for p in params:
        m = zero_moments(p, 8)
        for t in m[:2]:
            t.copy_(torch.randint(0, 256, t.shape, generator=g).to(torch.uint8))
        for t in m[2:]:
            t.copy_(torch.randint(60, 180, t.shape, generator=g).to(torch.uint8))
        moments.append(m)
    moments[0].m.copy_(torch.arange(256).to(torch.uint8))     # every code once
    moments[0].v.copy_(torch.arange(256).to(torch.uint8))
    opt = AdamW(params, [None] * 3, moments=moments)
    for dtype in (torch.float32, torch.bfloat16):
        for mom, (m, v) in zip(moments, opt.read_moments(dtype)):
            for kind, codes, exps, got in (("m", mom.m, mom.m_exp, m), ("v", mom.v, mom.v_exp, v)):
                want = R.decode(codes.cpu().numpy(), exps.cpu().numpy(), kind)
                assert np.array_equal(_np(got).astype(np.float64), want, equal_nan=True)
    # one of a pair, 32 bits
    opt = AdamW(params, [None] * 3, moments=[(torch.randn(p.numel(), device="cuda"), torch.rand(p.numel(), device="cuda"))
                                             for p in params])
    outs = [(torch.full_like(p, 3.0), None) for p in params]
    reader = opt.reader(outs)
    reader.run()
    assert all(torch.equal(o[0], m[0]) for o, m in zip(outs, opt.moments)) and reader.device_error() == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_wild_gradients(bits):
    """Zeros, subnormals, huge values, infinities and NaN: each stays with its element."""
    from hstu_jagged_attention_02_gb300.optim import AdamW
    params, grads = _tensors([1024, 300], 6)
    clean, quiet = _tensors([1024, 300], 6)
    at = [3, 260, 261, 700, 1000]
    for i, x in zip(at, (float("nan"), float("inf"), -float("inf"), 1e25, 1e-30)):
        grads[0][i] = x
    grads[1].zero_()
    quiet[1].zero_()
    a = AdamW(params, grads, state_bits=bits, **HYPER)
    b = AdamW(clean, quiet, state_bits=bits, **HYPER)
    for _ in range(2):
        a.step()
        b.step()
    keep = torch.tensor([i for i in range(1024) if i not in at], device="cuda")
    if bits == 32:
        assert torch.equal(params[0][keep], clean[0][keep])
    else:   # the blocks' powers of two may differ: the first step's parameters do not go by them
        assert bool(params[0][keep].isfinite().all())
    assert torch.equal(params[1], clean[1])
    assert bool(params[0][[3, 260, 261]].isnan().all()) and bool(params[0][[700, 1000]].isfinite().all())
    m, v = a.read_moments()[0]
    assert bool(m[[3, 260, 261]].isnan().all() if bits == 8 else not m[[3, 260, 261]].isfinite().any())
    assert bool(m[keep].isfinite().all()) and bool(v[keep].isfinite().all())
    assert all(not x.any() for x in a.read_moments()[1])


@pytest.mark.parametrize("bits", [32, 8])
def test_device_scalars_skips_and_graphs(bits):
    from hstu_jagged_attention_02_gb300.optim import AdamW
    sizes = [3000, 17, 512]
    params, grads = _tensors(sizes, 7)
    lr, scale = torch.tensor([1e-3], device="cuda"), torch.tensor([0.5], device="cuda")
    skip = torch.zeros(1, dtype=torch.int32, device="cuda")
    opt = AdamW(params, grads, lr=lr, betas=(0.9, 0.999), weight_decay=0.1, state_bits=bits, grad_scale=scale, skip=skip,
                seed=9, steps=41)
    other, half = _tensors(sizes, 7)
    for x in half:
        x.mul_(0.5)
    plain = AdamW(other, half, lr=1e-3, betas=(0.9, 0.999), weight_decay=0.1, state_bits=bits, seed=9, steps=41)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            opt.step()
    same = lambda: all(torch.equal(a, b) for a, b in zip(params, other)) and all(  # noqa: E731
        torch.equal(a, b) for x, y in zip(opt.moments, plain.moments) for a, b in zip(x, y))
    for k in range(3):
        graph.replay()
        plain.step()
        torch.cuda.synchronize()
        assert same(), k
    skip.fill_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert same() and opt.steps() == 44
    skip.zero_()
    lr.fill_(5e-4)
    plain.lr = 5e-4
    graph.replay()
    plain.step()
    torch.cuda.synchronize()
    assert same() and opt.steps() == plain.steps() == 45 and opt.device_error() == 0


def test_gradients_of_autograd():
    """Without a list the parameters' .grad of the moment counts; one without a gradient stays as it is."""
    from hstu_jagged_attention_02_gb300.optim import AdamW
    params, grads = _tensors([300, 40, 2048], 8)
    other, _ = _tensors([300, 40, 2048], 8)
    leaves = [p.requires_grad_() for p in params]
    opt = AdamW([p.detach() for p in leaves], [torch.zeros_like(p) for p in leaves], **HYPER)   # shares their memory
    opt = AdamW(leaves, None, **HYPER)
    ref = AdamW(other, grads, **HYPER)
    for _ in range(3):
        for p, g in zip(leaves, grads):
            p.grad = g.clone()
        opt.step()
        ref.step()
    assert all(torch.equal(a.detach(), b) for a, b in zip(leaves, other)) and opt.steps() == 3
    leaves[1].grad = None
    kept = leaves[1].detach().clone()
    opt.step()
    ref.step()
    assert torch.equal(leaves[1].detach(), kept) and torch.equal(leaves[2].detach(), other[2]) and opt.steps() == 4


def test_another_list_is_found():
    from hstu_jagged_attention_02_gb300 import binding as C
    from hstu_jagged_attention_02_gb300.optim import AdamW
    params, grads = _tensors([5000], 9)
    opt = AdamW(params, grads, **HYPER)
    before = params[0].clone()
    opt.desc.chunks -= 1
    opt.step()
    assert opt.device_error() == C.HSTU_ERR_DEVICE_CHECK and torch.equal(params[0], before)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            params[0].add_(0.0)
            # a list is laid out outside of captures: refused, and the capture goes on
            assert C.load().hstu_adamw_init(C.ctypes.byref(opt.desc), opt._table, opt.ws.data_ptr(), opt.ws_bytes,
                                            s.cuda_stream) == C.HSTU_ERR_INVALID_ARG
    graph.replay()
    torch.cuda.synchronize()


def test_a_step_that_raised_sends_the_list_with_the_next():
    from hstu_jagged_attention_02_gb300.optim import AdamW
    params, grads = _tensors([300, 2048], 11)
    other, _ = _tensors([300, 2048], 11)
    leaves = [p.requires_grad_() for p in params]
    opt, ref = AdamW(leaves, None, grad_dtype=torch.float32, **HYPER), AdamW(other, grads, **HYPER)
    for p, g in zip(leaves, grads):
        p.grad = g.clone()
    opt.step()
    ref.step()
    kept = leaves[1].grad
    leaves[0].grad = 2 * grads[0]
    leaves[1].grad = torch.zeros(2049, device="cuda")[1:]   # not 16-byte aligned
    with pytest.raises(ValueError):
        opt.step()
    assert opt.steps() == 1
    leaves[1].grad = kept
    opt.step()
    grads[0].mul_(2)
    ref.step()
    assert all(torch.equal(a.detach(), b) for a, b in zip(leaves, other)) and opt.steps() == 2
    leaves[0].data = leaves[0].data.clone()
    with pytest.raises(ValueError, match="is not where it was"):
        opt.step()
    assert opt.steps() == 2
