"""What layer norm, the products of groups and AdamW refuse on the host: the C
entries (they return before any CUDA call) and the Python classes' checks of
their tensors; and the plain forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

from hstu_jagged_attention_02_gb300 import binding as C
from tests import training_ref as R

torch = pytest.importorskip("torch")

BAD, NOT, WS = C.HSTU_ERR_INVALID_ARG, C.HSTU_ERR_UNSUPPORTED, C.HSTU_ERR_WORKSPACE
PTR = 1 << 20          # stands for a device address: nothing is read before the checks are through


def _status(fn, *args):
    try:
        fn(*args)
    except C.HSTUError as e:
        return e.status
    return 0


def _with(x, kw):
    for name, value in kw.items():
        setattr(x, name, value)
    return x


def _full(cls, **kw):
    a = cls()
    for name, _ in cls._fields_:
        setattr(a, name, PTR)
    return _with(a, kw)


def _ln(**kw):
    d = C.hstu_ln_desc()
    d.struct_size = ctypes.sizeof(d)
    d.x_dtype, d.y_dtype, d.D, d.eps, d.rows = C.HSTU_BF16, C.HSTU_FP32, 64, 1e-5, 10
    d.x_stride = d.y_stride = d.dx_stride = d.dres_stride = 64
    return _with(d, kw)


@pytest.mark.parametrize("kw,status", [
    (dict(struct_size=8), BAD), (dict(reserved=1), BAD), (dict(x_dtype=2), BAD), (dict(y_dtype=-1), BAD), (dict(D=0), BAD),
    (dict(rows=-1), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(D=16385), NOT), (dict(rows=1 << 31), NOT),
])
def test_ln_descriptions(kw, status):
    d = _ln(**kw)
    assert _status(C.hstu_ln_workspace_size, d) == status
    assert _status(C.hstu_ln_fwd, d, _full(C.hstu_ln_fwd_args), PTR, 1 << 30, 0) == status
    assert _status(C.hstu_ln_bwd, d, _full(C.hstu_ln_bwd_args), PTR, 1 << 30, 0) == status


@pytest.mark.parametrize("bwd,kw,ws,status", [
    (0, dict(x=None), (PTR, 256), BAD), (0, dict(y=None), (PTR, 256), BAD), (0, dict(x=PTR + 1), (PTR, 256), BAD),
    (0, dict(y=PTR + 2), (PTR, 256), BAD), (0, dict(bias=PTR + 2), (PTR, 256), BAD), (0, {}, (0, 256), WS),
    (0, {}, (PTR + 128, 256), WS), (0, {}, (PTR, 255), WS),
    (1, dict(dy=None), (PTR, 1 << 30), BAD), (1, dict(mean=None), (PTR, 1 << 30), BAD), (1, dict(dx=None), (PTR, 1 << 30), BAD),
    (1, dict(dres=PTR + 1), (PTR, 1 << 30), BAD), (1, dict(d_weight=PTR + 2), (PTR, 1 << 30), BAD), (1, {}, (PTR, 256), WS),
])
def test_ln_calls(bwd, kw, ws, status):
    fn, cls = (C.hstu_ln_bwd, C.hstu_ln_bwd_args) if bwd else (C.hstu_ln_fwd, C.hstu_ln_fwd_args)
    assert _status(fn, _ln(), _full(cls, **kw), *ws, 0) == status


def _group(**kw):
    d = C.hstu_group_desc()
    d.struct_size = ctypes.sizeof(d)
    d.groups, d.K, d.N, d.y_dtype, d.dx_dtype, d.rows = 3, 64, 128, C.HSTU_BF16, C.HSTU_FP32, 100
    d.x_stride, d.y_stride, d.dx_stride = 64, 128, 64
    return _with(d, kw)


@pytest.mark.parametrize("kw,status", [
    (dict(struct_size=8), BAD), (dict(reserved=1), BAD), (dict(flags=1), BAD), (dict(y_dtype=5), BAD), (dict(dx_dtype=-1), BAD),
    (dict(groups=0), BAD), (dict(K=0), BAD), (dict(N=-8), BAD), (dict(rows=-1), BAD), (dict(groups=4097), NOT),
    (dict(K=63), NOT), (dict(N=132), NOT), (dict(K=65544), NOT), (dict(rows=(1 << 30) + 1), NOT),
    (dict(K=65536, N=65536, rows=1 << 30), NOT),
])
def test_group_descriptions(kw, status):
    d = _group(**kw)
    assert _status(C.hstu_group_workspace_size, d) == status
    assert _status(C.hstu_group_fwd, d, _full(C.hstu_group_fwd_args), PTR, 1 << 40, 0) == status
    assert _status(C.hstu_group_bwd, d, _full(C.hstu_group_bwd_args), PTR, 1 << 40, 0) == (status if "flags" not in kw else BAD)


@pytest.mark.parametrize("bwd,desc,kw,ws,status", [
    (0, {}, dict(group_offsets=None), (PTR, 256), BAD), (0, {}, dict(w=None), (PTR, 256), BAD),
    (0, {}, dict(x=PTR + 8), (PTR, 256), BAD), (0, {}, dict(y=PTR + 4), (PTR, 256), BAD),
    (0, dict(x_stride=68), {}, (PTR, 256), BAD), (0, dict(x_stride=56), {}, (PTR, 256), BAD),
    (0, dict(y_stride=132), {}, (PTR, 256), BAD), (0, {}, {}, (0, 256), WS), (0, {}, {}, (PTR, 128), WS),
    (0, {}, {}, (PTR + 16, 256), WS),
    (1, {}, dict(dx=None, dw=None), (PTR, 1 << 30), BAD), (1, {}, dict(dy=None), (PTR, 1 << 30), BAD),
    (1, {}, dict(w=None), (PTR, 1 << 30), BAD), (1, {}, dict(x=None), (PTR, 1 << 30), BAD),
    (1, {}, dict(dw=PTR + 4), (PTR, 1 << 30), BAD), (1, dict(dx_stride=60), {}, (PTR, 1 << 30), BAD),
    (1, dict(flags=2), {}, (PTR, 1 << 30), NOT), (1, dict(rows=10_000_000), {}, (PTR, 256), WS),
])
def test_group_calls(bwd, desc, kw, ws, status):
    fn, cls = (C.hstu_group_bwd, C.hstu_group_bwd_args) if bwd else (C.hstu_group_fwd, C.hstu_group_fwd_args)
    assert _status(fn, _group(**desc), _full(cls, **kw), *ws, 0) == status


@pytest.mark.parametrize("E", [2, 7, 60])
def test_slots_hold_every_split(E):
    """The workspace's partial sums suffice for any offsets: pieces as the kernel cuts them."""
    rng = np.random.default_rng(E)
    for rows in (1, 600, 5000, 40_000, 300_000):
        for K, N in ((8, 8), (128, 256), (512, 2048), (264, 520), (640, 256)):
            _, ws, zero = C.hstu_group_workspace_size(_group(groups=E, K=K, N=N, rows=rows, x_stride=K, y_stride=N, dx_stride=K))
            halves, nt = -(-K // 128), -(-N // 256)
            pair = (rows // 64 + min(rows, E)) * -(-halves // 2) * nt >= 3496 and (halves % 2 == 0 or halves >= 5)
            cg = 2 if pair else 1
            slots = (ws - zero) // (4 * 128 * cg * 256)
            tiles = -(-halves // cg) * nt
            kper = max(8, int(np.ceil(2 * np.sqrt(-(-rows // 64)))), -(-(-(-rows // 64) * tiles) // (152 // cg)))
            for k in range(20):
                share = rng.random(E) ** (10 if k % 2 else 1)
                n = np.floor(rows * share / share.sum()).astype(int)
                blocks = -(-n // 64)
                if k == 0:   # one block more than a piece holds, as often as there are rows for it
                    n = [min(kper * 64 + 1, max(0, rows - i * (kper * 64 + 1))) for i in range(E)]
                    blocks = np.array([-(-x // 64) for x in n])
                pieces = [-(-b // kper) if b > kper else 0 for b in blocks]
                assert sum(pieces) * tiles <= slots
                assert 256 + sum(1 for x in pieces if x) * tiles * cg * 8 * 4 <= zero


def _adamw(**kw):
    d = C.hstu_adamw_desc()
    d.struct_size = ctypes.sizeof(d)
    d.state_bits, d.grad_dtype, d.num_tensors = 8, C.HSTU_FP32, 1
    d.lr, d.beta1, d.beta2, d.eps = 1e-3, 0.9, 0.999, 1e-8
    return _with(d, kw)


def _tensor(**kw):
    t = (C.hstu_adamw_tensor * 1)()
    t[0] = C.hstu_adamw_tensor(*[PTR] * 7, 1000, 0.1, 1.0)
    _with(t[0], kw)
    return t


@pytest.mark.parametrize("kw,status", [
    (dict(struct_size=8), BAD), (dict(state_bits=16), BAD), (dict(grad_dtype=3), BAD), (dict(num_tensors=-1), BAD),
    (dict(beta1=1.0), BAD), (dict(beta2=-0.1), BAD), (dict(beta2=float("nan")), BAD), (dict(eps=0.0), BAD),
    (dict(lr=float("inf")), BAD), (dict(lr=-1.0), BAD), (dict(steps_done=-2), BAD),
])
def test_adamw_descriptions(kw, status):
    d = _adamw(**kw)
    assert _status(C.hstu_adamw_workspace_size, d, _tensor()) == status
    assert _status(C.hstu_adamw_init, d, _tensor(), PTR, 1 << 30, 0) == status
    assert _status(C.hstu_adamw_step, d, C.hstu_adamw_step_args(), PTR, 1 << 30, 0) == status


@pytest.mark.parametrize("kw,status", [
    (dict(param=None), BAD), (dict(param=PTR + 4), BAD), (dict(grad=PTR + 8), BAD), (dict(copy=PTR + 4), BAD), (dict(m=None), BAD),
    (dict(v=PTR + 2), BAD), (dict(m_exp=None), BAD), (dict(n=-1), BAD), (dict(n=(1 << 44) + 1), NOT),
    (dict(weight_decay=-1.0), BAD), (dict(lr_scale=float("nan")), BAD),
])
def test_adamw_tensors(kw, status):
    assert _status(C.hstu_adamw_init, _adamw(), _tensor(**kw), PTR, 1 << 50, 0) == status


def test_adamw_workspaces():
    # a record of 80 bytes a chunk, of a block where there are few of them, of up to 8
    assert C.hstu_adamw_workspace_size(_adamw(), _tensor()) == 256 + 4 * 80
    assert C.hstu_adamw_workspace_size(_adamw(), _tensor(n=2049)) == 256 + 9 * 80
    assert C.hstu_adamw_workspace_size(_adamw(), _tensor(n=1 << 30)) == 256 + (1 << 19) * 80
    assert C.hstu_adamw_workspace_size(_adamw(num_tensors=0), None) == 256
    for ws in ((0, 1 << 20), (PTR + 128, 1 << 20), (PTR, 256)):
        assert _status(C.hstu_adamw_init, _adamw(), _tensor(), *ws, 0) == WS
        assert _status(C.hstu_adamw_step, _adamw(chunks=1), C.hstu_adamw_step_args(), *ws, 0) == WS
        assert _status(C.hstu_adamw_read, _adamw(chunks=1), *ws, 0) == WS
    assert _status(C.hstu_adamw_step, _adamw(), C.hstu_adamw_step_args(lr=PTR + 1), PTR, 1 << 20, 0) == BAD
    assert _status(C.hstu_adamw_read_init, _adamw(), _tensor(), (C.hstu_adamw_moments * 1)(), 4, PTR, 1 << 20, 0) == BAD
    assert _status(C.hstu_adamw_steps, None, 0) == BAD


def test_python_checks():
    from hstu_jagged_attention_02_gb300.groups import GroupProblem, group_rows
    from hstu_jagged_attention_02_gb300.norm import LNProblem
    from hstu_jagged_attention_02_gb300.optim import AdamW, Moments8, zero_moments
    z, bf = torch.zeros, torch.bfloat16
    x, w = z(10, 64), z(64)
    for args, kw in (((z(10),), {}), ((z(10, 64, dtype=torch.float16),), {}), ((x, z(63)), {}), ((x, w.bfloat16()), {}),
                     ((x, w), dict(out_dtype=torch.float16)), ((x, w), dict(dy=z(10, 63))), ((x, w), dict(mean=z(10))),
                     ((x, w), dict(y=z(64, 10).t())), ((x, w), dict(y=z(1, 64).expand(10, 64))), ((x, w), dict(dres=x)),
                     ((x, w), dict(num_rows=z(2, dtype=torch.int64))), ((x, z(64, device="meta")), {}), ((x, w), {})):
        with pytest.raises(ValueError):       # the last of them: tensors that are not on a GPU
            LNProblem(*args, **kw)
    a, b, off = z(10, 64, dtype=bf), z(3, 64, 128, dtype=bf), z(4, dtype=torch.int64)
    for args, kw in (((x, b, off), {}), ((a, b.float(), off), {}), ((a, z(3, 65, 128, dtype=bf), off), {}),
                     ((a, b, off[:3]), {}), ((a, b, off.int()), {}), ((a, b.transpose(1, 2).contiguous().transpose(1, 2), off), {}),
                     ((a, b, off), dict(dy=z(10, 64, dtype=bf))), ((a, b, off), dict(dy=z(10, 128))),
                     ((a, b, off), dict(y=z(10, 132, dtype=bf)[:, 2:130])), ((a, b, off), dict(out_dtype=torch.float16)),
                     ((a, b, off), {})):
        with pytest.raises(ValueError):
            GroupProblem(*args, **kw)
    with pytest.raises(C.HSTUError):
        GroupProblem(z(10, 60, dtype=bf), z(3, 60, 128, dtype=bf), off)
    with pytest.raises(ValueError):
        group_rows(torch.tensor([0, 3, 1]), 3)
    order, offsets = group_rows(torch.tensor([2, 0, 2, 1, 0]), 4)
    assert order.tolist() == [1, 4, 3, 0, 2] and offsets.tolist() == [0, 2, 3, 5, 5]
    p, g = z(100), z(100)
    buf = z(200)
    for args, kw in ((([], []), {}), (([p.bfloat16()], [g]), {}), (([p], [z(99)]), {}), (([p], [g, g]), {}),
                     (([z(10, 10).t()], [g]), {}), (([p, z(8)], [g, z(8, dtype=bf)]), {}), (([p], [g]), dict(copies=[p])),
                     (([p, p], [g, g]), {}), (([buf[:104], buf[100:]], [z(104), z(100)]), {}), (([buf[1:101]], [g]), {}),
                     (([p], [g]), dict(moments=[(z(100), z(99))])), (([p], [g]), dict(moments=[(g.int(), g)])),
                     (([p, z(8)], [g, z(8)]), dict(moments=[zero_moments(p, 8), zero_moments(z(8))])),
                     (([p], [g]), dict(moments=[Moments8(*zero_moments(p, 8)[:3], z(2, dtype=torch.uint8))])),
                     (([p], [g]), dict(weight_decay=[0.1, 0.2])), (([p], [g]), dict(lr=z(2))), (([p], [g]), dict(steps=-1)),
                     (([p], [g]), dict(state_bits=16)), (([p], [g]), dict(skip=z(1))), (([p], [g]), {})):
        with pytest.raises((ValueError, C.HSTUError)):
            AdamW(*args, **kw)


def test_random_words():
    # the generator's published test vectors
    zero = R.philox4x32(np.zeros((1, 4), np.uint64), (0, 0))[0]
    assert [int(x) for x in zero] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = R.philox4x32(np.full((1, 4), 0xFFFFFFFF, np.uint64), (0xFFFFFFFF, 0xFFFFFFFF))[0]
    assert [int(x) for x in ones] == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


@pytest.mark.parametrize("kind", ["m", "v"])
def test_8_bit_codes(kind):
    # values that the format holds stay; others go to a neighbour, up as often as the mean asks for
    rng = np.random.default_rng(1)
    word = rng.integers(0, 1 << 32, 256, dtype=np.uint64)
    have = R.values(kind)
    have = have[np.isfinite(have)] * 2.0 ** -20
    codes, exps = R.encode(np.resize(have, 256).astype(np.float32), word, kind)
    held = R.decode(codes, exps, kind)
    # 448 and what lies above the least exponent's reach: the block's unit may be twice as large as needed
    assert np.mean(held == np.resize(have, 256)) > 0.9
    x = np.full(1 << 16, 1.3, np.float32)
    x[::256] = 1.9
    codes, exps = R.encode(x, R.words(0, x.size, 7, 99), kind)
    got = R.decode(codes, exps, kind)
    rest = np.arange(x.size) % 256 != 0
    assert set(np.unique(got[rest])) == {1.25, 1.375}
    # a standard deviation of the mean is 0.061 / 255
    assert abs(got[rest].mean() - 1.3) < 6 * 0.061 / 255
