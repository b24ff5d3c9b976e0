"""Outputs of the training block's handles that share memory with what their
call reads, in part or with other strides, are refused on the host; the same
rows where the kernel allows it, and columns of one buffer, are not."""
import random

import pytest

torch = pytest.importorskip("torch")

from hstu_jagged_attention_02_gb300.groups import GroupProblem  # noqa: E402
from hstu_jagged_attention_02_gb300.norm import LNProblem  # noqa: E402

BF = torch.bfloat16


def _bytes(t):
    at, size = t.data_ptr(), t.element_size()
    place = (t.stride(0) * torch.arange(t.shape[0])[:, None] + t.stride(1) * torch.arange(t.shape[1])).reshape(-1) * size + at
    return {b for p in place.tolist() for b in range(p, p + size)}


def test_touch_by_every_byte():
    from hstu_jagged_attention_02_gb300.norm import _touch
    rng, buf = random.Random(1), torch.zeros(4096, dtype=torch.uint8)
    for _ in range(600):
        pair = []
        for _ in range(2):
            dt, size = rng.choice([(torch.float32, 4), (BF, 2)])
            rows, width = rng.choice([1, 2, 3, 7, 20]), rng.choice([1, 2, 5, 8])
            pitch = rng.choice([width, width + 1, width + 8, 24, 31, 32])
            whole = buf.view(dt)
            span = pitch * (rows - 1) + width
            if span > whole.numel():
                continue
            pair.append(whole.as_strided((rows, width), (pitch, 1), rng.randrange(min(whole.numel() - span, 200) + 1)))
        if len(pair) == 2:
            assert _touch(*pair) == _touch(*pair[::-1]) == bool(_bytes(pair[0]) & _bytes(pair[1]))
    assert not _touch(buf[:0], buf) and not _touch(None, buf) and _touch(buf[:1], buf) and not _touch(buf[:8], buf[8:])
    assert _touch(buf[:40].view(1, 40).expand(5, 40), buf[39:50]) and not _touch(buf[:40].view(1, 40).expand(5, 40), buf[40:50])


def _refused(match, cls, *args, **kw):
    with pytest.raises(ValueError, match=match):
        cls(*args, **kw)


# (a call that is not refused goes on to the device, which is missing here)
def test_group_outputs():
    w, off = torch.zeros(2, 64, 64, dtype=BF), torch.zeros(3, dtype=torch.int64)
    buf = torch.zeros(12 * 64, dtype=BF)
    x, y = buf[:640].view(10, 64), buf[64:704].view(10, 64)
    dy = torch.zeros(10, 64, dtype=BF)
    _refused("y shares memory with x", GroupProblem, x, w, off, y=y)
    _refused("y shares memory with w", GroupProblem, dy, w, off, y=w.view(128, 64)[3:13])
    _refused("dx shares memory with dy", GroupProblem, dy, w, off, dy=x, dx=y)
    _refused("dx shares memory with x", GroupProblem, x, w, off, dy=dy, dx=y)
    both = torch.zeros(2 * 64 * 64 + 1000)
    _refused("dx shares memory with dw", GroupProblem, dy, w, off, dy=dy.clone(), dw=both[:8192].view(2, 64, 64),
             dx=both[8128:8768].view(10, 64))
    wide = torch.zeros(10, 192, dtype=BF)
    _refused("y shares memory with x", GroupProblem, wide[:, :64], w, off, y=wide[:, 56:120])
    _refused("y shares memory with x", GroupProblem, wide.view(20, 96)[:10, :64], w, off, y=wide[:, 128:])
    _refused("CUDA", GroupProblem, wide[:, :64], w, off, y=wide[:, 64:128], dy=wide[:, 128:], dx=dy)
    _refused("CUDA", GroupProblem, dy, w, off, dy=x, y=torch.zeros(10, 64, dtype=BF), dx=torch.zeros(10, 64, dtype=BF))


def test_norm_outputs():
    buf = torch.zeros(12 * 64)
    x, y, v = buf[:640].view(10, 64), buf[64:704].view(10, 64), torch.zeros(64)
    dy = torch.zeros(10, 64)
    _refused("y shares memory with x", LNProblem, x, v, v, y=y)
    wide = torch.zeros(20, 64)
    _refused("y shares memory with x, and is not the same rows", LNProblem, wide[:10], v, v, y=wide.view(10, 128)[:, :64])
    _refused("y shares memory with weight", LNProblem, dy, buf[600:664], v, y=x)
    m = torch.zeros(20)
    _refused("mean shares memory with rstd", LNProblem, x, v, v, mean=m[:10], rstd=m[5:15])
    _refused("rstd shares memory with x", LNProblem, x, v, v, mean=m[:10], rstd=buf[:10])
    _refused("dx shares memory with dy", LNProblem, torch.zeros(10, 64), v, v, dy=x, dx=y)
    _refused("dx shares memory with dy", LNProblem, torch.zeros(10, 64), v, v, dy=buf[:320].view(BF).view(10, 64), dx=x)
    _refused("dx shares memory with dres", LNProblem, torch.zeros(10, 64), v, v, dy=dy, dres=x, dx=y)
    _refused("dx shares memory with mean", LNProblem, torch.zeros(10, 64), v, v, dy=dy, mean=buf[5:15], rstd=m[:10], dx=x)
    for kw in (dict(dy=x, dx=x), dict(dy=dy, dres=x, dx=x)):
        _refused("CUDA", LNProblem, torch.zeros(10, 64), v, v, **kw)
    _refused("CUDA", LNProblem, x, v, v, dy=dy, dx=x)
    _refused("CUDA", LNProblem, x, v, v, y=x)
    wide = torch.zeros(10, 128)
    _refused("CUDA", LNProblem, wide[:, :64], v, v, y=wide[:, 64:], dy=dy, dx=dy)
