"""The workspace of the weight gradients of groups (host only): the counters'
place is the same for every shape and holds every cut tile; the partial sums of
one group suffice for any of its lengths."""
import ctypes

import numpy as np
import pytest

from hstu_jagged_attention_02_gb300 import binding as C

SHAPES = [(8, 8), (128, 256), (512, 512), (512, 2048), (264, 520), (640, 256), (1096, 4096)]


def _sizes(E, rows, K, N):
    d = C.hstu_group_desc()
    d.struct_size = ctypes.sizeof(d)
    d.groups, d.K, d.N, d.y_dtype, d.dx_dtype, d.rows = E, K, N, C.HSTU_BF16, C.HSTU_BF16, rows
    d.x_stride, d.y_stride, d.dx_stride = K, N, K
    return C.hstu_group_workspace_size(d)


def _cut(E, rows, K, N):
    """CTAs of a tile, tiles, and the longest piece in blocks of 64 rows, as the kernel cuts them."""
    halves, nt = -(-K // 128), -(-N // 256)
    pair = (rows // 64 + min(rows, E)) * -(-halves // 2) * nt >= 76 * 46 and (halves % 2 == 0 or halves >= 5)
    cg = 2 if pair else 1
    tiles, shares, blocks = -(-halves // cg) * nt, 152 // cg, -(-rows // 64)
    kper = max(8, int(np.ceil(2 * np.sqrt(blocks))), -(-blocks * tiles // shares))
    if E == 1:
        least, best = max(8, int(np.ceil(2 * np.sqrt(blocks)))), None
        for n in range(1, blocks + 1):
            if n * tiles > 2 * shares:
                break
            length = -(-blocks // n)
            cost = -(-n * tiles // shares) * (length + (8 if n > 1 else 0))
            if length >= least and (best is None or cost < best):
                best, kper = cost, length
    return cg, tiles, kper


@pytest.mark.parametrize("E", [1, 2, 9, 300, 4096])
def test_counters_hold_every_cut_tile(E):
    places = set()
    for rows in (1, 63, 64, 600, 5_000, 40_000, 161_293, 1_000_000):
        for K, N in SHAPES:
            fwd, ws, zero = _sizes(E, rows, K, N)
            places.add(zero)
            cg, tiles, kper = _cut(E, rows, K, N)
            cut = min(E, rows // (64 * kper + 1))     # a cut group has more rows than a piece holds
            assert 256 + cut * tiles * cg * 8 * 4 <= zero and fwd == 256
    assert len(places) == 1


def test_slots_of_one_group():
    for rows in (1, 600, 5_000, 40_000, 161_293, 1_000_000):
        for K, N in SHAPES:
            _, ws, zero = _sizes(1, rows, K, N)
            cg, tiles, kper = _cut(1, rows, K, N)
            slots = (ws - zero) // (4 * 128 * cg * 256)
            for n in {rows, rows // 2, min(rows, 64 * kper + 1), max(0, rows - 63)}:
                blocks = -(-n // 64)
                assert blocks <= kper or -(-blocks // kper) * tiles <= slots
