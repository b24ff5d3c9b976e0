"""Appending to the paged 4-bit cache at its edges: a token that has no place
among tokens that have one, infinities and products beyond FP32, tables whose
entries are larger than one.  What is held is compared bit by bit with the
64-bit form (tests/serving_ref.py), as in tests/test_gpu_cache.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import serving_ref as R  # noqa: E402
from tests.test_gpu_cache import Batch, _cache, _f64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("bad", ["table", "page"])
def test_a_token_without_a_place_costs_no_other_its_own(big, bad):
    """Sequences of two tokens, the first ones behind the rotation's tables or
    in a page that does not exist, next to valid ones: with many tokens a warp
    takes four neighbours, of several sequences."""
    from hstu_jagged_attention_02_gb300 import binding as C
    from hstu_jagged_attention_02_gb300.cache import AppendProblem, hstu_cache_read
    H, d, page = 2, 64, 64
    top = 7400 if big else 300                                    # rows of the tables
    new, cached = [2, 2, 3, 1, top - 8], [top - 1, 0, top, 5, 0]   # 0: one inside, one behind; 2: all behind
    b = Batch(new, cached, H, d, page, seed=60)
    c = _cache(b, H, d, page)
    c.timestamps.fill_(-1)
    tab = R.rope_tables(top if bad == "table" else top + 8, d)
    if bad == "page":       # the pages of the tokens that are behind the tables in the other case
        b.table[0, top // page], b.table[2, top // page] = b.num_pages, -1
        b.table[2, (top + 2) // page] = -1
    cos, sin = (torch.from_numpy(x).cuda() for x in tab)
    pr = AppendProblem(c, b.k, b.v, b.off, b.cache_lens, b.table, timestamps=b.times, cos=cos, sin=sin, norm=True, eps=1e-5)
    pr.run()
    assert pr.device_error() == C.HSTU_ERR_DEVICE_CHECK
    # the tokens whose position and page exist, read back one sequence at a time
    off, kept = b.off.tolist(), 0
    for s in range(len(new)):
        good = [i for i in range(new[s]) if cached[s] + i < top] if bad == "table" else \
            [i for i in range(new[s]) if 0 <= int(b.table[s, (cached[s] + i) // page]) < b.num_pages]
        if not good:
            continue
        assert good == list(range(len(good)))
        n = len(good)
        k, v, t = hstu_cache_read(c, torch.tensor([0, n]).cuda(), b.starts[s:s + 1].contiguous(), b.table[s:s + 1].contiguous())
        r = slice(off[s], off[s] + n)
        at = np.arange(cached[s], cached[s] + n)
        want = R.qk_forward(_f64(b.k[r]), None, tab[0][at], tab[1][at], False, True, float(np.float32(1e-5)))
        np.testing.assert_array_equal(_f64(k), R.four_bit(want), err_msg=f"keys of {s}")
        np.testing.assert_array_equal(_f64(v), R.four_bit(_f64(b.v[r])), err_msg=f"values of {s}")
        assert torch.equal(t, b.times[r])
        kept += n
    # and nothing else was written: sequence 0 keeps its first, 2 nothing
    assert int((c.timestamps != -1).sum()) == kept


@pytest.mark.parametrize("d,rot,inter", [(64, 32, False), (128, 64, True), (128, 8, False), (64, 16, True), (128, 32, False)])
def test_infinite_keys_that_are_turned(d, rot, inter):
    # an infinity goes in as the largest code of the largest scale, in a feature that is turned as in one that is not;
    # where the turn itself has no value (infinity less infinity, infinity times zero) the group is NaN
    from hstu_jagged_attention_02_gb300.cache import hstu_cache_append, hstu_cache_read
    H, page, n = 3, 32, 40
    b = Batch([n], [0], H, d, page, seed=61)
    c = _cache(b, H, d, page)
    x = _f64(b.k)
    g = np.random.default_rng(62)
    for t in range(1, n):
        x[t, t % H, g.integers(0, d)] = np.inf if t % 2 else -np.inf
        if t % 5 == 0:
            x[t, t % H, g.integers(0, d)] = np.nan
    x[3, :, 0], x[3, :, rot // 2] = np.inf, np.inf          # both of a pair of halves
    x[7, :, 0], x[7, :, 1] = -np.inf, np.inf                # both of a pair of neighbours
    k = torch.from_numpy(x).bfloat16().cuda()
    tab = R.rope_tables(n, rot)
    cos, sin = (torch.from_numpy(z).cuda() for z in tab)
    hstu_cache_append(c, k, b.v, b.off, b.cache_lens, b.table, timestamps=b.times, cos=cos, sin=sin, interleaved=inter)
    got, _, _ = hstu_cache_read(c, b.off, b.starts, b.table)
    with np.errstate(invalid="ignore"):
        want = R.four_bit(R.turn(_f64(k), tab[0], tab[1], inter))
    assert np.isnan(want).any() and (np.abs(want) == 2688.0).any() and not np.isnan(want[1]).all()
    np.testing.assert_array_equal(_f64(got), want)


@pytest.mark.parametrize("rot,k_exp", [(32, -32), (64, -32), (64, 0), (64, 32)])
def test_keys_near_the_types_end(rot, k_exp):
    # magnitudes up to 2^126: the power of two alone would take them beyond FP32, the result is the largest code
    from hstu_jagged_attention_02_gb300.cache import hstu_cache_append, hstu_cache_read
    H, d, page, n = 2, 64, 32, 64
    b = Batch([n], [0], H, d, page, seed=63)
    c = _cache(b, H, d, page, k_exp=k_exp)
    e = torch.randint(60, 126, (n, H, d // 16, 1), generator=torch.Generator().manual_seed(64)).double()
    k = (b.k.double().cpu().clamp(-1.9, 1.9).view(n, H, d // 16, 16) * 2.0 ** e).view(n, H, d).bfloat16().cuda()
    tab = R.rope_tables(n, rot)
    cos, sin = (torch.from_numpy(z).cuda() for z in tab)
    hstu_cache_append(c, k, b.v, b.off, b.cache_lens, b.table, timestamps=b.times, cos=cos, sin=sin)
    got, _, _ = hstu_cache_read(c, b.off, b.starts, b.table)
    np.testing.assert_array_equal(_f64(got), R.four_bit(R.turn(_f64(k), tab[0], tab[1], False), k_exp))


@pytest.mark.parametrize("factor,k_exp,inter", [(16.0, 5, False), (100.0, 7, True), (1.25, 1, False)])
def test_tables_with_entries_above_one(factor, k_exp, inter):
    """Cosines and sines that carry a factor (as schemes for longer contexts
    fold one in): the features near a border grow with it, and are decided all
    the same."""
    from hstu_jagged_attention_02_gb300.cache import hstu_cache_append, hstu_cache_read
    H, d, page, n = 8, 128, 128, 12000
    b = Batch([n], [0], H, d, page, seed=65)
    c = _cache(b, H, d, page, k_exp=k_exp)
    gain = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(66))).cuda()
    tab = [(x * np.float32(factor)).astype(np.float32) for x in R.rope_tables(n, d)]
    cos, sin = (torch.from_numpy(x).cuda() for x in tab)
    hstu_cache_append(c, b.k, b.v, b.off, b.cache_lens, b.table, timestamps=b.times, cos=cos, sin=sin, norm=True, eps=1e-5,
                      k_gain=gain, interleaved=inter)
    k, _, _ = hstu_cache_read(c, b.off, b.starts, b.table)
    want = R.qk_forward(_f64(b.k), _f64(gain), tab[0], tab[1], inter, True, float(np.float32(1e-5)))
    np.testing.assert_array_equal(_f64(k), R.four_bit(want, k_exp))
