"""Appending to and reading from the paged 4-bit cache: every value held is
exactly the one that the definition gives in real arithmetic (64 bits here),
for raw keys and values (where ties are common) and for normed and rotated
keys."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import serving_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """n_b new tokens behind c_b cached ones, pages in random order."""

    def __init__(self, new, cached, H, d, page, seed, max_pages=None, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens = new, [a + b for a, b in zip(new, cached)]
        need = [-(-n // page) for n in self.lens]
        width = max(max(need), 1) if max_pages is None else max_pages
        order = torch.randperm(sum(need) + spare, generator=g).int()
        table, at = torch.full((len(new), width), -7, dtype=torch.int32), 0     # unused entries are no page
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.num_pages = sum(need) + spare
        T = sum(new)
        self.T = T
        self.k, self.v = (torch.randn(T, H, d, generator=g).bfloat16().cuda() for _ in range(2))
        self.times = (1_700_000_000 + torch.randint(0, 1 << 40, (T,), generator=g)).cuda()
        self.table = table.cuda()
        self.off = torch.tensor([0] + new).cumsum(0).cuda()
        self.cache_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.starts = torch.tensor(cached, dtype=torch.int32).cuda()
        self.pos = np.concatenate([np.arange(c, c + n) for c, n in zip(cached, new)]) if T else np.zeros(0, int)


def _cache(b, H, d, page, **kw):
    from hstu_jagged_attention_02_gb300.cache import PagedCache
    return PagedCache(b.num_pages, H=H, d=d, page_size=page, **kw)


@pytest.mark.parametrize("H,d,page", [(4, 128, 64), (3, 64, 32), (1, 128, 128), (5, 64, 64), (2, 128, 32)])
@pytest.mark.parametrize("new,cached", [([1], [0]), ([3, 0, 130, 1], [0, 5, 63, 64]), ([64, 65, 127], [1, 0, 31])])
def test_raw_keys_and_values_are_held_exactly(H, d, page, new, cached):
    from hstu_jagged_attention_02_gb300.cache import hstu_cache_append, hstu_cache_read
    b = Batch(new, cached, H, d, page, seed=7)
    c = _cache(b, H, d, page)
    hstu_cache_append(c, b.k, b.v, b.off, b.cache_lens, b.table, timestamps=b.times)
    k, v, t = hstu_cache_read(c, b.off, b.starts, b.table)
    np.testing.assert_array_equal(_f64(k), R.four_bit(_f64(b.k)))
    np.testing.assert_array_equal(_f64(v), R.four_bit(_f64(b.v)))
    assert torch.equal(t, b.times)


def test_the_bytes_of_a_page():
    # the layout in memory: K codes, K scales, V codes, V scales of each head, feature 2i in the low half
    from hstu_jagged_attention_02_gb300.cache import hstu_cache_append
    H, d, page = 2, 64, 32
    b = Batch([40], [0], H, d, page, seed=8)
    c = _cache(b, H, d, page)
    hstu_cache_append(c, b.k, b.v, b.off, b.cache_lens, b.table, timestamps=b.times)
    pages, table = c.pages.cpu().numpy(), b.table.cpu().numpy()
    lut = np.concatenate([R.E2M1, -R.E2M1])
    half = page * (d // 2 + d // 16)
    for x, at in ((b.k, 0), (b.v, half)):
        want = R.four_bit(_f64(x))
        for j in (0, 31, 32, 39):
            for h in range(H):
                part = pages[table[0, j // page], h, at:at + half]
                codes = part[:page * d // 2].reshape(page, d // 2)[j % page]
                scale = R.E4M3[part[page * d // 2:].reshape(page, d // 16)[j % page]]
                got = np.stack([lut[codes & 15], lut[codes >> 4]], 1).reshape(d) * np.repeat(scale, 16)
                np.testing.assert_array_equal(got, want[j, h])
    assert c.timestamps[int(table[0, 1]), 7] == b.times[39]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("norm,rot,inter,k_exp,v_exp", [
    (True, 1.0, False, 0, 0), (True, 0.5, True, -3, 2), (False, 1.0, True, 0, 0), (True, 0.0, False, 5, -5),
    (False, 0.125, False, 0, 0)])
def test_normed_and_rotated_keys_are_decided_as_real_numbers(d, norm, rot, inter, k_exp, v_exp):
    from hstu_jagged_attention_02_gb300.cache import hstu_cache_append, hstu_cache_read
    H, page, rot = 3, 64, int(rot * d)
    b = Batch([700, 1, 900], [0, 40, 77], H, d, page, seed=20 + d)
    c = _cache(b, H, d, page, k_exp=k_exp, v_exp=v_exp)
    gain = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(1))).cuda() if norm else None
    tab = R.rope_tables(1000, rot) if rot else None
    cos, sin = (torch.from_numpy(x).cuda() for x in tab) if rot else (None, None)
    hstu_cache_append(c, b.k, b.v, b.off, b.cache_lens, b.table, timestamps=b.times, cos=cos, sin=sin, rot_dim=rot,
                      interleaved=inter, norm=norm, eps=1e-5, k_gain=gain)
    k, v, _ = hstu_cache_read(c, b.off, b.starts, b.table)
    cs, sn = (x[b.pos] for x in tab) if rot else (np.ones((b.T, 0)), np.zeros((b.T, 0)))
    eps32 = float(np.float32(1e-5))
    want = R.qk_forward(_f64(b.k), None if gain is None else _f64(gain), cs, sn, inter, norm, eps32)
    np.testing.assert_array_equal(_f64(k), R.four_bit(want, k_exp))
    np.testing.assert_array_equal(_f64(v), R.four_bit(_f64(b.v), v_exp))


def test_borders_zeros_and_what_is_not_finite():
    from hstu_jagged_attention_02_gb300.cache import hstu_cache_append, hstu_cache_read
    H, d, page = 1, 64, 32
    b = Batch([16], [0], H, d, page, seed=3)
    x = np.zeros((16, 1, 64))
    steps = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, -5])
    for i in range(16):      # every border at several scales, positive and negative
        x[i, 0] = np.tile(steps, 4) * np.repeat([1.0, 2.0 ** (i - 8), -0.875, 1.125 * 2.0 ** -i], 16)
    x[3, 0, 0:16] = 0.0
    x[4, 0, 16:32] = 2.0 ** -12          # below half the smallest scale: zeros
    x[5, 0, 32:48] = 1e30                # above the largest: cut
    x[6, 0, 5], x[6, 0, 20], x[6, 0, 37] = np.nan, np.inf, -np.inf
    k = torch.from_numpy(x).bfloat16().cuda()
    c = _cache(b, H, d, page)
    hstu_cache_append(c, k, -k, b.off, b.cache_lens, b.table, timestamps=b.times)
    got, neg, _ = hstu_cache_read(c, b.off, b.starts, b.table)
    want = R.four_bit(np.clip(_f64(k), -1e38, 1e38))
    np.testing.assert_array_equal(_f64(got), want)
    np.testing.assert_array_equal(_f64(neg), -want)
    assert np.isnan(want[6, 0, :16]).all() and want[5, 0, 32] == 2688 and want[6, 0, 37] == -2688 and not want[4, 0, 16:32].any()


def test_only_its_places_are_written_and_padding_is_left():
    from hstu_jagged_attention_02_gb300.cache import AppendProblem, ReadProblem
    H, d, page = 2, 128, 32
    b = Batch([3, 33, 0], [30, 0, 9], H, d, page, seed=4, max_pages=5)
    c = _cache(b, H, d, page)
    c.pages.fill_(0xA5)
    c.timestamps.fill_(-1)
    # a batch padded to 50 rows
    pad = lambda t: torch.cat([t, t.new_zeros(50 - t.shape[0], *t.shape[1:])])  # noqa: E731
    pr = AppendProblem(c, pad(b.k), pad(b.v), b.off, b.cache_lens, b.table, timestamps=pad(b.times))
    pr.run()
    assert pr.device_error() == 0
    touched = torch.zeros(b.num_pages, page, dtype=torch.bool)
    table = b.table.cpu()
    for s, (n, L) in enumerate(zip(b.new, b.lens)):
        for j in range(L - n, L):
            touched[table[s, j // page], j % page] = True
    assert torch.equal((c.timestamps.cpu() != -1), touched)
    codes = c.pages[:, :, :page * d // 2].reshape(-1, H, page, d // 2).cpu()
    assert bool((codes.permute(0, 2, 1, 3)[~touched] == 0xA5).all())
    rd = ReadProblem(c, b.off, b.starts, b.table, total_tokens=50)
    rd.k.fill_(3.0)
    rd.timestamps.fill_(-5)
    rd.run()
    assert rd.device_error() == 0
    np.testing.assert_array_equal(_f64(rd.k)[:36], R.four_bit(_f64(b.k)))
    assert bool((rd.k[36:] == 3.0).all()) and bool((rd.timestamps[36:] == -5).all())


def test_many_sequences_and_a_graph():
    from hstu_jagged_attention_02_gb300.cache import AppendProblem, ReadProblem
    H, d, page = 1, 64, 32
    new = [(7 * i) % 4 for i in range(1500)]           # more sequences than one step of the search tells apart
    cached = [(13 * i) % 90 for i in range(1500)]
    b = Batch(new, cached, H, d, page, seed=5)
    c = _cache(b, H, d, page)
    wr = AppendProblem(c, b.k, b.v, b.off, b.cache_lens, b.table, timestamps=b.times)
    rd = ReadProblem(c, b.off, b.starts, b.table)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    wr.run()
    torch.cuda.synchronize()
    c.pages.zero_()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            wr.run()
            rd.run()
    graph.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(_f64(rd.k), R.four_bit(_f64(b.k)))
    assert torch.equal(rd.timestamps, b.times)
    assert wr.device_error() == 0 and rd.device_error() == 0


def test_strided_rows_without_times():
    from hstu_jagged_attention_02_gb300.cache import hstu_cache_append, hstu_cache_read
    H, d, page = 2, 64, 32
    b = Batch([45], [3], H, d, page, seed=6)
    both = torch.cat([b.k, b.v], 1)                     # side by side, as a projection leaves them
    c = _cache(b, H, d, page, timestamps=False)
    hstu_cache_append(c, both[:, :H], both[:, H:], b.off, b.cache_lens, b.table)
    k, v, t = hstu_cache_read(c, b.off, b.starts, b.table)
    assert t is None
    np.testing.assert_array_equal(_f64(k), R.four_bit(_f64(b.k)))
    np.testing.assert_array_equal(_f64(v), R.four_bit(_f64(b.v)))


@pytest.mark.parametrize("what", ["page", "length", "offsets", "rows", "position"])
def test_tables_that_do_not_fit_are_reported(what):
    from hstu_jagged_attention_02_gb300 import binding as C
    from hstu_jagged_attention_02_gb300.cache import AppendProblem
    H, d, page = 2, 64, 32
    b = Batch([5, 40], [0, 10], H, d, page, seed=9)
    c = _cache(b, H, d, page)
    cos, sin = (torch.from_numpy(x).cuda() for x in R.rope_tables(49 if what == "position" else 50, 64))
    if what == "page":
        b.table[1, 1] = b.num_pages
    elif what == "length":
        b.cache_lens[0] = 4                             # shorter than what is appended
    elif what == "offsets":
        b.off[2] = 46                                   # beyond the rows
    elif what == "rows":
        b.cache_lens[1] = 65                            # beyond the table's pages
    pr = AppendProblem(c, b.k, b.v, b.off, b.cache_lens, b.table, timestamps=b.times, cos=cos, sin=sin)
    pr.run()
    assert pr.device_error() == C.HSTU_ERR_DEVICE_CHECK
    pr.ws.zero_()
    assert pr.device_error() == 0


def test_many_keys_near_borders():
    """Enough normed and rotated keys that hundreds of rows hold a feature
    within 2^-20 of a border, where FP32 alone cannot tell the sides apart."""
    from hstu_jagged_attention_02_gb300.cache import hstu_cache_append, hstu_cache_read
    H, d, page, rot = 8, 128, 128, 128
    b = Batch([12000, 9000], [0, 0], H, d, page, seed=77)
    c = _cache(b, H, d, page, k_exp=1)
    gain = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(2))).cuda()
    tab = R.rope_tables(12000, rot)
    cos, sin = (torch.from_numpy(x).cuda() for x in tab)
    hstu_cache_append(c, b.k, b.v, b.off, b.cache_lens, b.table, timestamps=b.times, cos=cos, sin=sin, norm=True, eps=1e-5,
                      k_gain=gain)
    k, _, _ = hstu_cache_read(c, b.off, b.starts, b.table)
    want = R.qk_forward(_f64(b.k), _f64(gain), tab[0][b.pos], tab[1][b.pos], False, True, float(np.float32(1e-5)))
    np.testing.assert_array_equal(_f64(k), R.four_bit(want, 1))
