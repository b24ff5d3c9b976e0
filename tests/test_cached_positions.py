"""Positions of rows over the paged cache: the newest history tokens have the
places that appending gave them, candidates the one behind the cache; and a
whole step with rows of both kinds in one batch."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from hstu_jagged_attention_02_gb300.qk import cached_positions, jagged_positions  # noqa: E402
from tests import serving_ref as R  # noqa: E402


def test_positions_of_history_rows_and_candidates():
    off = torch.tensor([0, 5, 5, 8, 9])
    lens, nt = torch.tensor([40, 7, 20, 3], dtype=torch.int32), torch.tensor([2, 0, 3, 0], dtype=torch.int32)
    got = cached_positions(off, lens, nt)
    assert got.dtype == torch.int32 and got.tolist() == [37, 38, 39, 40, 40, 20, 20, 20, 2]
    # no candidates: the last positions; a padded batch: as many rows as asked for
    assert cached_positions(off, lens).tolist() == [35, 36, 37, 38, 39, 17, 18, 19, 2]
    assert cached_positions(off, lens, nt, total_tokens=12).tolist()[:9] == got.tolist()
    # a first pass: the whole history is new
    assert cached_positions(torch.tensor([0, 4]), torch.tensor([3], dtype=torch.int32),
                            torch.tensor([1], dtype=torch.int32)).tolist() == [0, 1, 2, 3]
    # candidates alone: behind the cache
    assert cached_positions(off, lens, off[1:] - off[:-1]).tolist() == \
        jagged_positions(off, off[1:] - off[:-1], starts=lens).tolist()
    assert cached_positions(torch.tensor([0, 0]), lens[:1]).tolist() == []


@pytest.mark.gpu
def test_a_step_with_new_tokens_and_candidates():
    """Norm and rotation by these positions, append, attend: the queries and the
    cached keys against the 64-bit forms at positions written out by hand, and
    the attention on them."""
    from hstu_jagged_attention_02_gb300.cache import PagedCache, hstu_attention_cached, hstu_cache_append, hstu_cache_read
    from hstu_jagged_attention_02_gb300.qk import hstu_qk_norm_rope, rope_tables
    f64 = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    g = torch.Generator().manual_seed(100)
    H, d, page = 2, 64, 32
    old, hist, cand = [200, 0, 37], [3, 20, 0], [5, 2, 12]        # cached before the step, new tokens, candidates
    lens = [a + b for a, b in zip(old, hist)]
    pos = [200, 201, 202] + [203] * 5 + list(range(20)) + [20] * 2 + [37] * 12
    cos, sin = rope_tables(204, d)                                # one row more than the longest cache
    tab = [f64(x) for x in (cos, sin)]
    gq, gk = ((1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    need = [-(-n // page) for n in lens]
    table, order, at = torch.zeros(3, max(need), dtype=torch.int32), torch.randperm(sum(need), generator=g).int(), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    table = table.cuda()
    cache = PagedCache(sum(need), H=H, d=d, page_size=page, timestamps=False)
    kv = torch.randn(sum(lens), 2 * H, d, generator=g).bfloat16().cuda()
    start = np.cumsum([0] + lens)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    offs = lambda n: torch.tensor([0] + n).cumsum(0).cuda()  # noqa: E731
    before = torch.cat([torch.arange(n) + s for n, s in zip(old, start)]).cuda()
    new = torch.cat([torch.arange(o, n) + s for o, n, s in zip(old, lens, start)]).cuda()
    for rows, n, length in ((before, old, old), (new, hist, lens)):
        hstu_cache_append(cache, kv[rows][:, :H], kv[rows][:, H:], offs(n), i32(length), table, cos=cos, sin=sin, norm=True, k_gain=gk)
    kc, vc, _ = hstu_cache_read(cache, offs(lens), None, table)
    every = np.concatenate([np.arange(n) for n in lens])
    want_k = R.qk_forward(f64(kv[:, :H]), f64(gk), tab[0][every], tab[1][every], False, True, float(np.float32(1e-6)))
    np.testing.assert_array_equal(f64(kc), R.four_bit(want_k))
    rows = [a + b for a, b in zip(hist, cand)]
    T, off = sum(rows), offs(rows)
    x = torch.randn(T, 3 * H, d, generator=g).bfloat16().cuda()
    got = cached_positions(off, i32(lens), i32(cand))
    assert got.tolist() == pos
    q, k = hstu_qk_norm_rope(x[:, :H], x[:, H:2 * H], got, cos, sin, q_gain=gq, k_gain=gk)
    for out, src, gain in ((q, x[:, :H], gq), (k, x[:, H:2 * H], gk)):
        want = R.qk_forward(f64(src), f64(gain), tab[0][pos], tab[1][pos], False, True, 1e-6)
        w = R.norm(f64(src), f64(gain), 1e-6)[0]
        # as in tests/test_gpu_qk.py: one rounding to BF16, FP32 arithmetic before it
        assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * R.spread(w, d, False))
    # a history row's position is its key's place in the cache: the same raw key is turned the same
    n = new.cpu().numpy()
    rows_of_history = [i for i in range(28) if not 3 <= i < 8]
    same, _ = hstu_qk_norm_rope(kv[new][:, :H], None, got[rows_of_history], cos, sin, q_gain=gk)
    w = R.norm(f64(kv[new][:, :H]), f64(gk), 1e-6)[0]
    assert np.all(np.abs(f64(same) - want_k[n]) <= 2.0 ** -8 * np.abs(want_k[n]) + 2.0 ** -20 * R.spread(w, d, False))
    v, rp = x[:, 2 * H:].contiguous(), 0.1 * torch.randn(H, 128, generator=g).cuda()
    o, y = hstu_attention_cached(cache, q, k, v, None, off, i32(lens), table, max_rows=max(rows), max_seq_len=300, alpha=d ** -0.5,
                                 num_targets=i32(cand), rab_pos=rp)
    ro = np.cumsum([0] + rows)
    for b in range(3):
        r, c = slice(ro[b], ro[b + 1]), slice(start[b], start[b + 1])
        wo, wy, bo, by = R.attention(f64(q[r]), f64(k[r]), f64(v[r]), None, f64(kc[c]), f64(vc[c]), None, None, cand[b],
                                     float(np.float32(d ** -0.5)), f64(rp), None, 300, True, float(np.float32(1e-5)))
        assert np.all(np.abs(f64(o[r]) - wo) <= bo) and np.all(np.abs(f64(y[r]) - wy) <= by)
