"""Cases of the serving path's operators: the per-head norm and rotation of
queries and keys (with its backward), appending to and reading from a paged
cache of 4-bit keys and values, and the HSTU attention over that cache; each
in a plain form of elementary torch operations and as the framework's call.

A 4-bit group is 16 features of one head: codes are e2m1 (0, .5, 1, 1.5, 2, 3,
4, 6 with a sign), the group's scale is e4m3.  A page holds, head by head,
[K codes | K scales | V codes | V scales] of page_size tokens: d / 2 bytes of
codes a token (feature 2i in the low half of byte i) and d / 16 of scales.
"""
import math
import random

import torch

own = False

DEV = "cuda"
P_BUCKETS, T_BUCKETS = 128, 64


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of each of 64 users: the latency of a serving step
        dict(name="qk forward, 64 tokens", op="qk_fwd", T=64, Hq=4, Hk=4, d=128, rot=128, pairs="half", norm=True,
             dtype="bf16", max_pos=8192),
        # the layer workload's batch (8 users of 8K to 32K tokens, 4 heads x 128)
        dict(name="qk forward, layer batch", op="qk_fwd", T=161_293, Hq=4, Hk=4, d=128, rot=128, pairs="half", norm=True,
             dtype="bf16", max_pos=32_896),
        # a heavy-tailed training batch
        dict(name="qk backward, heavy-tailed batch", op="qk_bwd", T=16_410, Hq=4, Hk=4, d=128, rot=128, pairs="half",
             norm=True, dtype="bf16", max_pos=8192),
        # FP32, fewer key heads, half of the features rotated in neighbouring pairs
        dict(name="qk backward, fp32 partial", op="qk_bwd", T=4_099, Hq=6, Hk=2, d=64, rot=32, pairs="interleaved",
             norm=True, dtype="fp32", max_pos=1024),
        # one new action of each of 64 users
        dict(name="append, 64 users x 1", op="append", B=64, new_lo=1, new_hi=1, cached_lo=200, cached_hi=8192, H=4,
             d=128, page=64, rot=128, norm=True, lens_seed=1),
        # whole histories (the layer workload's lengths) written to the cache
        dict(name="append, 8 histories", op="append", B=8, new_lo=8192, new_hi=32_768, cached_lo=0, cached_hi=0, H=4,
             d=128, page=64, rot=128, norm=True, lens_seed=2),
        # one user, a short history, one new token
        dict(name="attention, 1 user x 1 row", op="attn", B=1, hist_lo=1, hist_hi=1, cand_lo=0, cand_hi=0,
             cached_lo=300, cached_hi=300, H=4, d=128, page=64, times="own", lens_seed=3),
        # a decode step of 32 users
        dict(name="attention, 32 users x 1 row", op="attn", B=32, hist_lo=1, hist_hi=1, cand_lo=0, cand_hi=0,
             cached_lo=2048, cached_hi=8192, H=4, d=128, page=64, times="own", lens_seed=4),
        # the delta workload: 128 candidates against 2K to 8K cached tokens
        dict(name="attention, 32 users x 128 candidates", op="attn", B=32, hist_lo=0, hist_hi=0, cand_lo=128,
             cand_hi=128, cached_lo=2048, cached_hi=8192, H=4, d=128, page=64, times="request", lens_seed=5),
        # a few new actions and some candidates, 4 heads x 64
        dict(name="attention, 32 users, new and candidates", op="attn", B=32, hist_lo=0, hist_hi=9, cand_lo=5,
             cand_hi=23, cached_lo=16, cached_hi=1024, H=4, d=64, page=32, times="request", lens_seed=6),
        # one user with a long life
        dict(name="attention, 1 user, 131K cached", op="attn", B=1, hist_lo=1, hist_hi=1, cand_lo=0, cand_hi=0,
             cached_lo=131_011, cached_hi=131_011, H=4, d=128, page=128, times="own", lens_seed=7),
        # histories run through the model for the first time: every row sees the rows before it
        dict(name="attention, 4 first passes", op="attn", B=4, hist_lo=900, hist_hi=2100, cand_lo=0, cand_hi=40,
             cached_lo=0, cached_hi=0, H=4, d=128, page=64, times="own", lens_seed=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_fwd", "qk_bwd", "append", "attn", "attn", "attn"])
    if op in ("qk_fwd", "qk_bwd"):
        d = rng.choice([32, 64, 128])
        H = rng.choice([1, 2, 4, 6])
        c = dict(op=op, T=1, Hq=H, Hk=rng.choice([1, H]), d=d, rot=rng.choice([0, d // 4, d // 2, d]),
                 pairs=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.8, dtype=rng.choice(["bf16", "fp32"]),
                 max_pos=rng.randint(64, 32_896))
        return dict(c, T=min(_log(rng, 1, 160_000), int(6e8 / work(c)["bytes"])))
    d = rng.choice([64, 128])
    B = _log(rng, 1, 64)
    base = dict(op=op, B=B, H=rng.choice([1, 2, 3, 4]), d=d, page=rng.choice([32, 64, 128]), lens_seed=rng.randrange(1 << 30))
    if op == "append":
        hi = _log(rng, 1, max(2, 150_000 // B))
        cached = _log(rng, 1, 8192)
        return dict(base, new_lo=rng.choice([0, 1, (hi + 1) // 2]), new_hi=hi, cached_lo=cached // 3, cached_hi=cached,
                    rot=rng.choice([0, d // 2, d]), norm=rng.random() < 0.5)
    cached = _log(rng, 1, max(64, min(131_072, 250_000 // B)))
    kind = rng.choice(["decode", "candidates", "both", "first"])
    c = dict(base, hist_lo=0, hist_hi=0, cand_lo=0, cand_hi=0, cached_lo=cached // 3, cached_hi=cached,
             times=rng.choice(["own", "request"]))
    if kind == "decode":
        c.update(hist_lo=1, hist_hi=1)
    elif kind == "candidates":
        c.update(cand_lo=1, cand_hi=_log(rng, 1, 150))
    elif kind == "both":
        c.update(hist_hi=_log(rng, 1, 60), cand_hi=_log(rng, 1, 60))
    else:
        c.update(hist_lo=1, hist_hi=_log(rng, 1, max(2, min(1500, 6000 // B))), cached_lo=0, cached_hi=0,
                 cand_hi=rng.choice([0, 20]))
    return c


def _between(r, lo, hi):
    return r.randint(min(lo, hi), max(lo, hi))


def _rows(c):
    """Lengths of a case: (cached tokens, new or history rows, candidates) of every sequence."""
    r = random.Random(c["lens_seed"])
    cached, hist, cand = [], [], []
    for _ in range(c["B"]):
        if c["op"] == "append":
            n, m = _between(r, c["new_lo"], c["new_hi"]), 0
        else:
            n, m = _between(r, c["hist_lo"], c["hist_hi"]), _between(r, c["cand_lo"], c["cand_hi"])
        cached.append(_between(r, c["cached_lo"], c["cached_hi"]) + n)
        hist.append(n)
        cand.append(m)
    if sum(hist) + sum(cand) == 0:
        hist[0], cached[0] = 1, cached[0] + 1
    return cached, hist, cand


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 13)
    return g


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


def _tables(max_pos, rot):
    """cos and sin of position / 10000^(2i / rot), angles in 64 bits, kept in 32."""
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    a = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * (10000.0 ** (-2.0 * i / max(rot, 1)))
    return a.cos().float(), a.sin().float()


def _offsets(n):
    return torch.tensor([0] + n, dtype=torch.int64).cumsum(0).to(DEV)


def _bytes_of_head(c):
    return 2 * c["page"] * (c["d"] // 2 + c["d"] // 16)


def _table_of_pages(c, cached, seed):
    """Pages of every sequence in random order, with a few pages of nobody."""
    per = [-(-n // c["page"]) for n in cached]
    width, total = max(max(per), 1), sum(per)
    order = torch.randperm(total + 3, generator=torch.Generator().manual_seed(seed + 5))
    table, at = torch.zeros(c["B"], width, dtype=torch.int32), 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n].int()
        at += n
    return table.to(DEV), total + 3


def _cache_rows(c, table, lens, first):
    """Page and place in it of positions [first, lens) of every sequence, packed."""
    n = [a - f for a, f in zip(lens, first)]
    b = torch.repeat_interleave(torch.arange(c["B"]), torch.tensor(n)).to(DEV)
    start = (torch.tensor(first) - torch.tensor([0] + n).cumsum(0)[:-1]).to(DEV)
    pos = torch.arange(sum(n), device=DEV) + start[b]
    return table[b, pos // c["page"]].long(), pos % c["page"], pos


def _times(g, lens, b_of, start):
    """Integer seconds: each action some ten minutes after the one before."""
    gap = torch.empty(sum(lens), device=DEV).exponential_(1 / 600.0, generator=g).round().long()
    t = gap.cumsum(0)
    return 1_700_000_000 + t - t[start[b_of]]


def prepare(c, seed):
    g = _gen(seed)
    s = dict(c=c)
    if c["op"] in ("qk_fwd", "qk_bwd"):
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        T, Hq, Hk, d = c["T"], c["Hq"], c["Hk"], c["d"]
        # q and k lie side by side in the projection's output
        both = _normal(g, T, Hq + Hk, d, dtype=dt)
        s["q"], s["k"] = both[:, :Hq], both[:, Hq:]
        s["positions"] = torch.randint(0, c["max_pos"], (T,), device=DEV, generator=g, dtype=torch.int32)
        s["cos"], s["sin"] = _tables(c["max_pos"], c["rot"])
        s["gq"], s["gk"] = (1 + 0.2 * _normal(g, d) if c["norm"] else None for _ in range(2))
        if c["op"] == "qk_bwd":
            s["dq_out"], s["dk_out"] = _normal(g, T, Hq, d, dtype=dt), _normal(g, T, Hk, d, dtype=dt)
        return s
    cached, hist, cand = _rows(c)
    B, H, d = c["B"], c["H"], c["d"]
    s["table"], pages = _table_of_pages(c, cached, seed)
    s["lens"] = torch.tensor(cached, dtype=torch.int32, device=DEV)
    s["pages"] = torch.zeros(pages, H, _bytes_of_head(c), dtype=torch.uint8, device=DEV)
    s["page_times"] = torch.zeros(pages, c["page"], dtype=torch.int64, device=DEV)
    if c["op"] == "append":
        T = sum(hist)
        s["offsets"] = _offsets(hist)
        both = _normal(g, T, 2 * H, d, dtype=torch.bfloat16)
        s["k"], s["v"] = both[:, :H], both[:, H:]
        s["times"] = 1_700_000_000 + torch.randint(0, 1 << 20, (T,), device=DEV, generator=g)
        s["starts"] = torch.tensor([a - n for a, n in zip(cached, hist)], dtype=torch.int32, device=DEV)
        s["cos"], s["sin"] = _tables(max(cached), c["rot"])
        s["gk"] = 1 + 0.2 * _normal(g, d) if c["norm"] else None
        s["where"] = _cache_rows(c, s["table"], cached, [a - n for a, n in zip(cached, hist)])
        return s
    # the cache as it stands: keys and values of unit size, times ten minutes apart
    pg, at, pos = _cache_rows(c, s["table"], cached, [0] * B)
    b_of = torch.repeat_interleave(torch.arange(B), torch.tensor(cached)).to(DEV)
    start = torch.tensor([0] + cached).cumsum(0)[:-1].to(DEV)
    when = _times(g, cached, b_of, start)
    s["page_times"][pg, at] = when
    for lo in range(0, sum(cached), 1 << 16):
        hi = min(sum(cached), lo + (1 << 16))
        for which in (0, 1):
            codes, scales = _quantise(_normal(g, hi - lo, H, d, dtype=torch.bfloat16).double())
            _write(c, s["pages"], which, pg[lo:hi], at[lo:hi], codes, scales)
    T = sum(hist) + sum(cand)
    n = [a + b for a, b in zip(hist, cand)]
    s["offsets"] = _offsets(n)
    s["targets"] = torch.tensor(cand, dtype=torch.int32, device=DEV)
    s["max_rows"], s["max_len"] = max(n), max(a + b for a, b in zip(cached, cand))
    s["q"], s["k"], s["v"], s["u"] = (_normal(g, T, H, d, dtype=torch.bfloat16) for _ in range(4))
    s["u"] = s["u"].view(T, H * d)
    s["rab_pos"], s["rab_time"] = 0.02 * _normal(g, H, P_BUCKETS), 0.02 * _normal(g, H, T_BUCKETS)
    # a row's time: a history token's is the cache's; a candidate's is the request's, or (of other services) its own
    rb = torch.repeat_interleave(torch.arange(B), torch.tensor(n)).to(DEV)
    r = torch.arange(T, device=DEV) - s["offsets"][:-1][rb]
    h = torch.tensor(hist, device=DEV)[rb]
    last = start[rb] + s["lens"][rb] - 1
    is_hist = r < h
    row_tok = torch.where(is_hist, last - h + 1 + r, last.clamp(min=0))
    t_row = when[row_tok] if sum(cached) else torch.full((T,), 1_700_000_000, device=DEV)
    later = 600 if c["times"] == "request" else torch.randint(0, 5000, (T,), device=DEV, generator=g)
    s["times"] = torch.where(is_hist, t_row, t_row + later)
    s["alpha"] = d ** -0.5
    # padded view of the rows and tokens, which the plain form computes on
    M, L = max(n), max(max(cached), 1)
    s["row_at"] = (s["offsets"][:-1, None] + torch.arange(M, device=DEV)).clamp(max=T - 1)
    s["hist"] = torch.tensor(hist, device=DEV)
    s["M"], s["L"] = M, L
    s["row_of"] = (rb, r)
    return s


# -------------------------------------------------------------- plain form

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pow2(e, dtype=torch.float64):
    """2^e for integers -16 <= e <= 16, exactly."""
    return torch.tensor([2.0 ** i for i in range(-16, 17)], dtype=dtype, device=DEV)[(e + 16).long()]


def _e4m3(a):
    """To the nearest e4m3 value (ties to even), at most 448: as a value and as a byte.  a >= 0, 64 bits."""
    e = torch.frexp(a.clamp(min=1e-300))[1].clamp(min=-5, max=9) - 1          # 2^e <= a < 2^(e+1), subnormals at -6
    step = _pow2(e - 3)
    q = (a / step).round()                                                    # 8..16, or 0..8 where subnormal
    v = (q * step).clamp(max=448.0)
    e2 = torch.frexp(v.clamp(min=1e-300))[1].clamp(min=-5) - 1
    m = v / _pow2(e2 - 3)
    byte = torch.where(m >= 8, (e2 + 7) * 8 + (m - 8), m)
    return v, byte.to(torch.uint8)


def _quantise(x):
    """[T, H, d] in 64 bits -> codes [T, H, d] (0..15) and scale bytes [T, H, d / 16]."""
    T, H, d = x.shape
    x = x.reshape(T, H, d // 16, 16)
    top = x.abs().amax(-1)
    s, byte = _e4m3(top / torch.full_like(top, 6.0))       # a true quotient: by a number, torch multiplies by its inverse
    a = x.abs()
    s = s[..., None]
    # borders between neighbouring codes; a tie goes to the even code
    code = ((a > 0.25 * s).byte() + (a >= 0.75 * s).byte() + (a > 1.25 * s).byte() + (a >= 1.75 * s).byte()
            + (a > 2.5 * s).byte() + (a >= 3.5 * s).byte() + (a > 5.0 * s).byte())
    code = torch.where(s > 0, code, torch.zeros_like(code))
    code = code + 8 * torch.signbit(x).byte()
    return code.reshape(T, H, d), byte


def _parts(c):
    """Byte ranges of [K codes, K scales, V codes, V scales] in a head's part of a page."""
    nc, ns = c["page"] * c["d"] // 2, c["page"] * c["d"] // 16
    return (0, nc), (nc, nc + ns), (nc + ns, 2 * nc + ns), (2 * nc + ns, 2 * nc + 2 * ns)


def _write(c, pages, which, pg, at, codes, scales):
    packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
    (a, b), (e, f) = _parts(c)[2 * which:2 * which + 2]
    pages[:, :, a:b].view(pages.shape[0], c["H"], c["page"], -1).permute(0, 2, 1, 3)[pg, at] = packed
    pages[:, :, e:f].view(pages.shape[0], c["H"], c["page"], -1).permute(0, 2, 1, 3)[pg, at] = scales


def _values(c, pages, which, pg, at, dtype):
    """Values [.., H, d] of the tokens at (pg, at)."""
    (a, b), (e, f) = _parts(c)[2 * which:2 * which + 2]
    codes = pages[:, :, a:b].view(pages.shape[0], c["H"], c["page"], -1).permute(0, 2, 1, 3)[pg, at]
    byte = pages[:, :, e:f].view(pages.shape[0], c["H"], c["page"], -1).permute(0, 2, 1, 3)[pg, at].int()
    codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV, dtype=dtype)
    ex, man = (byte >> 3) & 15, (byte & 7).to(dtype)
    s = torch.where(ex > 0, (8 + man) * _pow2(ex - 10, dtype), man * 2.0 ** -9)
    return lut[codes] * s.repeat_interleave(16, -1)


def _norm_rope(x, gain, cos, sin, rot, pairs, norm):
    """The rows x [T, H, d] of the operator's precision; cos, sin [T, rot / 2]."""
    if norm:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain
    if rot == 0:
        return x
    a, b, rest = _pairs(x, rot, pairs)
    cos, sin = cos[:, None], sin[:, None]
    return _unpairs(a * cos - b * sin, b * cos + a * sin, rest, pairs)


def _pairs(x, rot, pairs):
    r, rest = x[..., :rot], x[..., rot:]
    return (r[..., :rot // 2], r[..., rot // 2:], rest) if pairs == "half" else (r[..., 0::2], r[..., 1::2], rest)


def _unpairs(a, b, rest, pairs):
    return torch.cat([a, b, rest], -1) if pairs == "half" else torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)


def _norm_rope_grad(x, dout, gain, cos, sin, rot, pairs, norm):
    dw = dout
    if rot:
        a, b, rest = _pairs(dout, rot, pairs)
        cos, sin = cos[:, None], sin[:, None]
        dw = _unpairs(a * cos + b * sin, b * cos - a * sin, rest, pairs)
    if not norm:
        return dw, None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    xr = x * r
    e = dw * gain
    return r * (e - xr * (e * xr).mean(-1, keepdim=True)), (dw * xr).sum((0, 1))


def _buckets(dt):
    """0 for equal times, else the number of binary digits of the gap, at most T_BUCKETS - 1."""
    return torch.frexp(dt.abs().double())[1].long().clamp(max=T_BUCKETS - 1)


def _plain_attn(s):
    c = s["c"]
    B, H, d, M, L = c["B"], c["H"], c["d"], s["M"], s["L"]
    j = torch.arange(L, device=DEV)
    lens = s["lens"].long()
    pg = s["table"].long()[:, (j // c["page"])]
    at = (j % c["page"]).expand(B, L)
    live = j < lens[:, None]                                                   # [B, L]
    K = _values(c, s["pages"], 0, pg, at, torch.float32).permute(0, 2, 1, 3)   # [B, H, L, d]
    V = torch.where(live[:, None, :, None], _values(c, s["pages"], 1, pg, at, torch.float32).permute(0, 2, 1, 3), 0.0)
    q, k, v = (s[x].float()[s["row_at"]].permute(0, 2, 1, 3) for x in ("q", "k", "v"))   # [B, H, M, d]
    r = torch.arange(M, device=DEV)
    cand = r >= s["hist"][:, None]                                             # [B, M]
    pos = torch.where(cand, lens[:, None], lens[:, None] - s["hist"][:, None] + r)
    tq, tk = s["times"][s["row_at"]], s["page_times"][pg, at]
    see = live[:, None, :] & (j <= pos[:, :, None])                            # [B, M, L]
    bias = s["rab_pos"][:, (pos[:, :, None] - j).clamp(0, P_BUCKETS - 1)].transpose(0, 1)
    bias = bias + s["rab_time"][:, _buckets(tq[:, :, None] - tk[:, None, :])].transpose(0, 1)
    z = s["alpha"] * (q @ K.transpose(-1, -2)) + bias
    p = torch.where(see[:, None], z * torch.sigmoid(z), 0.0)
    o = p @ V
    zs = s["alpha"] * (q * k).sum(-1) + (s["rab_pos"][:, 0] + s["rab_time"][:, 0])[:, None]
    o = o + torch.where(cand[:, None], zs * torch.sigmoid(zs), 0.0)[..., None] * v
    o = (o / s["max_len"])[s["row_of"][0], :, s["row_of"][1]]                   # [T, H, d]
    f = o.reshape(o.shape[0], H * d)
    f = f - f.mean(-1, keepdim=True)
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-5) * s["u"].float()
    return {"o": o.bfloat16(), "y": y.bfloat16()}


def _plain(s):
    c = s["c"]
    if c["op"] == "attn":
        return _plain_attn(s)
    if c["op"] == "append":
        k = s["k"].double()
        pg, at, pos = s["where"]
        k = _norm_rope(k, s["gk"].double() if c["norm"] else None, s["cos"][pos].double(), s["sin"][pos].double(),
                       c["rot"], "half", c["norm"])
        _write(c, s["pages"], 0, pg, at, *_quantise(k))
        _write(c, s["pages"], 1, pg, at, *_quantise(s["v"].double()))
        s["page_times"][pg, at] = s["times"]
        return {"k": _values(c, s["pages"], 0, pg, at, torch.float32).bfloat16(),
                "v": _values(c, s["pages"], 1, pg, at, torch.float32).bfloat16(), "times": s["page_times"][pg, at]}
    at = s["positions"].long()
    cos, sin = s["cos"][at], s["sin"][at]
    how = (c["rot"], c["pairs"], c["norm"])
    if c["op"] == "qk_fwd":
        return {n: _norm_rope(s[n].float(), s["g" + n], cos, sin, *how).to(s[n].dtype) for n in ("q", "k")}
    out = {}
    out["dq"], out["dgq"] = _norm_rope_grad(s["q"].float(), s["dq_out"].float(), s["gq"], cos, sin, *how)
    out["dk"], out["dgk"] = _norm_rope_grad(s["k"].float(), s["dk_out"].float(), s["gk"], cos, sin, *how)
    return {n: x.to(s["q"].dtype) if n in ("dq", "dk") else x for n, x in out.items() if x is not None}


# ----------------------------------------------------------- the framework

def _open(s):
    """The handles that a program keeps beside its buffers."""
    c = s["c"]
    if c["op"] in ("qk_fwd", "qk_bwd"):
        from hstu_jagged_attention_02_gb300.qk import QKProblem
        return QKProblem(s["q"], s["k"], s["positions"], s["cos"], s["sin"], rot_dim=c["rot"],
                         interleaved=c["pairs"] == "interleaved", norm=c["norm"], eps=1e-6, q_gain=s["gq"], k_gain=s["gk"],
                         dq_out=s.get("dq_out"), dk_out=s.get("dk_out"))
    from hstu_jagged_attention_02_gb300.cache import AppendProblem, CachedProblem, PagedCache, ReadProblem
    cache = PagedCache(H=c["H"], d=c["d"], page_size=c["page"], pages=s["pages"], timestamps=s["page_times"])
    if c["op"] == "append":
        write = AppendProblem(cache, s["k"], s["v"], s["offsets"], s["lens"], s["table"], timestamps=s["times"],
                              cos=s["cos"], sin=s["sin"], rot_dim=c["rot"], norm=c["norm"], eps=1e-6, k_gain=s["gk"])
        return write, ReadProblem(cache, s["offsets"], s["starts"], s["table"], total_tokens=s["k"].shape[0])
    return CachedProblem(cache, s["q"], s["k"], s["v"], s["u"], s["offsets"], s["lens"], s["table"], num_targets=s["targets"],
                         timestamps=s["times"], rab_pos=s["rab_pos"], rab_time=s["rab_time"], max_rows=s["max_rows"],
                         max_seq_len=s["max_len"], alpha=s["alpha"], norm="layernorm", eps=1e-5)


def run(s):
    if not own:
        return _plain(s)
    h = s.get("handle")
    if h is None:
        h = s["handle"] = _open(s)
    op = s["c"]["op"]
    if op == "qk_fwd":
        h.forward()
        return {"q": h.q_out, "k": h.k_out}
    if op == "qk_bwd":
        h.backward()
        return {n: x for n, x in (("dq", h.dq), ("dgq", h.d_q_gain), ("dk", h.dk), ("dgk", h.d_k_gain)) if x is not None}
    if op == "append":
        h[0].run()
        h[1].run()
        return {"k": h[1].k, "v": h[1].v, "times": h[1].timestamps}
    h.forward()
    return {"o": h.o, "y": h.y}


# -------------------------------------------------------------------- work

def work(c):
    if c["op"] in ("qk_fwd", "qk_bwd"):
        n = c["T"] * (c["Hq"] + c["Hk"]) * c["d"]
        e = 2 if c["dtype"] == "bf16" else 4
        tables = 4 * c["rot"] * min(c["T"], c["max_pos"]) + 4 * c["T"]
        return {"bytes": n * e * (2 if c["op"] == "qk_fwd" else 3) + tables, "flops": n * (8 if c["op"] == "qk_fwd" else 16)}
    cached, hist, cand = _rows(c)
    H, d = c["H"], c["d"]
    packed = 2 * (d // 2 + d // 16)
    if c["op"] == "append":
        T = sum(hist)
        return {"bytes": T * (H * (2 * d * 2 + packed + 2 * d * 2) + 8 + 8) + 4 * c["rot"] * min(T, max(cached)), "flops": T * H * d * 30}
    T = sum(hist) + sum(cand)
    pairs = sum(m * (n + 1) + h * (n - h) + h * (h + 1) // 2 for n, h, m in zip(cached, hist, cand))
    return {"bytes": sum(cached) * (H * packed + 8) + T * H * d * 2 * 6 + 8 * T, "flops": pairs * H * 4 * d}


# ------------------------------------------------- the definition, 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "attn":
        return _exact_attn(s)
    if c["op"] == "append":
        pos = s["where"][2]
        k = torch.empty(*s["k"].shape, dtype=torch.float64, device=DEV)
        v = torch.empty_like(k)
        for lo in range(0, k.shape[0], 1 << 14):
            hi = lo + (1 << 14)
            k[lo:hi] = _exact_4bit(_exact_rows(s["k"][lo:hi], s["gk"], s["cos"][pos[lo:hi]], s["sin"][pos[lo:hi]], c["rot"],
                                               "half", c["norm"]))
            v[lo:hi] = _exact_4bit(s["v"][lo:hi].double())
        return {"k": k, "v": v, "times": None}
    at = s["positions"].long()
    cos, sin = s["cos"][at], s["sin"][at]
    if c["op"] == "qk_fwd":
        return {n: _exact_rows(s[n], s["g" + n], cos, sin, c["rot"], c["pairs"], c["norm"]) for n in ("q", "k")}
    out = {}
    for n in ("q", "k"):
        # through the derivative of the definition
        x = s[n].double().detach().requires_grad_()
        leaves = [x]
        if c["norm"]:
            leaves.append(s["g" + n].double().detach().requires_grad_())
        y = _exact_rows(x, leaves[-1] if c["norm"] else None, cos, sin, c["rot"], c["pairs"], c["norm"])
        got = torch.autograd.grad(y, leaves, s["d%s_out" % n].double())
        out["d" + n] = got[0]
        if c["norm"]:
            out["dg" + n] = got[1]
    return out


def _exact_rows(x, gain, cos, sin, rot, pairs, norm):
    """The pairs as complex numbers turned by the position's angle."""
    x = x.double()
    if norm:
        x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * gain.double()
    if rot == 0:
        return x
    i = torch.arange(rot // 2, device=DEV)
    a, b = (i, i + rot // 2) if pairs == "half" else (2 * i, 2 * i + 1)
    w = torch.complex(x[..., a], x[..., b]) * torch.complex(cos.double(), sin.double())[:, None]
    y = torch.zeros_like(x)
    y = y.index_copy(-1, a, w.real).index_copy(-1, b, w.imag)
    rest = torch.arange(rot, x.shape[-1], device=DEV)
    return y.index_copy(-1, rest, x[..., rot:])


def _exact_4bit(x):
    """The nearest of all values that a group can hold (a tie to the even code, the even mantissa)."""
    T, H, d = x.shape
    x = x.reshape(-1, 16)
    scales = torch.tensor([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127],
                          dtype=torch.float64, device=DEV)
    want = x.abs().amax(-1)
    s = scales[_nearest(scales * 6, want)][:, None]
    levels = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    y = torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0)
    return (torch.sign(x) * levels[_nearest(levels, y)] * s).reshape(T, H, d)


def _nearest(levels, x):
    """Index of the level nearest to x; halfway, the even index."""
    mid = (levels[1:] + levels[:-1]) / 2
    below = torch.searchsorted(mid, x.contiguous())                  # number of borders < x
    tie = mid[below.clamp(max=mid.numel() - 1)] == x
    return torch.where(tie & (below % 2 == 1), below + 1, below).clamp(max=levels.numel() - 1)


def _exact_attn(s):
    c = s["c"]
    H, d, N = c["H"], c["d"], s["max_len"]
    off, lens, cand = s["offsets"].tolist(), s["lens"].tolist(), s["targets"].tolist()
    o = torch.zeros(off[-1], H, d, dtype=torch.float64, device=DEV)
    rp, rt = s["rab_pos"].double(), s["rab_time"].double()
    silu = lambda z: z / (1 + torch.exp(-z))  # noqa: E731
    edges = 2 ** torch.arange(0, T_BUCKETS - 1, device=DEV)
    bits = lambda dt: torch.bucketize(dt.abs(), edges, right=True)  # noqa: E731
    for b in range(c["B"]):
        L, rows = lens[b], slice(off[b], off[b + 1])
        n, m = off[b + 1] - off[b], cand[b]
        pos = torch.tensor([min(L - (n - m) + r, L) for r in range(n)], dtype=torch.int64, device=DEV)
        tok = torch.arange(L, device=DEV)
        pg, at = s["table"][b].long()[tok // c["page"]], tok % c["page"]
        K, V = (_values(c, s["pages"], w, pg, at, torch.float64) for w in (0, 1))
        tk, tq = s["page_times"][pg, at], s["times"][rows]
        q, k, v = (s[x][rows].double() for x in ("q", "k", "v"))
        gap = pos[:, None] - tok[None, :]
        bt = bits(tq[:, None] - tk[None, :])
        for h in range(H):
            z = s["alpha"] * (q[:, h] @ K[:, h].T) + rp[h][gap.clamp(0, P_BUCKETS - 1)] + rt[h][bt]
            o[rows, h] = (silu(z) * (gap >= 0)) @ V[:, h]
        if m:
            own_z = s["alpha"] * (q[n - m:] * k[n - m:]).sum(-1) + rp[:, 0] + rt[:, 0]
            o[off[b + 1] - m:off[b + 1]] += silu(own_z)[..., None] * v[n - m:]
    o = o / N
    f = o.reshape(o.shape[0], -1)
    mean, var = f.mean(-1, keepdim=True), f.var(-1, unbiased=False, keepdim=True)
    return {"o": o, "y": (f - mean) / (var + 1e-5).sqrt() * s["u"].double()}
