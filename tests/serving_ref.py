"""Plain 64-bit NumPy forms of the serving path's operators: norm and rotation
of queries and keys, the 4-bit paged cache, the attention over it.  Written
from the definitions; they share no code with the package."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)])[:127]


def rope_tables(max_pos, rot, base=10000.0):
    i = np.arange(rot // 2)
    a = np.arange(max_pos)[:, None] * base ** (-2.0 * i / max(rot, 1))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def norm(x, gain, eps):
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    return x * r * (1.0 if gain is None else gain), r


def turn(w, cos, sin, interleaved, back=False):
    """w [T, H, d] turned by the angles of cos, sin [T, rot / 2]."""
    rot = 2 * cos.shape[1]
    a, b = pairs(rot, interleaved)
    c, s = cos[:, None].astype(np.float64), sin[:, None].astype(np.float64) * (-1.0 if back else 1.0)
    out = w.copy()
    out[..., a] = w[..., a] * c - w[..., b] * s
    out[..., b] = w[..., b] * c + w[..., a] * s
    return out


def spread(w, rot, interleaved):
    """|w| plus the partner's |w|: the size of a turned feature's terms."""
    a, b = pairs(rot, interleaved)
    m = np.abs(w)
    out = m.copy()
    out[..., a] = m[..., a] + m[..., b]
    out[..., b] = m[..., a] + m[..., b]
    return out


def qk_forward(x, gain, cos, sin, interleaved, with_norm, eps):
    w = norm(x, gain, eps)[0] if with_norm else x
    return turn(w, cos, sin, interleaved)


def qk_backward(x, dout, gain, cos, sin, interleaved, with_norm, eps):
    """(dx, dgain, bound): bound [T, H, d] is the size of dx's terms."""
    e = turn(dout, cos, sin, interleaved, back=True)
    size = spread(dout, 2 * cos.shape[1], interleaved)
    if not with_norm:
        return e, None, size
    _, r = norm(x, None, eps)
    g = 1.0 if gain is None else gain
    xr = x * r
    dx = r * (e * g - xr * np.mean(e * g * xr, -1, keepdims=True))
    bound = r * (size * np.abs(g) + np.abs(xr) * np.mean(np.abs(size * g * xr), -1, keepdims=True))
    return dx, (e * xr).sum((0, 1)), bound


def nearest(levels, x):
    """Index of the level nearest to x >= 0; halfway, the even index."""
    mid = (levels[1:] + levels[:-1]) / 2
    i = np.searchsorted(mid, x, side="left")
    tie = (i < len(mid)) & (mid[np.minimum(i, len(mid) - 1)] == x)
    return np.minimum(np.where(tie & (i % 2 == 1), i + 1, i), len(levels) - 1)


def four_bit(x, exp=0):
    """The values that the cache holds for x [..., d] (d a multiple of 16)."""
    g = x.reshape(-1, 16) * 2.0 ** -exp
    top = np.abs(g).max(-1)
    s = E4M3[nearest(6.0 * E4M3, top)][:, None]
    with np.errstate(all="ignore"):
        v = np.sign(g) * E2M1[nearest(E2M1, np.where(s > 0, np.abs(g) / np.where(s > 0, s, 1.0), 0.0))] * s
    v[np.isnan(top)] = np.nan
    return (v * 2.0 ** exp).reshape(x.shape)


def silu(z):
    return z / (1.0 + np.exp(-z))


def time_bucket(dt, tb):
    return np.minimum(np.array([int(abs(int(v))).bit_length() for v in dt.ravel()], dtype=np.int64).reshape(dt.shape), tb - 1)


def attention(q, k, v, u, k_cache, v_cache, t_rows, t_cache, m, alpha, rab_pos, rab_time, N, ln, eps):
    """One sequence: rows [n, H, d] over cached [L, H, d]; the last m rows are
    candidates.  Returns o, y and bounds on what FP16 scores, FP32 sums and a
    last rounding to BF16 may change in them."""
    n, H, d = q.shape
    L = k_cache.shape[0]
    pos = np.array([L if r >= n - m else L - (n - m) + r for r in range(n)])
    gap = pos[:, None] - np.arange(L)[None]
    see = gap >= 0
    o, size = np.zeros((n, H, d)), np.zeros((n, H, d))
    P = rab_pos.shape[1] if rab_pos is not None else 1
    for h in range(H):
        z = alpha * q[:, h] @ k_cache[:, h].T
        zs = abs(alpha) * np.abs(q[:, h]) @ np.abs(k_cache[:, h]).T
        if rab_pos is not None:
            b = rab_pos[h][np.clip(gap, 0, P - 1)]
            z, zs = z + b, zs + np.abs(b)
        if rab_time is not None and t_rows is not None:
            b = rab_time[h][time_bucket(t_rows[:, None] - t_cache[None], rab_time.shape[1])]
            z, zs = z + b, zs + np.abs(b)
        w = np.where(see, silu(z), 0.0)
        o[:, h] = w @ v_cache[:, h]
        # one FP16 rounding of 16 w (2^-11 relative, 2^-25 where subnormal), the exponential and the
        # quotient (2^-18), the score's FP32 sum (2^-19 of its terms, |dw/dz| < 1.1), FP32 sums over the row
        dw = np.where(see, np.abs(w) * (2.0 ** -11 + 2.0 ** -17) + 1.1 * 2.0 ** -19 * zs + 2.0 ** -29, 0.0)
        size[:, h] = dw @ np.abs(v_cache[:, h])
        if m:
            zc = alpha * (q[n - m:, h] * k[n - m:, h]).sum(-1)
            if rab_pos is not None:
                zc = zc + rab_pos[h][0]
            if rab_time is not None and t_rows is not None:
                zc = zc + rab_time[h][0]
            o[n - m:, h] += silu(zc)[:, None] * v[n - m:, h]
            size[n - m:, h] += 2.0 ** -17 * (np.abs(silu(zc)) + np.abs(alpha) * (np.abs(q * k))[n - m:, h].sum(-1))[:, None] \
                * np.abs(v[n - m:, h])
    o, size = o / N, size / N + 1e-30
    f, df = o.reshape(n, H * d), size.reshape(n, H * d)
    gate = 1.0 if u is None else u
    if ln:
        c = f - f.mean(-1, keepdims=True)
        r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
        y = c * r * gate
        dy = np.abs(gate) * r * (df + df.mean(-1, keepdims=True) + np.abs(c) * r * np.sqrt((df * df).mean(-1, keepdims=True)))
        dy = 1.05 * dy + 2.0 ** -18 * (np.abs(y) + np.abs(gate) * r * np.abs(f).max(-1, keepdims=True))
    else:
        y, dy = f * gate, df * np.abs(gate) + 2.0 ** -20 * np.abs(f * gate)
    half = 2.0 ** -8
    return o, y, size + half * (np.abs(o) + size), dy + half * (np.abs(y) + dy)
