"""Plain 64-bit NumPy forms of the training block's operators: layer norm,
products of ragged groups, AdamW, and the moments in 8 bits.  Written from the
definitions; they share no code with the package."""
import numpy as np


def ln_stats(x, eps):
    mean = x.mean(-1)
    return mean, 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(-1) + eps)


def ln_forward(x, w, b, eps):
    """y, mean, rstd, and the size of y's terms."""
    mean, rstd = ln_stats(x, eps)
    one, none = 1.0 if w is None else w, 0.0 if b is None else b
    y = (x - mean[:, None]) * rstd[:, None] * one + none
    size = (np.abs(x) + np.abs(x).mean(-1, keepdims=True)) * rstd[:, None] * np.abs(one) + np.abs(none)
    return y, mean, rstd, size


def ln_backward(x, w, mean, rstd, dy):
    """dx, dw, db with the sizes of their terms, from statistics that are given."""
    h, r = (x - mean[:, None]) * rstd[:, None], rstd[:, None]
    e = dy * (1.0 if w is None else w)
    dx = r * (e - e.mean(-1, keepdims=True) - h * (e * h).mean(-1, keepdims=True))
    ha, ea = (np.abs(x) + np.abs(mean)[:, None]) * r, np.abs(e)
    size = r * (ea + ea.mean(-1, keepdims=True) + ha * (ea * ha).mean(-1, keepdims=True))
    return (dx, size), ((dy * h).sum(0), (np.abs(dy) * ha).sum(0)), (dy.sum(0), np.abs(dy).sum(0))


def groups_forward(x, w, off):
    y, size = np.zeros((x.shape[0], w.shape[2])), np.zeros((x.shape[0], w.shape[2]))
    for g in range(w.shape[0]):
        r = slice(off[g], off[g + 1])
        y[r], size[r] = x[r] @ w[g], np.abs(x[r]) @ np.abs(w[g])
    return y, size


def groups_backward(x, w, off, dy):
    dw, dws = np.zeros(w.shape), np.zeros(w.shape)
    for g in range(w.shape[0]):
        r = slice(off[g], off[g + 1])
        dw[g], dws[g] = x[r].T @ dy[r], np.abs(x[r]).T @ np.abs(dy[r])
    return groups_forward(dy, w.transpose(0, 2, 1), off), (dw, dws)


def philox4x32(counter, key):
    """Philox4x32-10 word for word: counters uint64 [n, 4] below 2^32, key (2 words)."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1)


def words(first_block, n, step, seed):
    """A tensor's words of 32 bits, one an element: the tensor's blocks begin at first_block."""
    q = np.arange(first_block * 64, (first_block + (n + 255) // 256) * 64, dtype=np.uint64)
    ctr = np.stack([q & np.uint64(0xFFFFFFFF), q >> np.uint64(32), np.full_like(q, step & 0xFFFFFFFF),
                    np.full_like(q, step >> 32)], -1)
    return philox4x32(ctr, (seed & 0xFFFFFFFF, seed >> 32)).reshape(-1)[:n]


def values(kind):
    """The 256 values (times the block's power of two) of the first ("m") or second ("v") moment."""
    bias, out = (7, []) if kind == "m" else (15, [])
    for code in range(256):
        mag = code & 127 if kind == "m" else code
        e, f = mag >> 3, mag & 7
        x = f / 8 * 2.0 ** (1 - bias) if e == 0 else (1 + f / 8) * 2.0 ** (e - bias)
        if kind == "m" and mag == 127:
            x = np.nan
        out.append(-x if kind == "m" and code > 127 else x)
    return np.array(out)


OFF = {"m": 134, "v": 142}


def decode(codes, exps, kind):
    n = codes.size
    return values(kind)[codes] * np.repeat(2.0 ** (exps.astype(np.float64) - OFF[kind]), 256)[:n]


def encode(x, word, kind):
    """x FP32; up to the next value or down to the one below by the random words' odds: codes, exponent bytes."""
    n = x.size
    pad = np.zeros((n + 255) // 256 * 256)
    a = np.abs(x.astype(np.float64))
    pad[:n] = np.where(np.isfinite(a), a, 0.0)
    top = pad.reshape(-1, 256).max(-1)
    exps = np.maximum(np.where(top > 0, np.frexp(np.maximum(top, 1e-300))[1] - 1 + 127, 0), 16)
    t = a * np.repeat(2.0 ** (OFF[kind] - exps), 256)[:n]
    half = (word & np.uint64(0xFFFF)) if kind == "m" else (word >> np.uint64(16))
    mags = values(kind)[:127] if kind == "m" else values(kind)
    fine = np.isfinite(t)
    down = np.searchsorted(mags, np.where(fine, t, 0.0), side="right") - 1
    gap = np.diff(np.append(mags, 2 * mags[-1] - mags[-2]))[down]
    up = (np.where(fine, t, 0.0) - mags[down]) / gap + (half.astype(np.float64) * 16 + 8) / 2 ** 20 >= 1
    code = np.minimum(down + up, len(mags) - 1)
    code = np.where(fine, code, 127 if kind == "m" else 255)
    if kind == "m":
        code = code | np.where(np.signbit(x), 128, 0)
    return code.astype(np.uint8), exps.astype(np.uint8)


def moments(m, v, g, b1, b2, scale=None):
    """The new moments as FP32 numbers, product by product (m, v, g, scale FP32)."""
    f = np.float32
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        g = g if scale is None else g * f(scale)
        return m * f(b1) + g * f(1 - b1), v * f(b2) + (g * g) * f(1 - b2)


def adamw(p, m, v, t, lr, b1, b2, eps, wd):
    """The parameters from the new moments, in 64 bits, and the size of what they move by."""
    mh, vh = m / (1 - b1 ** t), v / (1 - b2 ** t)
    step = lr * mh / (np.sqrt(vh) + eps)
    return p * (1 - lr * wd) - step, np.abs(step)
