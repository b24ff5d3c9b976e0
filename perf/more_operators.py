"""Cases of the training block's operators: layer norm with its backward (the
sums of the weight's and the bias's gradients among it), products of ragged
groups of rows with a weight matrix each (forward, and both gradients), and the
AdamW step over many tensors with moments in 32 or in 8 bits; each in a plain
form of elementary torch operations and as the framework's call.

Moments in 8 bits.  256 neighbouring elements of a tensor form a block; for
each of the two moments a block has one byte e, the exponent field of its
largest magnitude as an FP32 number, at least 16.  The first moment is a sign,
4 exponent bits (bias 7) and 3 of mantissa, times 2^(e - 134); the second one
5 exponent bits (bias 15) and 3 of mantissa, times 2^(e - 142).  What is written is rounded
up or down at random, with the odds that make the mean right: element i of
the blocks, counted through all tensors in their order, takes word i mod 4 of
Philox4x32-10 at the counter (i div 4, step), keyed by the seed; its low 16 bits
decide for the first moment, its high ones for the second.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 256


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of each of 64 users: the latency of a serving step
        dict(name="norm forward, 64 tokens", op="ln_fwd", T=64, D=512, x="bf16", y="bf16"),
        # the layer workload's batch (8 users of 8K to 32K tokens, 4 heads x 128): the residual stream into a projection
        dict(name="norm forward, layer batch", op="ln_fwd", T=161_293, D=512, x="fp32", y="bf16"),
        # a heavy-tailed training batch
        dict(name="norm backward, heavy-tailed batch", op="ln_bwd", T=16_410, D=512, x="bf16", y="bf16"),
        # FP32 rows of an odd width
        dict(name="norm backward, fp32 rows of 301", op="ln_bwd", T=4_099, D=301, x="fp32", y="fp32"),
        # the same serving step through a projection with a weight for each of 8 kinds of tokens
        dict(name="products, 64 tokens in 8 groups", op="gg_fwd", T=64, E=8, K=512, N=2048, skew=0.5, y="bf16", lens_seed=1),
        # the layer workload's batch through the layer's input projection, one weight for each of 8 kinds
        dict(name="products, layer batch in 8 groups", op="gg_fwd", T=161_293, E=8, K=512, N=2048, skew=1.0, y="bf16",
             lens_seed=2),
        # both gradients of it for a heavy-tailed training batch, 16 kinds of which a few hold most tokens
        dict(name="gradients, heavy-tailed, 16 groups", op="gg_bwd", T=16_410, E=16, K=512, N=2048, skew=1.2, y="bf16",
             lens_seed=3),
        # many small groups, widths that fill no tile
        dict(name="gradients, 1111 rows in 24 groups", op="gg_bwd", T=1_111, E=24, K=264, N=520, skew=1.0, y="bf16",
             lens_seed=4),
        # the tensors of one layer: W1, W2, the two bias tables, a norm's weight and bias, weights of 7 tasks and a temperature
        dict(name="adamw, one layer", op="adamw", layers=1, D=512, experts=0, bits=32, grad="fp32", copies=True),
        # a stack of 16 such layers
        dict(name="adamw, 16 layers", op="adamw", layers=16, D=512, experts=0, bits=32, grad="fp32", copies=True),
        # the same stack with moments in 8 bits, and the moments read back
        dict(name="adamw 8 bits, 16 layers", op="adamw", layers=16, D=512, experts=0, bits=8, grad="fp32", copies=True),
        # 2 layers whose input projection has 16 weights, BF16 gradients, moments in 8 bits, and the moments read back
        dict(name="adamw 8 bits, 2 layers of 16 groups", op="adamw", layers=2, D=512, experts=16, bits=8, grad="bf16",
             copies=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "gg_fwd", "gg_bwd", "adamw", "adamw"])
    if op in ("ln_fwd", "ln_bwd"):
        c = dict(op=op, T=1, D=rng.choice([_log(rng, 1, 4096), 8 * _log(rng, 4, 512)]), x=rng.choice(["bf16", "fp32"]),
                 y=rng.choice(["bf16", "fp32"]))
        return dict(c, T=_log(rng, 1, min(160_000, int(4e8 / work(c)["bytes"]))))
    if op in ("gg_fwd", "gg_bwd"):
        c = dict(op=op, T=1, E=_log(rng, 1, 64), K=8 * _log(rng, 4, 128), N=8 * _log(rng, 4, 256), skew=rng.choice([0.0, 0.7, 1.3]),
                 y=rng.choice(["bf16", "fp32"]) if op == "gg_fwd" else "bf16", lens_seed=rng.randrange(1 << 30))
        return dict(c, T=_log(rng, 1, min(160_000, int((3e11 if op == "gg_fwd" else 1.5e11) / (4 * c["K"] * c["N"])))))
    return dict(op=op, layers=rng.randint(1, 12), D=8 * rng.randint(4, 64), experts=rng.choice([0, 0, 3]), bits=rng.choice([32, 8]),
                grad=rng.choice(["fp32", "bf16"]), copies=rng.random() < 0.5)


def _groups(c):
    """Rows of every group: sizes like 1 / rank^skew in random order, some groups empty where there are many."""
    r = random.Random(c["lens_seed"])
    share = [(i + 1.0) ** -c["skew"] for i in range(c["E"])]
    if c["E"] > 8:
        share = [0.0 if i and r.random() < 0.1 else w for i, w in enumerate(share)]
    n = [int(c["T"] * w / sum(share)) for w in share]
    for _ in range(c["T"] - sum(n)):
        n[r.choices(range(c["E"]), share)[0]] += 1
    r.shuffle(n)
    return n


def _tensors(c):
    """(elements, whether it decays) of every tensor."""
    D, one = c["D"], []
    one.append((max(1, c["experts"]) * D * 4 * D, True))
    one.append((D * D, True))
    one += [(4 * 128, False), (4 * 64, False), (D, False), (D, False), (7, False), (1, False)]
    return one * c["layers"]


# ------------------------------------------------------------------ inputs

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)
    return g


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, device=DEV, generator=g, dtype=torch.float32).to(dtype)


def prepare(c, seed):
    g = _gen(seed)
    s = dict(c=c, seed=seed)
    if c["op"] in ("ln_fwd", "ln_bwd"):
        T, D = c["T"], c["D"]
        # rows of a residual stream: sizes that differ from row to row, a mean that is not zero
        size = 0.2 + torch.rand(T, 1, device=DEV, generator=g) * 3
        s["x"] = (_normal(g, T, D) * size + 0.3 * _normal(g, T, 1)).to(TYPES[c["x"]])
        s["w"], s["b"] = 1 + 0.2 * _normal(g, D), 0.1 * _normal(g, D)
        if c["op"] == "ln_bwd":
            s["dy"] = _normal(g, T, D, dtype=TYPES[c["y"]])
            x = s["x"].double()
            s["mean"] = x.mean(-1).float()
            s["rstd"] = (x.var(-1, unbiased=False) + 1e-5).rsqrt().float()
        return s
    if c["op"] in ("gg_fwd", "gg_bwd"):
        n = _groups(c)
        s["n"] = n
        s["offsets"] = torch.tensor([0] + n, dtype=torch.int64).cumsum(0).to(DEV)
        s["x"] = _normal(g, c["T"], c["K"], dtype=torch.bfloat16)
        s["w"] = (_normal(g, c["E"], c["K"], c["N"]) * c["K"] ** -0.5).bfloat16()
        if c["op"] == "gg_bwd":
            s["dy"] = _normal(g, c["T"], c["N"], dtype=torch.bfloat16)
        return s
    # the tensors lie in one buffer a kind, each begins on a block
    sizes = _tensors(c)
    ends, total = [], 0
    for n, _ in sizes:
        ends.append((total, n))
        total += -(-n // BLOCK) * BLOCK
    s["where"], s["decays"] = ends, [d for _, d in sizes]
    live = torch.zeros(total, device=DEV)
    decay = torch.zeros(total, device=DEV)
    for (at, n), d in zip(ends, s["decays"]):
        live[at:at + n] = 1
        decay[at:at + n] = 0.01 if d else 0.0
    s["hyper"] = dict(lr=3e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
    s["steps"] = 1000 + seed % 7
    s["decay"] = decay
    s["p"] = 0.02 * _normal(g, total) * live
    s["copy"] = s["p"].bfloat16() if c["copies"] else None
    # gradients whose sizes differ from row to row, moments of some hundred steps of them
    size = 1e-3 * torch.exp(2 * _normal(g, total // BLOCK, 1))
    s["g"] = ((_normal(g, total // BLOCK, BLOCK) * size).view(-1) * live).to(TYPES[c["grad"]])
    m = (_normal(g, total // BLOCK, BLOCK) * size * 0.23).view(-1) * live
    v = ((0.6 + 0.8 * torch.rand(total // BLOCK, BLOCK, device=DEV, generator=g)) * size).view(-1).square() * live
    s["scale"] = torch.full((1,), 0.75, device=DEV)      # what clipping by the gradients' norm left
    s["key"] = 0x1234_5678_9ABC + seed
    if c["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        s["m"], s["me"] = _nearest8(m, 134, 120, 0x7E)
        s["v"], s["ve"] = _nearest8(v, 142, 112, 0xFF)
        if "values" not in _TABLES:
            _TABLES["values"] = [_decode_table(4, 7, True), _decode_table(5, 15, False)]
    return s


# ------------------------------------------- moments in 8 bits, plain form

_TABLES = {}


def _decode_table(bits, bias, signed):
    t = []
    for code in range(256):
        mag = code & 127 if signed else code
        e, f = mag >> 3, mag & 7
        x = math.ldexp(f / 8, 1 - bias) if e == 0 else math.ldexp(1 + f / 8, e - bias)
        x = math.nan if signed and mag == 127 else x
        t.append(-x if signed and code > 127 else x)
    return torch.tensor(t, dtype=torch.float32, device=DEV)


def _pow2(e):
    """2^e for integer tensors -126 <= e <= 127, FP32."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _top(x):
    """The byte of every block of |x| (FP32): the exponent field of its largest finite value, at least 16."""
    a = x.view(-1, BLOCK).abs()
    a = torch.where(a < math.inf, a, torch.zeros_like(a))
    return (a.amax(-1).view(torch.int32) >> 23).clamp(min=16)


def _codes(x, e, off, shift, top, noise):
    """Magnitude codes of x (FP32) in blocks with the bytes e; noise: what is added to the 20 bits that fall away."""
    a = x.view(-1, BLOCK).abs() * _pow2(off - e)[:, None] * 2.0 ** -shift
    bits = (a.view(torch.int32) + noise) >> 20
    return torch.where(a < math.inf, bits.clamp(max=top), torch.full_like(bits, 0x7F if top == 0x7E else top))


def _pack8(x, e, off, shift, top, noise):
    code = _codes(x, e, off, shift, top, noise)
    if top == 0x7E:
        code = code | (torch.signbit(x).view(-1, BLOCK).int() << 7)
    return code.to(torch.uint8).view(-1)


def _nearest8(x, off, shift, top):
    """Codes nearest to x, and the blocks' bytes."""
    e = _top(x)
    return _pack8(x, e, off, shift, top, 1 << 19), e.to(torch.uint8)


def _values8(code, e, off, which):
    return (_TABLES["values"][which][code.view(-1, BLOCK).long()] * _pow2(e.int() - off)[:, None]).view(-1)


def _philox(n4, step, key):
    """[n4, 4] words of 32 bits at the counters (i, step), in int64 tensors."""
    low = 0xFFFFFFFF
    i = torch.arange(n4, device=DEV, dtype=torch.int64)
    x0, x1 = i & low, i >> 32
    x2, x3 = torch.full_like(i, step & low), torch.full_like(i, step >> 32)
    k0, k1 = key & low, key >> 32
    for _ in range(10):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57
        x0, x1, x2, x3 = ((b >> 32) & low) ^ x1 ^ k0, b & low, ((a >> 32) & low) ^ x3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([x0, x1, x2, x3], -1)


# -------------------------------------------------------------- plain form

def _plain_ln(s):
    x, w = s["x"].float(), s["w"]
    if s["c"]["op"] == "ln_fwd":
        mean = x.mean(-1, keepdim=True)
        xc = x - mean
        rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + 1e-5)
        y = (xc * rstd * w + s["b"]).to(TYPES[s["c"]["y"]])
        return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]}
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    e = dy * w
    dx = rstd * (e - e.mean(-1, keepdim=True) - xh * (e * xh).mean(-1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def _plain_groups(s):
    c = s["c"]
    out = {}
    if c["op"] == "gg_fwd":
        out["y"] = torch.empty(c["T"], c["N"], device=DEV, dtype=TYPES[c["y"]])
    else:
        out["dx"], out["dw"] = torch.empty_like(s["x"]), torch.empty(c["E"], c["K"], c["N"], device=DEV)
    at = 0
    for e, n in enumerate(s["n"]):
        x, w = s["x"][at:at + n].float(), s["w"][e].float()
        if c["op"] == "gg_fwd":
            out["y"][at:at + n] = x @ w
        else:
            dy = s["dy"][at:at + n].float()
            out["dx"][at:at + n] = dy @ w.T
            out["dw"][e] = x.T @ dy
        at += n
    return out


def _plain_adamw(s):
    c, h = s["c"], s["hyper"]
    s["steps"] += 1
    b1, b2 = h["beta1"], h["beta2"]
    c1, c2 = 1 - b1 ** s["steps"], 1 - b2 ** s["steps"]
    g = s["g"].float() * s["scale"]
    m, v = s["m"], s["v"]
    if c["bits"] == 8:
        m, v = _values8(m, s["me"], 134, 0), _values8(v, s["ve"], 142, 1)
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    p = s["p"] * (1 - h["lr"] * s["decay"]) - (h["lr"] / c1) * (m / (v.sqrt() * c2 ** -0.5 + h["eps"]))
    s["p"] = p
    out = {"p": p}
    if c["copies"]:
        out["copy"] = s["copy"] = p.bfloat16()
    if c["bits"] == 32:
        s["m"], s["v"] = m, v
        return dict(out, m=m, v=v)
    word = _philox(p.numel() // 4, s["steps"], s["key"]).view(-1, BLOCK)
    s["me"], s["ve"] = _top(m), _top(v)
    s["m"] = _pack8(m, s["me"], 134, 120, 0x7E, ((word & 0xFFFF) << 4) + 8)
    s["v"] = _pack8(v, s["ve"], 142, 112, 0xFF, ((word >> 16) << 4) + 8)
    return dict(out, m=_values8(s["m"], s["me"], 134, 0).bfloat16(), v=_values8(s["v"], s["ve"], 142, 1).bfloat16())


# ----------------------------------------------------------- the framework

def _open(s):
    """The handles that a program keeps beside its buffers."""
    c = s["c"]
    if c["op"] in ("ln_fwd", "ln_bwd"):
        from hstu_jagged_attention_02_gb300.norm import LNProblem
        return LNProblem(s["x"], s["w"], s["b"], eps=1e-5, out_dtype=TYPES[c["y"]], dy=s.get("dy"), mean=s.get("mean"),
                         rstd=s.get("rstd"))
    if c["op"] in ("gg_fwd", "gg_bwd"):
        from hstu_jagged_attention_02_gb300.groups import GroupProblem
        return GroupProblem(s["x"], s["w"], s["offsets"], out_dtype=TYPES[c["y"]], dy=s.get("dy"))
    from hstu_jagged_attention_02_gb300.optim import AdamW, Moments8
    cut = lambda t: [t[at:at + n] for at, n in s["where"]]  # noqa: E731
    if c["bits"] == 32:
        moments = list(zip(cut(s["m"]), cut(s["v"])))
    else:
        es = [(s["me"][at // BLOCK:-(-(at + n) // BLOCK)], s["ve"][at // BLOCK:-(-(at + n) // BLOCK)]) for at, n in s["where"]]
        moments = [Moments8(m, v, me, ve) for m, v, (me, ve) in zip(cut(s["m"]), cut(s["v"]), es)]
        s["m16"], s["v16"] = (torch.zeros(s["p"].numel(), device=DEV, dtype=torch.bfloat16) for _ in range(2))
    h = s["hyper"]
    return AdamW(cut(s["p"]), cut(s["g"]), lr=h["lr"], betas=(h["beta1"], h["beta2"]), eps=h["eps"],
                 weight_decay=[h["weight_decay"] if d else 0.0 for d in s["decays"]], copies=cut(s["copy"]) if c["copies"] else None,
                 moments=moments, grad_scale=s["scale"], steps=s["steps"], seed=s["key"])


def run(s):
    if not own:
        op = s["c"]["op"]
        return _plain_ln(s) if op in ("ln_fwd", "ln_bwd") else (_plain_groups(s) if op in ("gg_fwd", "gg_bwd") else _plain_adamw(s))
    h = s.get("handle")
    if h is None:
        h = s["handle"] = _open(s)
    c = s["c"]
    if c["op"] == "ln_fwd":
        h.forward()
        return {"y": h.y, "mean": h.mean, "rstd": h.rstd}
    if c["op"] == "ln_bwd":
        h.backward()
        return {"dx": h.dx, "dw": h.d_weight, "db": h.d_bias}
    if c["op"] == "gg_fwd":
        h.forward()
        return {"y": h.y}
    if c["op"] == "gg_bwd":
        h.backward()
        return {"dx": h.dx, "dw": h.dw}
    h.step()
    out = {"p": s["p"], "m": s["m"], "v": s["v"]}
    if c["copies"]:
        out["copy"] = s["copy"]
    if c["bits"] == 8:
        if "read" not in s:
            s["read"] = h.reader([(s["m16"][at:at + n], s["v16"][at:at + n]) for at, n in s["where"]])
        s["read"].run()
        out.update(m=s["m16"], v=s["v16"])
    return out


# -------------------------------------------------------------------- work

def work(c):
    size = {"bf16": 2, "fp32": 4}
    if c["op"] in ("ln_fwd", "ln_bwd"):
        n = c["T"] * c["D"]
        if c["op"] == "ln_fwd":
            return {"bytes": n * (size[c["x"]] + size[c["y"]]) + 8 * c["T"] + 8 * c["D"], "flops": 8 * n}
        return {"bytes": n * (2 * size[c["x"]] + size[c["y"]]) + 8 * c["T"] + 12 * c["D"], "flops": 16 * n}
    if c["op"] in ("gg_fwd", "gg_bwd"):
        used = sum(1 for n in _groups(c) if n)
        T, K, N = c["T"], c["K"], c["N"]
        if c["op"] == "gg_fwd":
            return {"bytes": 2 * T * K + 2 * used * K * N + size[c["y"]] * T * N, "flops": 2 * T * K * N}
        return {"bytes": 2 * T * (K + N) + 2 * used * K * N + 2 * T * K + 4 * c["E"] * K * N, "flops": 4 * T * K * N}
    n = sum(k for k, _ in _tensors(c))
    # parameter and moments read and written, gradient read, copy written; 8 bits: codes read back as values too
    moments = 16 if c["bits"] == 32 else 4 + 2 + 4
    return {"bytes": n * (8 + size[c["grad"]] + (2 if c["copies"] else 0) + moments), "flops": n * (16 if c["bits"] == 32 else 60)}


# ------------------------------------------------- the definition, 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("ln_fwd", "ln_bwd"):
        x = s["x"].double().requires_grad_(c["op"] == "ln_bwd")
        if c["op"] == "ln_fwd":
            var, mean = torch.var_mean(x, -1, unbiased=False)
            r = 1 / (var + 1e-5).sqrt()
            return {"y": (x - mean[:, None]) * r[:, None] * s["w"].double() + s["b"].double(), "mean": mean, "rstd": r}
        # through the derivative of the definition
        w, b = (s[n].double().requires_grad_() for n in ("w", "b"))
        var, mean = torch.var_mean(x, -1, unbiased=False, keepdim=True)
        dx, dw, db = torch.autograd.grad((x - mean) / (var + 1e-5).sqrt() * w + b, (x, w, b), s["dy"].double())
        return {"dx": dx, "dw": dw, "db": db}
    if c["op"] in ("gg_fwd", "gg_bwd"):
        parts = list(zip(s["x"].split(s["n"]), s["w"].unbind(0), s["dy"].split(s["n"]) if "dy" in s else s["n"]))
        if c["op"] == "gg_fwd":
            return {"y": torch.cat([torch.mm(x.double(), w.double()) for x, w, _ in parts])}
        return {"dx": torch.cat([torch.einsum("tn,kn->tk", d.double(), w.double()) for _, w, d in parts]),
                "dw": torch.stack([torch.einsum("tk,tn->kn", x.double(), d.double()) for x, _, d in parts])}
    return _exact_adamw(s)


def _exact_adamw(s):
    c, h = s["c"], s["hyper"]
    b1, b2, t = h["beta1"], h["beta2"], s["steps"] + 1
    g = s["g"].double() * s["scale"].double()
    if c["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        m, v = (tab.double()[code.long()] * torch.exp2((e.double() - off).repeat_interleave(BLOCK))
                for tab, code, e, off in zip(_TABLES["values"], (s["m"], s["v"]), (s["me"], s["ve"]), (134, 142)))
    m += (1 - b1) * (g - m)
    v += (1 - b2) * (g * g - v)
    mh, vh = m / (1 - math.pow(b1, t)), v / (1 - math.pow(b2, t))
    p = s["p"].double()
    p = p - h["lr"] * (s["decay"].double() * p + mh / (vh.sqrt() + h["eps"]))
    out = {"p": p}
    if c["copies"]:
        out["copy"] = p
    if c["bits"] == 8:
        word = _philox(p.numel() // 4, t, s["key"]).view(-1)
        m = _exact8(m, word & 0xFFFF, 4, 7, 134)
        v = _exact8(v, word >> 16, 5, 15, 142)
    return dict(out, m=m, v=v)


def _exact8(x, word, ebits, bias, off):
    """Up to the next value that can be held, or down to the one below, by the odds in word."""
    a = x.abs()
    top = a.view(-1, BLOCK).amax(-1)
    e = (torch.frexp(top)[1] - 1 + 127).clamp(min=16)                       # 2^(e - 127) <= top < 2^(e - 126)
    unit = torch.exp2((e - off).double()).repeat_interleave(BLOCK)
    a = a / unit
    least = 1 - bias
    step = torch.exp2((torch.frexp(a.clamp(min=2.0 ** least))[1] - 1 - 3).double())
    down = torch.floor(a / step)
    up = (a / step - down) + (word.double() * 16 + 8) / 2 ** 20 >= 1
    return torch.sign(x) * (down + up.double()) * step * unit
