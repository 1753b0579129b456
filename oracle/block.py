"""Plain 64-bit forms of the block operators (feed-forward block, norms around a
residual sum, AdamW with 32- and 8-bit states), written from their definitions in
elementary torch operations on whatever device the inputs are on. For tests only: it
shares no code with the HIP library."""
from __future__ import annotations

import math

import torch

from .head import philox4x32  # noqa: F401  (the generator, pinned to its published values)

BLOCK = 256
INF = float("inf")


# ---- feed-forward block --------------------------------------------------------------

def activate(kind, a):
    """(act(a), act'(a))"""
    if kind in ("silu", "sigmoid"):
        s = 1 / (1 + torch.exp(-a))
        return (a * s, s * (1 + a * (1 - s))) if kind == "silu" else (s, s * (1 - s))
    if kind == "gelu":
        c = 0.5 * torch.erfc(-a / math.sqrt(2))
        return a * c, c + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (a + 0.044715 * a ** 3))
        return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * k * (1 + 3 * 0.044715 * a * a)
    assert kind == "relu"
    return torch.where(a > 0, a, 0.0 * a), (a > 0).double()


def feed_forward(x, wg, wu, wd, act):
    """(y, a, u, h)"""
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    a, u = x @ wg.t(), x @ wu.t()
    h = activate(act, a)[0] * u
    return h @ wd.t(), a, u, h


def feed_forward_grad(dy, x, wg, wu, wd, act):
    """(dx, dwg, dwu, dwd, da, du)"""
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    _, a, u, h = feed_forward(x, wg, wu, wd, act)
    f, df = activate(act, a)
    dh = dy @ wd
    da, du = dh * u * df, dh * f
    return da @ wg + du @ wu, da.t() @ x, du.t() @ x, dy.t() @ h, da, du


# ---- norms around a residual sum --------------------------------------------------------

def stats(z, kind, eps):
    mean = z.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(z[:, :1])
    return mean, 1 / torch.sqrt(((z - mean) ** 2).mean(1, keepdim=True) + eps)


def _or(v, value, like):
    return torch.full((1,), value, dtype=torch.float64, device=like.device) if v is None else v.to(like.device).double()


def row_gates(gate, rows, like):
    """The gate of each row, [rows][C] or a 1."""
    if gate is None:
        return torch.ones(1, 1, dtype=torch.float64, device=like.device)
    g = gate.to(like.device).double().reshape(-1, gate.shape[-1])
    return g[torch.arange(rows, device=like.device) // max(rows // g.shape[0], 1)]


def residual_norm(b, r, gate, pw, pb, w, bias, kind, post, eps, rs, bs):
    """(out, y, stats [N][4], p)"""
    b, r = b.double(), r.double()
    zero = torch.zeros_like(b[:, :1])
    m1, r1 = stats(b, kind, eps) if post else (zero, zero)
    p = (b - m1) * r1 * _or(pw, 1, b) + _or(pb, 0, b) if post else b
    out = rs * r + bs * row_gates(gate, b.shape[0], b) * p
    m2, r2 = stats(out, kind, eps)
    return out, (out - m2) * r2 * _or(w, 1, b) + _or(bias, 0, b), torch.cat([m1, r1, m2, r2], 1), p


def _through(g, h, rstd, kind):
    t = g - h * (g * h).mean(1, keepdim=True)
    return rstd * (t - g.mean(1, keepdim=True) if kind == "layer" else t)


def residual_norm_grad(dy, dout, b, out, st, gate, pw, pb, w, kind, post, rs, bs):
    """dict of dr, db, weight, bias, and where they exist post_weight, post_bias, gate; t"""
    dy, b, out = dy.double(), b.double(), out.double()
    m1, r1, m2, r2 = (v[:, None] for v in st.double().reshape(-1, 4).unbind(1))
    oh = (out - m2) * r2
    t = _through(dy * _or(w, 1, b), oh, r2, kind)
    if dout is not None:
        t = t + dout.double()
    dp = bs * row_gates(gate, b.shape[0], b) * t
    res = {"dr": rs * t, "weight": (dy * oh).sum(0), "bias": dy.sum(0), "t": t}
    p = b
    if post:
        bh = (b - m1) * r1
        p = bh * _or(pw, 1, b) + _or(pb, 0, b)
        res.update(db=_through(dp * _or(pw, 1, b), bh, r1, kind), post_weight=(dp * bh).sum(0), post_bias=dp.sum(0))
    else:
        res["db"] = dp
    if gate is not None:
        g = gate.reshape(-1, gate.shape[-1])
        rows = b.shape[0] // g.shape[0]
        res["gate"] = torch.stack([bs * (t * p)[k * rows:(k + 1) * rows].sum(0) for k in range(g.shape[0])])
    return res


# ---- AdamW -----------------------------------------------------------------------------

def numbers(first, n, step, seed):
    """The 16-bit numbers (for m, for v) of elements first .. first + n - 1."""
    words = []
    for q in range(first // 4, (first + n + 3) // 4):
        words += philox4x32((q & 0xFFFFFFFF, q >> 32, step & 0xFFFFFFFF, step >> 32),
                            (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    w = torch.tensor(words[first % 4:first % 4 + n], dtype=torch.int64)
    return w & 0xFFFF, w >> 16


def code(x, u, power, top):
    """The code of x, in units of the scale (x = top^power is the scale itself)."""
    c = torch.floor(x.clamp(min=0) ** (1.0 / power))
    c = torch.where(c ** power > x, c - 1, c)
    c = torch.where((c + 1) ** power <= x, c + 1, c)
    share = (x - c ** power) * 65536
    return (c + (share > u.double() * ((c + 1) ** power - c ** power)).double()).clamp(max=top)


def adamw(p, g, m, v, t, lr, beta1, beta2, eps, decay):
    """(p, m, v) in 64 bits."""
    p, g, m, v = (z.double() for z in (p, g, m, v))
    m, v = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    den = torch.sqrt(v / (1 - beta2 ** t)) + eps
    return p * (1 - lr * decay) - lr * (m / (1 - beta1 ** t)) / den, m, v


def nearest(scale, exact):
    """Whether an fp32 scale is the exact one rounded to nearest. Formed in 64 bits in another
    order, the exact one is off by four roundings of 2^-53, and where it lies halfway between
    two fp32 numbers (0.9 M + 0.1 g does, for M and g of few digits that 5 divides) either may
    be taken."""
    step = torch.nextafter(scale, torch.tensor(INF)).double() - scale.double()
    return bool(((scale.double() - exact).abs() <= step / 2 + 2.0 ** -51 * exact).all())


def encode(m, v, first, t, seed, scales=None):
    """(m codes, v codes, m scales, v scales) of one tensor's new m and v; with `scales` for
    those, once they are seen to be nearest."""
    n = m.numel()
    if scales is not None:
        for s, z in zip(scales, (m.abs(), v)):
            top = torch.stack([b.max() for b in z.split(BLOCK)])
            assert nearest(s, top), "scales"
    um, uv = numbers(first, n, t, seed)
    mk, vk, ms, vs = [], [], [], []
    for i in range(0, n, BLOCK):
        a, b = m[i:i + BLOCK], v[i:i + BLOCK]
        M, V = (a.abs().max().float(), b.max().float()) if scales is None else (q[i // BLOCK] for q in scales)
        if not (torch.isfinite(M) and torch.isfinite(V)) or torch.isnan(a).any() or torch.isnan(b).any():
            ms.append(float("nan"))
            vs.append(float("nan"))
            mk.append(torch.zeros(a.numel()))
            vk.append(torch.zeros(a.numel()))
            continue
        ms.append(M.item())
        vs.append(V.item())
        x = a.abs() * (127.0 ** 2 / M.double()) if M > 0 else torch.zeros_like(a)
        y = b * (255.0 ** 4 / V.double()) if V > 0 else torch.zeros_like(b)
        mk.append(code(x, um[i:i + BLOCK], 2, 127) * torch.sign(a))
        vk.append(torch.where(b > 0, code(y, uv[i:i + BLOCK], 4, 255).clamp(min=1), torch.zeros_like(b)))
    return (torch.cat(mk).to(torch.int8), torch.cat(vk).to(torch.uint8), torch.tensor(ms), torch.tensor(vs))


def decode(mk, vk, ms, vs):
    k, q = mk.double(), vk.double()
    s, z = ms.double().repeat_interleave(BLOCK)[:k.numel()], vs.double().repeat_interleave(BLOCK)[:k.numel()]
    return torch.sign(k) * s * (k / 127) ** 2, z * (q / 255) ** 4
