"""Plain 64-bit forms of the training-head operators (layer norm, dropout,
linear cross entropy), written from their definitions in elementary torch
operations on whatever device the inputs are on. Checker only: it shares no
code with the HIP library."""
from __future__ import annotations

import numpy as np
import torch

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox4x32(counter, key, rounds=10):
    """Philox4x32 on Python integers: 4 counter words, 2 key words -> 4 words."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        p0, p1 = c[0] * M0, c[2] * M1
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + W0) & 0xFFFFFFFF, (k[1] + W1) & 0xFFFFFFFF]
    return c


def numbers(first: int, n: int, seed: int, offset: int) -> np.ndarray:
    """The 16-bit numbers of elements first .. first + n - 1."""
    e = np.uint64(first) + np.arange(n, dtype=np.uint64)
    blk = e // np.uint64(8) + np.uint64(offset)
    m = np.uint64(0xFFFFFFFF)
    s = np.uint64(32)
    c = [blk & m, blk >> s, np.zeros_like(blk), np.zeros_like(blk)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(M0), c[2] * np.uint64(M1)
        c = [(p1 >> s) ^ c[1] ^ np.uint64(k[0]), p1 & m, (p0 >> s) ^ c[3] ^ np.uint64(k[1]), p0 & m]
        k = [(k[0] + W0) & 0xFFFFFFFF, (k[1] + W1) & 0xFFFFFFFF]
    j = (e % np.uint64(8)).astype(np.int64)
    word = np.stack(c)[j // 2, np.arange(n)]
    return ((word >> (np.uint64(16) * (j % 2).astype(np.uint64))) & np.uint64(0xFFFF)).astype(np.int64)


def drop_factors(shape, p, seed, offset=0, first=0, device="cpu"):
    """What each element is multiplied by (0 where dropped), float64."""
    T = int(np.floor(p * 65536 + 0.5))
    n = int(np.prod(shape))
    if T == 0:
        return torch.ones(shape, dtype=torch.float64, device=device)
    if T == 65536:
        return torch.zeros(shape, dtype=torch.float64, device=device)
    keep = numbers(first, n, seed, offset) >= T
    return torch.from_numpy(np.where(keep, 65536.0 / (65536 - T), 0.0)).reshape(shape).to(device)


def _vec(v, dim, nd, like):
    if v is None:
        return None
    return v.to(like.device).double().reshape([-1 if i == dim else 1 for i in range(nd)])


def layer_norm(x, weight, bias, eps, dim):
    """(y, mean, rstd) with the channels at `dim`, before dropout."""
    x = x.double()
    mean = x.mean(dim, keepdim=True)
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(dim, keepdim=True) + eps)
    y = d * rstd
    if weight is not None:
        y = y * _vec(weight, dim, x.dim(), x)
    if bias is not None:
        y = y + _vec(bias, dim, x.dim(), x)
    return y, mean.squeeze(dim), rstd.squeeze(dim)


def layer_norm_grad(dz, x, weight, mean, rstd, dim):
    """(dx, dweight, dbias) for dz, the gradient of y after dropout's own."""
    x, dz = x.double(), dz.double()
    r = rstd.double().unsqueeze(dim)
    h = (x - mean.double().unsqueeze(dim)) * r
    g = dz if weight is None else dz * _vec(weight, dim, x.dim(), x)
    dx = r * (g - g.mean(dim, keepdim=True) - h * (g * h).mean(dim, keepdim=True))
    rest = [i for i in range(x.dim()) if i != dim]
    return dx, (dz * h).sum(rest) if rest else dz * h, dz.sum(rest) if rest else dz


def cross_entropy(x, w, target):
    """(loss, lse) per row; both 0 where the target is outside [0, V)."""
    ok = (target >= 0) & (target < w.shape[0])
    logits = torch.where(ok[:, None], x.double(), 0.0) @ w.double().t()
    lse = torch.logsumexp(logits, 1)
    hit = logits.gather(1, torch.where(ok, target, 0)[:, None]).squeeze(1)
    zero = torch.zeros_like(lse)
    return torch.where(ok, lse - hit, zero), torch.where(ok, lse, zero)


def cross_entropy_grad(grad, x, w, target, lse=None):
    """(dx, dw, G) in 64 bits."""
    ok = (target >= 0) & (target < w.shape[0])
    xd = torch.where(ok[:, None], x.double(), 0.0)
    wd = w.double()
    logits = xd @ wd.t()
    lse = torch.logsumexp(logits, 1) if lse is None else lse.double()
    G = torch.exp(logits - lse[:, None])
    rows = torch.nonzero(ok).squeeze(1)
    G[rows, target[rows]] -= 1.0
    G = torch.where(ok[:, None], G * grad.double()[:, None], 0.0)
    return G @ wd, G.t() @ xd, G
