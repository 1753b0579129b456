"""Workloads of the training-head operators: layer norm over the channels of
a feature map, dropout from a counter-based generator, and the softmax cross
entropy of a linear classifier, each with its gradient.

A case is a dict of plain values. ``prepare`` makes the inputs on the GPU,
``run`` takes one pass through an operator (elementary torch operations in
fp32, or the library's kernels where ``own`` is true), ``exact`` computes the
definition in 64 bits, ``work`` states the bytes and operations of a pass.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


# ---- cases -----------------------------------------------------------------

def _ln(name, op, layout, N, C, P, xt, yt, p=0.0):
    return {"name": name, "op": op, "layout": layout, "N": N, "C": C, "P": P, "x": xt, "y": yt, "p": p}


def _xent(name, op, N, V, D, t):
    return {"name": name, "op": op, "N": N, "V": V, "D": D, "t": t}


def listed():
    return [
        # one position of a 512-channel feature map: a single request, latency only
        _ln("ln_fwd_one", "ln_fwd", "nhwc", 1, 512, 1, "bf16", "bf16"),
        # the default output of the 64-channel 56x56 layer (fp32 NCHW), normalised
        # over its channels and handed on in half precision
        _ln("ln_fwd_nchw", "ln_fwd", "nchw", 32, 64, 3136, "f32", "f16"),
        # the largest training batch of wide rows, dropout fused into the output
        _ln("ln_fwd_wide_drop", "ln_fwd", "nhwc", 32768, 4096, 1, "bf16", "bf16", 0.1),
        # gradient on the 256-channel 56x56 layer's NCHW output in fp32
        _ln("ln_bwd_nchw", "ln_bwd", "nchw", 64, 256, 3136, "f32", "f32"),
        # gradient with an odd channel count and an odd number of rows
        _ln("ln_bwd_odd", "ln_bwd", "nhwc", 50001, 1001, 1, "f16", "f16"),
        # the same wide rows as above, backward through the fused dropout
        _ln("ln_bwd_wide_drop", "ln_bwd", "nhwc", 32768, 4096, 1, "bf16", "bf16", 0.1),
        # pooled features of one small batch, an odd element count
        {"name": "drop_small", "op": "drop", "n": 32 * 511 + 3, "t": "f32", "p": 0.5},
        # the activations of a large batch in half precision
        {"name": "drop_large", "op": "drop", "n": 1 << 27, "t": "bf16", "p": 0.1},
        # scoring one row against a large class matrix: the matrix is read once
        _xent("xent_loss_one", "xent_loss", 1, 65536, 2048, "bf16"),
        # evaluation of an odd batch over an odd number of classes
        _xent("xent_loss_odd", "xent_loss", 4097, 50001, 1032, "f16"),
        # fine-tuning step of a 1000-class head on 512 pooled channels, fp32
        _xent("xent_train_small", "xent_train", 64, 1000, 512, "f32"),
        # training step over a large class set
        _xent("xent_train_large", "xent_train", 8192, 131072, 4096, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "drop", "xent_loss", "xent_train", "xent_train"])
    t = rng.choice(["f32", "f16", "bf16"])
    if op == "drop":
        return {"op": op, "n": _log(rng, 1000, 1 << 26), "t": t, "p": rng.choice([0.1, 0.25, 0.5])}
    if op in ("ln_fwd", "ln_bwd"):
        layout = rng.choice(["nhwc", "nchw"])
        C = _log(rng, 32, 1024) if layout == "nchw" else _log(rng, 32, 8192)
        if rng.random() < 0.5:
            C = -(-C // 32) * 32
        side = rng.choice([7, 14, 28, 56])
        P = side * side if layout == "nchw" else 1
        N = _log(rng, 1, max(1, (1 << 26) // (C * P)))
        yt = rng.choice([t, "f16", "bf16"]) if t == "f32" else t
        return {"op": op, "layout": layout, "N": N, "C": C, "P": P, "x": t, "y": yt,
                "p": rng.choice([0.0, 0.0, 0.1, 0.5])}
    D = _log(rng, 64, 4096)
    r = rng.random()
    if r < 0.4:
        D = -(-D // 64) * 64
    elif r < 0.8:
        D = -(-D // 8) * 8
    return {"op": op, "N": _log(rng, 1, 8192), "V": _log(rng, 100, 131072 if t != "f32" else 50000), "D": D, "t": t}


# ---- the operators in their plain form ---------------------------------------

_M32 = 0xFFFFFFFF


def _philox_u16(n, seed, offset):
    """The 16-bit numbers of elements 0 .. n-1, as int64: Philox4x32-10, one
    128-bit block per 8 elements, block b on counter (b, 0) with the seed as key."""
    nb = -(-n // 8)
    ctr = torch.arange(nb, device=DEV, dtype=torch.int64) + offset
    c0, c1 = ctr & _M32, (ctr >> 32) & _M32
    c2, c3 = torch.zeros_like(c0), torch.zeros_like(c0)
    k0, k1 = seed & _M32, (seed >> 32) & _M32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57          # 64-bit products, wrapped
        c0, c1, c2, c3 = (((b >> 32) & _M32) ^ c1 ^ k0, b & _M32, ((a >> 32) & _M32) ^ c3 ^ k1, a & _M32)
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    w = torch.stack([c0, c1, c2, c3], dim=1)
    return torch.stack([w & 0xFFFF, w >> 16], dim=2).reshape(-1)[:n]


def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _drop_plain(x, p, seed, offset):
    """x (contiguous, any shape, fp32) with each element dropped or scaled."""
    T = _threshold(p)
    keep = (_philox_u16(x.numel(), seed, offset) >= T).reshape(x.shape)
    return torch.where(keep, x * (65536.0 / (65536 - T)), torch.zeros((), device=x.device))


def _ln_fwd_plain(s):
    x = s["x"].float()
    c = s["cdim"]
    mean = x.mean(dim=c, keepdim=True)
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(dim=c, keepdim=True) + EPS)
    y = d * rstd * s["wv"] + s["bv"]
    if s["p"] > 0:
        y = _drop_plain(y, s["p"], s["seed"], s["offset"])
    return [y.to(s["yt"]), mean.squeeze(c), rstd.squeeze(c)]


def _ln_bwd_plain(s):
    x, dz = s["x"].float(), s["dy"].float()
    c = s["cdim"]
    if s["p"] > 0:
        dz = _drop_plain(dz, s["p"], s["seed"], s["offset"])
    rstd = s["rstd"].unsqueeze(c)
    xhat = (x - s["mean"].unsqueeze(c)) * rstd
    g = dz * s["wv"]
    dx = rstd * (g - g.mean(dim=c, keepdim=True) - xhat * (g * xhat).mean(dim=c, keepdim=True))
    rest = [i for i in range(x.dim()) if i != c]
    return [dx.to(s["x"].dtype), (dz * xhat).sum(dim=rest), dz.sum(dim=rest)]


def _xent_plain(s, train):
    x, w, t = s["x"].float(), s["w"].float(), s["target"]
    V = w.shape[0]
    ok = (t >= 0) & (t < V)
    x = torch.where(ok[:, None], x, torch.zeros((), device=DEV))
    logits = x @ w.t()
    m = logits.amax(dim=1, keepdim=True)
    e = (logits - m).exp_()
    tot = e.sum(dim=1, keepdim=True)
    lse = (m + tot.log()).squeeze(1)
    tc = torch.where(ok, t, torch.zeros_like(t))
    zero = torch.zeros((), device=DEV)
    hit = logits.gather(1, tc[:, None]).squeeze(1)
    loss = torch.where(ok, lse - hit, zero)
    lse = torch.where(ok, lse, zero)
    if not train:
        return [loss, lse]
    del logits
    g = torch.where(ok, s["grad"], zero)
    G = e.mul_(g[:, None] / tot)
    rows = torch.arange(t.numel(), device=DEV)
    G[rows, tc] -= g
    return [loss, lse, (G @ w).to(s["x"].dtype), (G.t() @ x).to(s["w"].dtype)]


# ---- prepare and run -----------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def rnd(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype)

    op = case["op"]
    s = {"op": op, "seed": (0x1234567_00000000 + 7919 * seed) & (2 ** 63 - 1), "offset": 0}
    if op == "drop":
        s["p"] = case["p"]
        s["x"] = rnd(case["n"]).to(TYPES[case["t"]])
        if own:
            s["y"] = torch.empty_like(s["x"])
        return s
    if op in ("ln_fwd", "ln_bwd"):
        N, C, P = case["N"], case["C"], case["P"]
        nchw = case["layout"] == "nchw"
        shape = (N, C, P) if nchw else (N, C)
        stat = (N, P) if nchw else (N,)
        vec = (C, 1) if nchw else (C,)
        s.update(p=case["p"], layout=case["layout"], cdim=1, yt=TYPES[case["y"]])
        # convolution features: each channel with its own level and spread
        level, spread = rnd(*vec), 1.0 + 0.5 * rnd(*vec).abs()
        s["x"] = (rnd(*shape) * spread + level).to(TYPES[case["x"]])
        s["weight"] = 1.0 + 0.2 * rnd(C)
        s["bias"] = 0.2 * rnd(C)
        s["wv"], s["bv"] = s["weight"].view(vec), s["bias"].view(vec)
        if op == "ln_bwd":
            xf = s["x"].float()
            s["mean"] = xf.mean(dim=1)
            xf = xf - s["mean"].unsqueeze(1)
            s["rstd"] = 1.0 / torch.sqrt((xf * xf).mean(dim=1) + EPS)
            del xf
            s["dy"] = rnd(*shape, dtype=torch.float32).to(s["yt"])
        if own:
            import cnn_convolution_amd as conv
            if op == "ln_fwd":
                s["out"] = (torch.empty(shape, dtype=s["yt"], device=DEV), torch.empty(stat, device=DEV),
                            torch.empty(stat, device=DEV))
            else:
                s["out"] = (torch.empty_like(s["x"]), torch.empty(C, device=DEV), torch.empty(C, device=DEV))
                n = conv.layer_norm_workspace_size(s["x"], layout=s["layout"], y_dtype=s["yt"], dropout_p=s["p"])
                s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
        return s
    N, V, D, t = case["N"], case["V"], case["D"], TYPES[case["t"]]
    # a partly trained head: logits of spread 2, the target's raised; one row in
    # sixteen carries no target (padding)
    w = rnd(V, D) * (2.0 / math.sqrt(D))
    target = torch.randint(0, V, (N,), generator=gen, device=DEV)
    s["x"] = (rnd(N, D) + 1.5 * w[target]).to(t)
    s["w"] = w.to(t)
    del w
    pad = torch.rand(N, generator=gen, device=DEV) < 1.0 / 16
    pad[0] = False
    s["target"] = torch.where(pad, torch.full_like(target, -1), target)
    # the mean's gradient, times the loss scale of half precision training
    scale = float(N) if case["t"] == "f16" else 1.0
    s["grad"] = (scale / (~pad).sum()).expand(N).float().contiguous()
    if own:
        import cnn_convolution_amd as conv
        s["loss"], s["lse"] = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
        n = conv.linear_cross_entropy_workspace_size(s["x"], s["w"], backward=op == "xent_train")
        s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
        if op == "xent_train":
            s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
    return s


def _run_own(s):
    import cnn_convolution_amd as conv
    op = s["op"]
    if op == "drop":
        conv.dropout_into(s["x"], s["y"], s["p"], s["seed"], s["offset"])
        return [s["y"]]
    if op == "ln_fwd":
        y, mean, rstd = s["out"]
        conv.layer_norm_into(s["x"], s["weight"], s["bias"], y, mean, rstd, EPS, layout=s["layout"],
                             dropout_p=s["p"], seed=s["seed"], offset=s["offset"])
        return [y, mean, rstd]
    if op == "ln_bwd":
        dx, dw, db = s["out"]
        conv.layer_norm_backward_into(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], dx, dw, db, s["ws"],
                                      layout=s["layout"], dropout_p=s["p"], seed=s["seed"], offset=s["offset"])
        return [dx, dw, db]
    conv.linear_cross_entropy_into(s["x"], s["w"], s["target"], s["loss"], s["lse"], s["ws"])
    if op == "xent_loss":
        return [s["loss"], s["lse"]]
    conv.linear_cross_entropy_backward_into(s["grad"], s["x"], s["w"], s["target"], s["lse"], s["dx"], s["dw"],
                                            s["ws"])
    return [s["loss"], s["lse"], s["dx"], s["dw"]]


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "drop":
        x = state["x"]
        return [_drop_plain(x.float(), state["p"], state["seed"], state["offset"]).to(x.dtype)]
    if op == "ln_fwd":
        return _ln_fwd_plain(state)
    if op == "ln_bwd":
        return _ln_bwd_plain(state)
    return _xent_plain(state, op == "xent_train")


def work(case):
    op = case["op"]
    if op == "drop":
        return {"bytes": 2 * case["n"] * SIZE[case["t"]], "flops": case["n"]}
    if op in ("ln_fwd", "ln_bwd"):
        n, rows, C = case["N"] * case["C"] * case["P"], case["N"] * case["P"], case["C"]
        sx, sy = SIZE[case["x"]], SIZE[case["y"]]
        if op == "ln_fwd":
            return {"bytes": n * (sx + sy) + 8 * C + 8 * rows, "flops": 7 * n}
        return {"bytes": n * (2 * sx + sy) + 12 * C + 8 * rows, "flops": 13 * n}
    N, V, D, es = case["N"], case["V"], case["D"], SIZE[case["t"]]
    if op == "xent_loss":
        return {"bytes": (N * D + V * D) * es + 16 * N, "flops": 2 * N * V * D}
    return {"bytes": 2 * (N * D + V * D) * es + 20 * N, "flops": 6 * N * V * D}


# ---- the definition in 64 bits ---------------------------------------------------

def _keep_exact(n, seed, offset, p):
    """Which of elements 0 .. n-1 are kept: the counter blocks in 64-bit words on
    the GPU, multiplied in 16-bit limbs."""
    lo = torch.arange(offset, offset + (n + 7) // 8, device=DEV, dtype=torch.int64)

    def mulhilo(c, m):                                   # 32 x 32 bits -> high, low word
        ml, mh = m & 0xFFFF, m >> 16
        pl, ph = c * ml, c * mh                          # below 2^48
        low = pl + ((ph & 0xFFFF) << 16)
        return (ph >> 16) + (low >> 32), low & _M32

    x = [lo % (1 << 32), lo // (1 << 32), lo * 0, lo * 0]
    key = [seed % (1 << 32), seed // (1 << 32)]
    for r in range(10):
        h0, l0 = mulhilo(x[0], 0xD2511F53)
        h1, l1 = mulhilo(x[2], 0xCD9E8D57)
        ka = (key[0] + r * 0x9E3779B9) % (1 << 32)
        kb = (key[1] + r * 0xBB67AE85) % (1 << 32)
        x = [h1 ^ x[1] ^ ka, l1, h0 ^ x[3] ^ kb, l0]
    keep = torch.empty((lo.numel(), 8), dtype=torch.bool, device=DEV)
    T = int(p * 65536 + 0.5)
    for j in range(8):
        u = x[j // 2] % 65536 if j % 2 == 0 else x[j // 2] // 65536
        keep[:, j] = u >= T
    return keep.reshape(-1)[:n], 65536.0 / (65536 - T)


def _exact_ln(case, s):
    x = s["x"].double()
    c = 1
    p = case["p"]
    shape = x.shape
    w = s["weight"].double().reshape([-1 if i == c else 1 for i in range(x.dim())])
    b = s["bias"].double().reshape(w.shape)
    if case["op"] == "ln_fwd":
        mu = x.sum(c, keepdim=True) / case["C"]
        var = torch.square(x - mu).sum(c, keepdim=True) / case["C"]
        rstd = torch.rsqrt(var + EPS)
        y = (x - mu) * rstd * w + b
        if p > 0:
            keep, sc = _keep_exact(x.numel(), s["seed"], s["offset"], p)
            y = y * sc * keep.reshape(shape)
        return [y, mu.squeeze(c), rstd.squeeze(c)]
    dz = s["dy"].double()
    if p > 0:
        keep, sc = _keep_exact(x.numel(), s["seed"], s["offset"], p)
        dz = dz * sc * keep.reshape(shape)
    rstd = s["rstd"].double().unsqueeze(c)
    xh = (x - s["mean"].double().unsqueeze(c)) * rstd
    g = dz * w
    a = g.sum(c, keepdim=True) / case["C"]
    h = (g * xh).sum(c, keepdim=True) / case["C"]
    others = tuple(i for i in range(x.dim()) if i != c)
    return [(g - a - xh * h) * rstd, torch.sum(dz * xh, others), torch.sum(dz, others)]


def _exact_xent(case, s):
    N, V, D = case["N"], case["V"], case["D"]
    x, w = s["x"].double(), s["w"].double()
    t = s["target"]
    valid = torch.logical_and(t >= 0, t < V)
    loss = torch.zeros(N, dtype=torch.float64, device=DEV)
    lse = torch.zeros_like(loss)
    train = case["op"] == "xent_train"
    dx = torch.zeros_like(x) if train else None
    dw = torch.zeros_like(w) if train else None
    step = max(1, (1 << 27) // V)                        # rows at a time, logits of at most 1 GB
    for i in range(0, N, step):
        keep = torch.nonzero(valid[i:i + step]).squeeze(1) + i
        if keep.numel() == 0:
            continue
        xi, ti = x[keep], t[keep]
        z = torch.matmul(xi, w.t())
        l = torch.logsumexp(z, 1)
        r = torch.arange(keep.numel(), device=DEV)
        lse[keep] = l
        loss[keep] = l - z[r, ti]
        if train:
            q = torch.exp(z - l[:, None])
            q[r, ti] -= 1.0
            q *= s["grad"].double()[keep][:, None]
            dx[keep] = torch.matmul(q, w)
            dw += torch.matmul(q.t(), xi)
    return [loss, lse, dx, dw] if train else [loss, lse]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "drop":
        keep, sc = _keep_exact(case["n"], s["seed"], s["offset"], case["p"])
        return [s["x"].double() * sc * keep]
    if case["op"] in ("ln_fwd", "ln_bwd"):
        return _exact_ln(case, s)
    return _exact_xent(case, s)
