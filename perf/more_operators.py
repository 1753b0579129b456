"""Workloads of the head's block operators: the gated feed-forward block, the
norms before and after a block fused with its gate and residual scale (both with
their gradients), and an AdamW step over many tensors with states in 32 or in 8
bits.

A case is a dict of plain values. ``prepare`` makes the inputs on the GPU,
``run`` takes one pass through an operator (elementary torch operations in fp32,
fp64 for the levels of 8-bit states, or the library's kernels where ``own`` is
true), ``exact`` computes the definition in 64 bits, ``work`` states the bytes
and operations of a pass.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01
BLOCK = 256                                  # elements of an 8-bit state that share a scale


# ---- cases -----------------------------------------------------------------

def _ff(name, op, N, D, F, t, act):
    return {"name": name, "op": op, "N": N, "D": D, "F": F, "t": t, "act": act}


def _rn(name, op, N, C, G, r, b, kind, post=True):
    return {"name": name, "op": op, "N": N, "C": C, "G": G, "r": r, "b": b, "kind": kind, "post": post}


def _adam(name, count, total, p, g, copy, bits):
    return {"name": name, "op": "adamw", "count": count, "total": total, "p": p, "g": g, "copy": copy, "bits": bits}


def listed():
    return [
        # one request's single position through a large block: the weights are read once
        _ff("ff_fwd_one", "ff_fwd", 1, 4096, 8192, "bf16", "silu"),
        # a few positions, rows and features that are no whole vectors
        _ff("ff_fwd_ragged", "ff_fwd", 37, 1001, 2003, "f16", "gelu"),
        # fine-tuning step on 512 pooled channels of 64 images, fp32
        _ff("ff_train_small", "ff_train", 64, 512, 1024, "f32", "relu"),
        # training step over an odd batch, odd hidden size
        _ff("ff_train_odd", "ff_train", 4097, 1032, 3001, "f16", "gelu"),
        # the largest training step
        _ff("ff_train_large", "ff_train", 8192, 4096, 16384, "bf16", "silu"),
        # one position between two blocks: latency only
        _rn("rn_fwd_one", "rn_fwd", 1, 512, 1, "bf16", "bf16", "layer"),
        # the largest batch of wide rows between two blocks, one gate per channel
        _rn("rn_fwd_wide", "rn_fwd", 32768, 4096, 1, "bf16", "bf16", "rms"),
        # gradient with an fp32 residual stream, an odd channel count and a gate per image
        # (69 images of 17 x 17 positions)
        _rn("rn_bwd_odd", "rn_bwd", 69 * 289, 1001, 69, "f32", "f16", "layer"),
        # gradient of the wide rows
        _rn("rn_bwd_wide", "rn_bwd", 32768, 4096, 1, "bf16", "bf16", "rms"),
        # the step of a small head: a norm's vectors and a classifier, fp32
        _adam("adamw_small", 5, 52000, "f32", "f32", "", 32),
        # many tensors of all sizes, half-precision gradients, states in 8 bits
        _adam("adamw_many_8bit", 150, 40000000, "f32", "bf16", "bf16", 8),
        # the largest step: few large tensors, fp32 states and half-precision copies
        _adam("adamw_large", 7, 200000000, "f32", "bf16", "bf16", 32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ff_fwd", "ff_train", "ff_train", "rn_fwd", "rn_bwd", "adamw"])
    t = rng.choice(["f32", "f16", "bf16"])
    if op in ("ff_fwd", "ff_train"):
        D, F = _log(rng, 64, 4096), _log(rng, 64, 16384)
        r = rng.random()
        if r < 0.4:
            D, F = -(-D // 64) * 64, -(-F // 64) * 64
        elif r < 0.7:
            D, F = -(-D // 8) * 8, -(-F // 8) * 8
        most = 8192 if t != "f32" else max(1, min(8192, (1 << 34) // (D * F)))
        return {"op": op, "N": _log(rng, 1, most), "D": D, "F": F, "t": t,
                "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])}
    if op in ("rn_fwd", "rn_bwd"):
        C = _log(rng, 32, 8192)
        if rng.random() < 0.5:
            C = -(-C // 32) * 32
        N = _log(rng, 1, max(1, (1 << 26) // C))
        G = rng.choice([0, 1, 1, _log(rng, 1, 64)])
        N = max(1, N // max(G, 1)) * max(G, 1)
        return {"op": op, "N": N, "C": C, "G": G, "r": t, "b": rng.choice([t, "f16", "bf16"]) if t == "f32" else t,
                "kind": rng.choice(["layer", "rms"]), "post": rng.random() < 0.75}
    g = rng.choice([t, "bf16", "f32"])
    return {"op": "adamw", "count": _log(rng, 1, 200), "total": _log(rng, 1000, 1 << 26), "p": t, "g": g,
            "copy": rng.choice(["", "bf16", "f16"]) if t == "f32" else "", "bits": rng.choice([32, 8])}


def _sizes(case):
    """The tensors' sizes: spread over their logarithm, most of them odd."""
    r = random.Random(7 * case["count"] + case["total"])
    w = [math.exp(r.uniform(0.0, math.log(2000.0))) for _ in range(case["count"])]
    return [max(1, int(case["total"] * v / sum(w))) for v in w]


# ---- the operators in their plain form ---------------------------------------

def _act(kind, a):
    """(act(a), act'(a))"""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-a))
        return a * s, s * (1.0 + a * (1.0 - s))
    if kind == "gelu":
        c = 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5)))
        return a * c, c + a * torch.exp(-0.5 * a * a) * (1.0 / math.sqrt(2.0 * math.pi))
    if kind == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (a + 0.044715 * a * a * a))
        return 0.5 * a * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * a * a)
    if kind == "relu":
        on = (a > 0).to(a.dtype)
        return a * on, on
    s = 1.0 / (1.0 + torch.exp(-a))
    return s, s * (1.0 - s)


def _ff_plain(s, train):
    t = s["x"].dtype
    x, wg, wu, wd = s["x"].float(), s["wg"].float(), s["wu"].float(), s["wd"].float()
    u = x @ wu.t()
    f, df = _act(s["act"], x @ wg.t())
    h = f * u
    y = (h @ wd.t()).to(t)
    if not train:
        return [y]
    dy = s["dy"].float()
    dh = dy @ wd
    da, du = dh * u * df, dh * f
    return [y, (da @ wg + du @ wu).to(t), (da.t() @ x).to(t), (du.t() @ x).to(t), (dy.t() @ h).to(t)]


def _stats(x, kind):
    mean = x.mean(dim=1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    d = x - mean
    return mean, 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + EPS)


def _rows_gate(s):
    """The gate of each row."""
    g = s["gate"]
    return 1.0 if g is None else g.repeat_interleave(s["branch"].shape[0] // g.shape[0], dim=0)


def _rn_fwd_plain(s):
    b, r = s["branch"].float(), s["residual"].float()
    zero = torch.zeros_like(b[:, :1])
    pm, pr = _stats(b, s["kind"]) if s["post"] else (zero, zero)
    p = (b - pm) * pr * s["pw"] + s["pb"] if s["post"] else b
    out = s["rs"] * r + s["bs"] * _rows_gate(s) * p
    m, rstd = _stats(out, s["kind"])
    y = (out - m) * rstd * s["w"] + s["b"]
    return [out.to(s["residual"].dtype), y.to(s["branch"].dtype), torch.cat([pm, pr, m, rstd], dim=1)]


def _norm_back(g, xhat, rstd, kind):
    t = g - xhat * (g * xhat).mean(dim=1, keepdim=True)
    return rstd * (t - g.mean(dim=1, keepdim=True)) if kind == "layer" else rstd * t


def _rn_bwd_plain(s):
    dy, dout, b, out = s["dy"].float(), s["dout"].float(), s["branch"].float(), s["out"].float()
    pm, pr, m, rstd = s["stats"].split(1, dim=1)
    oh = (out - m) * rstd
    t = dout + _norm_back(dy * s["w"], oh, rstd, s["kind"])
    g = s["gate"]
    dp = s["bs"] * _rows_gate(s) * t
    res = [(s["rs"] * t).to(s["out"].dtype)]
    if s["post"]:
        bh = (b - pm) * pr
        p = bh * s["pw"] + s["pb"]
        res += [_norm_back(dp * s["pw"], bh, pr, s["kind"]).to(s["branch"].dtype), (dp * bh).sum(dim=0), dp.sum(dim=0)]
    else:
        p = b
        res += [dp.to(s["branch"].dtype)]
    if g is not None:
        res += [s["bs"] * (t * p).reshape(g.shape[0], -1, g.shape[1]).sum(dim=1)]
    return res + [(dy * oh).sum(dim=0), dy.sum(dim=0)]


_M32 = 0xFFFFFFFF


def _words(block, step, seed):
    """Philox4x32-10 on counter (block, step) with the seed as key: four words."""
    c0, c1 = block & _M32, (block >> 32) & _M32
    c2, c3 = torch.full_like(c0, step & _M32), torch.full_like(c0, step >> 32)
    k0, k1 = seed & _M32, (seed >> 32) & _M32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57          # 64-bit products, wrapped
        c0, c1, c2, c3 = ((b >> 32) & _M32) ^ c1 ^ k0, b & _M32, ((a >> 32) & _M32) ^ c3 ^ k1, a & _M32
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    return torch.stack([c0, c1, c2, c3], dim=1).reshape(-1)


def _levels(x, u, power, top):
    """x in [0, top^power] between the powers of two neighbouring integers: the
    upper one where u (of 65536) says so."""
    c = torch.floor(torch.sqrt(x) if power == 2 else torch.sqrt(torch.sqrt(x)))
    lo = c ** power
    c = torch.where(lo > x, c - 1, c)
    c = torch.where((c + 1) ** power <= x, c + 1, c)
    lo = c ** power
    return (c + ((x - lo) * 65536 > u * ((c + 1) ** power - lo)).double()).clamp(max=top)


def _per_block(x):
    return x.reshape(-1, BLOCK)


def _quantise(m, v, pos, count, step, seed):
    """8-bit codes and scales of m and v (64 bits, one value per element) in the
    padded layout."""
    mp, vp = torch.zeros(count, dtype=torch.float64, device=DEV), torch.zeros(count, dtype=torch.float64, device=DEV)
    mp[pos], vp[pos] = m, v
    w = _words(torch.arange(count // 4, device=DEV), step, seed)
    ms, vs = _per_block(mp.abs().float()).amax(dim=1), _per_block(vp.float()).amax(dim=1)
    mx = _per_block(mp.abs()) * torch.where(ms > 0, 16129.0 / ms.double(), 0.0)[:, None]
    vx = _per_block(vp) * torch.where(vs > 0, 255.0 ** 4 / vs.double(), 0.0)[:, None]
    mk = _levels(mx, _per_block(w & 0xFFFF).double(), 2, 127.0) * _per_block(mp).sign()
    vk = torch.where(_per_block(vp) > 0, _levels(vx, _per_block(w >> 16).double(), 4, 255.0).clamp(min=1.0), 0.0)
    return mk.reshape(-1).to(torch.int8), vk.reshape(-1).to(torch.uint8), ms, vs


def _values(mk, vk, ms, vs):
    """What the codes stand for, in 64 bits."""
    k, q = _per_block(mk).double(), _per_block(vk).double()
    return ((k * k.abs() * (ms.double() / 16129.0)[:, None]).reshape(-1),
            (q ** 4 * (vs.double() / 255.0 ** 4)[:, None]).reshape(-1))


def _adam_plain(s):
    p, g, pos = s["flat"].float(), s["grad"].float() * s["gscale"], s["pos"]
    if s["bits"] == 8:
        m, v = _values(s["mk"], s["vk"], s["ms"], s["vs"])
        gd = g.double()
        m, v = BETA1 * m[pos] + (1 - BETA1) * gd, BETA2 * v[pos] + (1 - BETA2) * gd * gd
        s["mk"], s["vk"], s["ms"], s["vs"] = _quantise(m, v, pos, s["mk"].numel(), s["step"], s["seed"])
        m, v = m.float(), v.float()
    else:
        m, v = BETA1 * s["m"][pos] + (1 - BETA1) * g, BETA2 * s["v"][pos] + (1 - BETA2) * g * g
        s["m"][pos], s["v"][pos] = m, v
    den = torch.sqrt(v / (1 - BETA2 ** s["step"])) + ADAM_EPS
    p = p * (1 - LR * DECAY) - LR * (m / (1 - BETA1 ** s["step"])) / den
    s["flat"].copy_(p)
    res = [s["flat"]]
    if s["copy"] is not None:
        s["copy"].copy_(p)
        res.append(s["copy"])
    if s["bits"] == 8:
        m, v = _values(s["mk"], s["vk"], s["ms"], s["vs"])
        return res + [m.float(), v.float()]
    return res + [s["m"], s["v"]]


# ---- prepare and run -----------------------------------------------------------

def _prepare_ff(case, s, rnd):
    N, D, F, t = case["N"], case["D"], case["F"], TYPES[case["t"]]
    # normalised inputs, weights that keep the spread
    s["x"] = rnd(N, D).to(t)
    s["wg"] = (rnd(F, D) * (1.2 / math.sqrt(D))).to(t)
    s["wu"] = (rnd(F, D) * (1.0 / math.sqrt(D))).to(t)
    s["wd"] = (rnd(D, F) * (1.0 / math.sqrt(F))).to(t)
    s["act"] = case["act"]
    train = case["op"] == "ff_train"
    if train:
        # a mean loss's gradient; fp16 with the loss scaled
        s["dy"] = (rnd(N, D) * (0.5 if case["t"] == "f16" else 1.0 / 256)).to(t)
    if own:
        import cnn_convolution_amd as conv
        s["y"] = torch.empty_like(s["x"])
        n = conv.feed_forward_workspace_size(s["x"], s["wg"], s["wu"], s["wd"], saved=train, dy=s.get("dy"))
        s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
        s["saved"] = None
        if train:
            n = conv.feed_forward_saved_size(s["x"], s["wg"])
            s["saved"] = torch.empty(n, dtype=torch.uint8, device=DEV)
            s["grads"] = [torch.empty_like(s[k]) for k in ("x", "wg", "wu", "wd")]


def _prepare_rn(case, s, rnd):
    N, C, G = case["N"], case["C"], case["G"]
    s.update(kind=case["kind"], post=case["post"], rs=0.9, bs=1.1)
    # channels with their own level and spread, a residual stream larger than the branch
    spread, level = 1.0 + 0.5 * rnd(1, C).abs(), 0.5 * rnd(1, C)
    s["branch"] = (rnd(N, C) * spread + level).to(TYPES[case["b"]])
    s["residual"] = (2.0 * rnd(N, C) + level).to(TYPES[case["r"]])
    s["gate"] = 0.5 + 0.3 * rnd(G, C) if G else None
    for k in ("w", "pw"):
        s[k] = 1.0 + 0.2 * rnd(C)
    for k in ("b", "pb"):
        s[k] = 0.2 * rnd(C)
    s["options"] = {"kind": s["kind"], "post": s["post"], "residual_scale": s["rs"], "branch_scale": s["bs"]}
    if not s["post"]:
        s["pw"] = s["pb"] = None
    if case["op"] == "rn_bwd":
        s["out"], _, s["stats"] = _rn_fwd_plain(s)
        s["dy"] = rnd(N, C).to(TYPES[case["b"]])
        s["dout"] = rnd(N, C).to(TYPES[case["r"]])
    if own:
        import cnn_convolution_amd as conv
        if case["op"] == "rn_fwd":
            s["res"] = [torch.empty_like(s["residual"]), torch.empty_like(s["branch"]), torch.empty(N, 4, device=DEV)]
        else:
            vec = [torch.empty(C, device=DEV) if k else None for k in (s["post"], s["post"], True, True)]
            s["res"] = [torch.empty_like(s["out"]), torch.empty_like(s["branch"]), *vec,
                        torch.empty_like(s["gate"]) if G else None]
            n = conv.residual_norm_workspace_size(s["branch"], gate=s["gate"], post=s["post"])
            s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)


def _prepare_adam(case, s, rnd, seed):
    sizes = _sizes(case)
    n = sum(sizes)
    first, at = [], 0
    for k in sizes:                                       # the states' layout: whole blocks
        first.append(at)
        at += -(-k // BLOCK) * BLOCK
    start = torch.tensor(first, device=DEV) - torch.tensor([sum(sizes[:i]) for i in range(len(sizes))], device=DEV)
    s["pos"] = torch.arange(n, device=DEV) + start.repeat_interleave(torch.tensor(sizes, device=DEV))
    # every tensor's gradients at their own scale, some elements still without any
    scale = torch.exp(2.0 * rnd(len(sizes))).repeat_interleave(torch.tensor(sizes, device=DEV)) * 1e-2
    s.update(bits=case["bits"], step=1000 + seed % 97, seed=(0x9E37_00000000 + 7919 * seed) & (2 ** 62 - 1), gscale=0.5)
    s["flat"] = (0.05 * rnd(n)).to(TYPES[case["p"]])
    s["grad"] = (2.0 * scale * rnd(n)).to(TYPES[case["g"]])
    s["copy"] = torch.empty(n, dtype=TYPES[case["copy"]], device=DEV) if case["copy"] else None
    seen = (rnd(n) > -1.5).float()
    m, v = 0.25 * scale * rnd(n) * seen, scale * scale * (0.2 + rnd(n).square()) * seen
    if case["bits"] == 8:
        s["mk"], s["vk"], s["ms"], s["vs"] = _quantise(m.double(), v.double(), s["pos"], at, 999, seed)
    else:
        s["m"], s["v"] = torch.zeros(at, device=DEV), torch.zeros(at, device=DEV)
        s["m"][s["pos"]], s["v"][s["pos"]] = m, v
    s["params"], s["grads"] = list(s["flat"].split(sizes)), list(s["grad"].split(sizes))
    s["copies"] = None if s["copy"] is None else list(s["copy"].split(sizes))
    if own:
        import cnn_convolution_amd as conv
        st = s["state"] = conv.adamw_state(s["params"], bits=case["bits"])
        if case["bits"] == 8:
            st.exp_avg.copy_(s["mk"])
            st.exp_avg_sq.copy_(s["vk"])
            st.exp_avg_scale.copy_(s["ms"])
            st.exp_avg_sq_scale.copy_(s["vs"])
            s["values"] = [torch.empty(at, device=DEV), torch.empty(at, device=DEV)]
        else:
            st.exp_avg.copy_(s["m"])
            st.exp_avg_sq.copy_(s["v"])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s = {"op": case["op"]}
    if case["op"] in ("ff_fwd", "ff_train"):
        _prepare_ff(case, s, rnd)
    elif case["op"] in ("rn_fwd", "rn_bwd"):
        _prepare_rn(case, s, rnd)
    else:
        _prepare_adam(case, s, rnd, seed)
    return s


def _run_own(s):
    import cnn_convolution_amd as conv
    op = s["op"]
    if op in ("ff_fwd", "ff_train"):
        w = (s["wg"], s["wu"], s["wd"])
        conv.feed_forward_into(s["x"], *w, s["y"], s["saved"], s["ws"], activation=s["act"])
        if op == "ff_fwd":
            return [s["y"]]
        conv.feed_forward_backward_into(s["dy"], s["x"], *w, s["saved"], *s["grads"], s["ws"], activation=s["act"])
        return [s["y"], *s["grads"]]
    if op == "rn_fwd":
        conv.residual_norm_into(s["branch"], s["residual"], *s["res"], EPS, gate=s["gate"], post_weight=s["pw"],
                                post_bias=s["pb"], weight=s["w"], bias=s["b"], **s["options"])
        return s["res"]
    if op == "rn_bwd":
        dr, db, dpw, dpb, dw, dbias, dgate = s["res"]
        conv.residual_norm_backward_into(s["dy"], s["dout"], s["branch"], s["out"], s["stats"], dr, db, s["ws"],
                                         gate=s["gate"], post_weight=s["pw"], post_bias=s["pb"], weight=s["w"],
                                         dgate=dgate, dpost_weight=dpw, dpost_bias=dpb, dweight=dw, dbias=dbias,
                                         **s["options"])
        return [dr, db] + ([dpw, dpb] if s["post"] else []) + ([] if dgate is None else [dgate]) + [dw, dbias]
    conv.adamw(s["params"], s["grads"], s["state"], s["step"], LR, BETA1, BETA2, ADAM_EPS, DECAY,
               grad_scale=s["gscale"], copies=s["copies"], seed=s["seed"])
    res = [s["flat"]] + ([] if s["copy"] is None else [s["copy"]])
    if s["bits"] == 8:
        conv.adamw_state_values_into(s["state"], *s["values"])
        return res + s["values"]
    return res + [s["state"].exp_avg, s["state"].exp_avg_sq]


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op in ("ff_fwd", "ff_train"):
        return _ff_plain(state, op == "ff_train")
    if op == "rn_fwd":
        return _rn_fwd_plain(state)
    if op == "rn_bwd":
        return _rn_bwd_plain(state)
    return _adam_plain(state)


def work(case):
    op = case["op"]
    if op in ("ff_fwd", "ff_train"):
        N, D, F, es = case["N"], case["D"], case["F"], SIZE[case["t"]]
        if op == "ff_fwd":
            return {"bytes": (2 * N * D + 3 * D * F) * es, "flops": 6 * N * D * F}
        return {"bytes": (4 * N * D + 6 * D * F) * es, "flops": 18 * N * D * F}
    if op in ("rn_fwd", "rn_bwd"):
        n, r, b = case["N"] * case["C"], SIZE[case["r"]], SIZE[case["b"]]
        vec = 4 * case["C"] * (case["G"] + (4 if case["post"] else 2))
        if op == "rn_fwd":
            return {"bytes": 2 * n * (r + b) + vec + 16 * case["N"], "flops": 16 * n}
        return {"bytes": 3 * n * (r + b) + 2 * vec + 16 * case["N"], "flops": 36 * n}
    n = sum(_sizes(case))
    per = 2 * SIZE[case["p"]] + SIZE[case["g"]] + (SIZE[case["copy"]] if case["copy"] else 0)
    # 8 bits: codes in and out, and what they stand for written once
    return {"bytes": n * (per + (16 if case["bits"] == 32 else 12)), "flops": 16 * n}


# ---- the definition in 64 bits ---------------------------------------------------

def _exact_act(kind, a):
    if kind in ("silu", "sigmoid"):
        s = torch.sigmoid(a)
        return (a * s, s + a * s * (1 - s)) if kind == "silu" else (s, s * (1 - s))
    if kind == "gelu":
        c = torch.special.ndtr(a)
        return a * c, c + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":                              # a * logistic(2 z)
        z = math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
        s = torch.sigmoid(2 * z)
        return a * s, s + a * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * a ** 2)
    return torch.clamp(a, min=0), torch.where(a > 0, 1.0, 0.0)


def _exact_ff(case, s):
    x, wg, wu, wd = (s[k].double() for k in ("x", "wg", "wu", "wd"))
    gate, up = torch.matmul(x, wg.T), torch.matmul(x, wu.T)
    val, slope = _exact_act(case["act"], gate)
    hidden = val * up
    res = [torch.matmul(hidden, wd.T)]
    if case["op"] == "ff_train":
        dy = s["dy"].double()
        dwd = torch.matmul(dy.T, hidden)
        back = torch.matmul(dy, wd)
        dgate, dup = back * up * slope, back * val
        res += [torch.matmul(dgate, wg) + torch.matmul(dup, wu), torch.matmul(dgate.T, x), torch.matmul(dup.T, x), dwd]
    return res


def _exact_rn(case, s):
    N, C, layer = case["N"], case["C"], case["kind"] == "layer"

    def moments(z):
        mu = z.sum(1) / C if layer else z.new_zeros(N)
        var = torch.square(z - mu[:, None]).sum(1) / C
        return mu, torch.rsqrt(var + EPS)

    def through(dz, zhat, r):                            # the gradient through a norm
        res = dz - zhat * ((dz * zhat).sum(1) / C)[:, None]
        if layer:
            res = res - (dz.sum(1) / C)[:, None]
        return res * r[:, None]

    b = s["branch"].double()
    G = case["G"]
    gate = torch.ones(1, 1, C, dtype=torch.float64, device=DEV) if G == 0 else s["gate"].double()[:, None, :]
    w = s["w"].double()
    pw, pb = (s["pw"].double(), s["pb"].double()) if case["post"] else (None, None)

    def gated(z):                                        # rows times their group's gate
        return (z.reshape(max(G, 1), -1, C) * gate).reshape(N, C)

    if case["op"] == "rn_fwd":
        if case["post"]:
            m1, r1 = moments(b)
            p = (b - m1[:, None]) * r1[:, None] * pw + pb
        else:
            m1 = r1 = b.new_zeros(N)
            p = b
        out = s["residual"].double() * s["rs"] + gated(p) * s["bs"]
        m2, r2 = moments(out)
        return [out, (out - m2[:, None]) * r2[:, None] * w + s["b"].double(), torch.stack([m1, r1, m2, r2], dim=1)]
    m1, r1, m2, r2 = s["stats"].double().unbind(1)
    dy = s["dy"].double()
    oh = (s["out"].double() - m2[:, None]) * r2[:, None]
    t = s["dout"].double() + through(dy * w, oh, r2)
    dp = gated(t) * s["bs"]
    res = [t * s["rs"]]
    p = b
    if case["post"]:
        bh = (b - m1[:, None]) * r1[:, None]
        p = bh * pw + pb
        res += [through(dp * pw, bh, r1), torch.sum(dp * bh, 0), torch.sum(dp, 0)]
    else:
        res += [dp]
    if G:
        res += [torch.sum((t * p).reshape(G, -1, C), 1) * s["bs"]]
    return res + [torch.sum(dy * oh, 0), torch.sum(dy, 0)]


def _exact_halves(count, step, seed):
    """The 16-bit numbers of elements 0 .. count - 1 for m and for v: the words
    multiplied in 16-bit limbs."""
    q = torch.arange(count // 4, device=DEV, dtype=torch.int64)

    def mulhilo(c, m):                                   # 32 x 32 bits -> high, low word
        ml, mh = m & 0xFFFF, m >> 16
        pl, ph = c * ml, c * mh                          # below 2^48
        low = pl + ((ph & 0xFFFF) << 16)
        return (ph >> 16) + (low >> 32), low & _M32

    x = [q % (1 << 32), q // (1 << 32), q * 0 + step % (1 << 32), q * 0 + step // (1 << 32)]
    key = [seed % (1 << 32), seed // (1 << 32)]
    for r in range(10):
        h0, l0 = mulhilo(x[0], 0xD2511F53)
        h1, l1 = mulhilo(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ ((key[0] + r * 0x9E3779B9) % (1 << 32)), l1,
             h0 ^ x[3] ^ ((key[1] + r * 0xBB67AE85) % (1 << 32)), l0]
    word = torch.empty(count, dtype=torch.int64, device=DEV)
    for j in range(4):
        word[j::4] = x[j]
    return word % 65536, word // 65536


def _exact_codes(x, u, power, top):
    """Codes of x (in units of the scale): the number of levels at or below it, one
    more with the probability of where it lies in its interval."""
    level = (torch.arange(top + 2, dtype=torch.float64, device=DEV) / top) ** power
    c = torch.searchsorted(level, x.contiguous(), right=True) - 1
    part = (x - level[c]) / (level[(c + 1).clamp(max=top + 1)] - level[c])
    return torch.clamp(c + (part * 65536 > u), max=top)


def _exact_adam(case, s):
    pos, step = s["pos"], s["step"]
    p, g = s["flat"].double(), s["grad"].double() * s["gscale"]
    if case["bits"] == 8:
        k, q = s["mk"].double(), s["vk"].double()
        m0 = torch.sign(k) * torch.square(k / 127) * s["ms"].double().repeat_interleave(BLOCK)
        v0 = torch.square(torch.square(q / 255)) * s["vs"].double().repeat_interleave(BLOCK)
    else:
        m0, v0 = s["m"].double(), s["v"].double()
    m, v = m0[pos] + (1 - BETA1) * (g - m0[pos]), v0[pos] + (1 - BETA2) * (g * g - v0[pos])
    new = p - LR * DECAY * p
    new = new - LR * m / (1 - BETA1 ** step) / (torch.sqrt(v) / math.sqrt(1 - BETA2 ** step) + ADAM_EPS)
    ms, vs = torch.zeros_like(m0), torch.zeros_like(v0)
    ms[pos], vs[pos] = m, v
    res = [new] + ([new] if case["copy"] else [])
    if case["bits"] == 32:
        return res + [ms, vs]
    um, uv = _exact_halves(ms.numel(), step, s["seed"])
    top = ms.abs().reshape(-1, BLOCK).amax(1).float().double().repeat_interleave(BLOCK)
    unit = torch.where(top > 0, top, 1.0)
    mq = torch.sign(ms) * torch.square(_exact_codes(ms.abs() / unit, um, 2, 127).double() / 127) * top
    top = vs.reshape(-1, BLOCK).amax(1).float().double().repeat_interleave(BLOCK)
    unit = torch.where(top > 0, top, 1.0)
    c = _exact_codes(vs / unit, uv, 4, 255)
    c = torch.where(vs > 0, c.clamp(min=1), 0)
    return res + [mq, torch.square(torch.square(c.double() / 255)) * top]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("ff_fwd", "ff_train"):
        return _exact_ff(case, s)
    if case["op"] in ("rn_fwd", "rn_bwd"):
        return _exact_rn(case, s)
    return _exact_adam(case, s)
