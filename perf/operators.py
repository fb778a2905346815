"""Timed cases of the operators around the MoE-LoRA expert layer in a fine-tuning step.

Three operators, each with inputs as a training program has them in hand:

* ``norm``    the norm after a block, the gated and scaled residual sum, and the
              norm before the next block (``lib.moe_block_norm_fwd`` / ``_bwd``)
                p = y rstd(y) (w_post + off) or y,   r = x + s a(gate) p,
                n = r rstd(r) (w_pre + off),         rstd(z) = 1/sqrt(mean z^2 + eps)
* ``router``  the router's load-balancing and z losses, and the gradient of its
              logits through the top-k weights and both losses
              (``lib.moe_router_loss_fwd`` / ``lib.moe_router_bwd``)
                aux = E sum_e f_e mean_t P_te,  f_e = counts_e / (T k),  z = mean_t lse_t^2
* ``adamw``   one AdamW step over many tensors, moments in 32 bits or in 8
              (``lib.moe_adamw_step``).  8 bits: m and sqrt(v) as float8_e4m3 with
              a power-of-two scale (E8M0) for each block of 256 values, rounded
              with the dither u = frac(step phi + i sqrt2) of value i.

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits, rounded once at the end; with ``own`` true it calls the framework.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BETAS = (0.9, 0.999)
LR = 1e-4
ADAM_EPS = 1e-8
AUX, ZED = 0.01, 0.001
BLOCK = 256                    # values that share a scale in 8-bit states
DITHER_T, DITHER_I = 2654435769, 1779033703   # fractional parts of phi and sqrt 2, times 2^32
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


# ------------------------------------------------------------------- cases

def _norm(name, dir, T, d, x="bf16", y="bf16", gate="none", sigmoid=False, post=True, pre=True,
          learn=True):
    c = {"op": "norm", "dir": dir, "T": T, "d": d, "x": x, "y": y, "gate": gate,
         "sigmoid": sigmoid, "post": post, "pre": pre, "learn": learn}
    return dict(c, name=name) if name else c


def _router(name, dir, T, E, k, zipf=0.0, blocked=0):
    c = {"op": "router", "dir": dir, "T": T, "E": E, "k": k, "zipf": zipf, "blocked": blocked}
    return dict(c, name=name) if name else c


def _adamw(name, n, numel, param="bf16", grad="fp32", master=True, bits=32, clip=0.0, lora=""):
    c = {"op": "adamw", "n": n, "numel": numel, "lora": lora, "param": param, "grad": grad,
         "master": master, "bits": bits, "clip": clip}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token generated while a fine-tuned model is sampled: latency only
        _norm("norm fwd 1x2048", "fwd", 1, 2048),
        # a forward at the Qwen3-30B-A3B-shaped layer's size
        _norm("norm fwd 4096x2048", "fwd", 4096, 2048),
        # its backward, with a learned gate for each channel and both norm weights trained
        _norm("norm bwd 4096x2048 channel", "bwd", 4096, 2048, gate="channel"),
        # a ragged packed batch and a width no vector divides: a sigmoid gate for each token
        _norm("norm both 1037x1001 token", "both", 1037, 1001, gate="token", sigmoid=True),
        # a large batch at the gpt-oss-shaped width with the residual stream in 32 bits,
        # a gate for each element and frozen norm weights
        _norm("norm both 32768x2880 fp32", "both", 32768, 2880, x="fp32", gate="element",
              learn=False),
        # the losses of one step's router
        _router("router fwd 4096x128", "fwd", 4096, 128, 8),
        # the skewed router with experts that are switched off, and a ragged count of both
        _router("router both 1000x60", "both", 1000, 60, 4, zipf=3.0, blocked=4),
        # a whole batch of a million tokens
        _router("router both 1Mx128", "both", 1 << 20, 128, 8),
        # norm weights, gates and biases of a small model: many short fp32 tensors
        _adamw("adamw 24 short fp32", 24, 2048, param="fp32", master=False),
        # ragged bf16 tensors with bf16 gradients and no master copy
        _adamw("adamw 40 ragged bf16 8bit", 40, 100003, grad="bf16", master=False, bits=8),
        # the LoRA weights of one Qwen3-30B-A3B-shaped layer, clipped by the global norm
        _adamw("adamw lora 32bit clip", 4, 0, lora="128,2048,768,64", clip=1.0),
        # the same with moments in 8 bits
        _adamw("adamw lora 8bit", 4, 0, lora="128,2048,768,64", bits=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case, no costlier than the largest listed one."""
    op = rng.choice(["norm", "norm", "router", "adamw"])
    if op == "norm":
        d = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024), 2048, 2880])
        T = max(1, min(_log(rng, 1, 65536), 32768 * 2880 // d))
        x, y = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")])
        if (x, y) == ("fp32", "fp32"):
            T = max(1, T // 2)
        post, pre = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        gate = rng.choice(["none", "token", "channel", "element"])
        return _norm("", rng.choice(["fwd", "bwd", "both"]), T, d, x, y, gate,
                     gate != "none" and rng.random() < 0.5, post, pre, rng.random() < 0.7)
    if op == "router":
        E = rng.choice([8, 32, 64, 128, _log(rng, 5, 512)])
        T = max(1, min(_log(rng, 1, 1 << 20), (1 << 27) // E))
        blocked = rng.choice([0, 0, E // 16])
        k = min(rng.choice([1, 2, 4, 8]), E - blocked)
        return _router("", rng.choice(["fwd", "both"]), T, E, k, rng.choice([0.0, 3.0]), blocked)
    total = _log(rng, 1000, 40_000_000)
    n = min(_log(rng, 1, 200), total)
    param = rng.choice(["bf16", "bf16", "fp32"])
    return _adamw("", n, max(1, total // n), param, rng.choice(["fp32", "bf16"]),
                  param == "bf16" and rng.random() < 0.6, rng.choice([32, 8]),
                  rng.choice([0.0, 1.0]))


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(DEV)
    g.manual_seed(int(seed) * 7919 + 11)
    return {"norm": _prepare_norm, "router": _prepare_router,
            "adamw": _prepare_adamw}[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _prepare_norm(c, g):
    T, d, xt, yt = c["T"], c["d"], TYPES[c["x"]], TYPES[c["y"]]
    s = {"case": c, "op": "norm", "scale": 0.75, "off": 0.0}
    # a residual stream has channels far larger than the rest, a block's output has less spread
    s["x"] = (_randn(g, T, d) * torch.exp(0.8 * _randn(g, d))).to(xt)
    s["y"] = (0.5 * _randn(g, T, d)).to(yt)
    s["w_post"] = 1.0 + 0.2 * _randn(g, d) if c["post"] else None
    s["w_pre"] = 1.0 + 0.2 * _randn(g, d) if c["pre"] else None
    s["gate"] = {"none": lambda: None, "token": lambda: _randn(g, T), "channel": lambda: _randn(g, d),
                 "element": lambda: _randn(g, T, d).to(yt)}[c["gate"]]()
    s["dr"] = _randn(g, T, d).to(xt)
    s["dn"] = _randn(g, T, d).to(yt) if c["pre"] else None
    f32 = dict(dtype=torch.float32, device=DEV)
    # what the forward saved (it writes them again where the pass has one)
    r, _, rs_y, rs_r = _norm_fwd(s)
    s["r"] = r.to(xt)
    s["rstd_y"], s["rstd_r"] = rs_y, rs_r
    s["n"] = torch.empty(T, d, dtype=yt, device=DEV) if c["pre"] else None
    s["dx"], s["dy"] = torch.empty(T, d, dtype=xt, device=DEV), torch.empty(T, d, dtype=yt,
                                                                            device=DEV)
    s["dgate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
    s["dw_post"] = torch.empty(d, **f32) if c["post"] and c["learn"] else None
    s["dw_pre"] = torch.empty(d, **f32) if c["pre"] and c["learn"] else None
    s["ws"] = None
    return s


def _prepare_router(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    logits = _randn(g, T, E)
    rank = torch.randperm(E, generator=g, device=DEV) + 1
    logits += c["zipf"] * rank.float().pow(-1.2)
    if c["blocked"]:
        logits[:, rank > E - c["blocked"]] = -math.inf
    val, ids = torch.topk(logits, k, dim=1)
    return {"case": c, "op": "router", "logits": logits, "ids": ids.to(torch.int32),
            "w": torch.softmax(val, 1), "dw": 0.1 * _randn(g, T, k),
            "counts": torch.bincount(ids.reshape(-1), minlength=E).to(torch.int32),
            "losses": torch.empty(2, device=DEV), "lse": torch.empty(T, device=DEV),
            "pmean": torch.empty(E, device=DEV), "dlogits": torch.empty_like(logits), "ws": None}


def _sizes(c):
    if c["lora"]:
        E, d, f, r = (int(v) for v in c["lora"].split(","))
        return [E * r * d, E * 2 * f * r, E * r * f, E * d * r]
    # lengths from a quarter to one and three quarters of the mean, even and odd ones
    return [max(1, int(c["numel"] * (0.25 + 1.5 * math.modf(i * 0.6180339887 + 0.5)[0])))
            for i in range(c["n"])]


def _prepare_adamw(c, g):
    sizes = _sizes(c)
    padded = [-(-n // BLOCK) * BLOCK for n in sizes]
    start = [sum(padded[:i]) for i in range(len(sizes))]
    total = sum(padded)
    inside = torch.zeros(total, dtype=torch.bool, device=DEV)
    [inside[o:o + n].fill_(True) for o, n in zip(start, sizes)]
    # gradients whose size varies over blocks of weights, as rows of a matrix do
    size = 1e-3 * torch.exp(1.5 * _randn(g, total // BLOCK)).repeat_interleave(BLOCK) * inside
    grad = (_randn(g, total) * size).to(TYPES[c["grad"]])
    m = 0.3 * _randn(g, total) * size
    v = (size * torch.exp(0.5 * _randn(g, total))).square()
    p = 0.02 * _randn(g, total) * inside
    s = {"case": c, "op": "adamw", "sizes": sizes, "padded": padded, "start": start, "step": 100,
         "grad": grad, "param": p.to(TYPES[c["param"]]), "master": p if c["master"] else None,
         "decay": [0.01 if i % 2 == 0 else 0.0 for i in range(len(sizes))],
         "norm": torch.zeros(1, device=DEV) if c["clip"] else None, "scales": None, "table": None}
    # 1 - lr decay for each block, and each value's index in its tensor
    s["kept"] = torch.cat([torch.full((n // BLOCK, 1), 1 - LR * wd, device=DEV)
                           for n, wd in zip(padded, s["decay"])])
    if c["bits"] == 8:
        local = s["local"] = torch.cat([torch.arange(n, device=DEV) for n in padded])
        m8, bm = _to8(m, local, 99, False)
        r8, br = _to8(v.sqrt(), local, 99, True)
        s.update(m=m8, v=r8, scales=torch.stack([bm, br], 1).contiguous())
    else:
        s.update(m=m, v=v)
    return s


# ------------------------------------------------------------- plain forms

def run(state):
    if own:
        return {"norm": _own_norm, "router": _own_router, "adamw": _own_adamw}[state["op"]](state)
    return {"norm": _plain_norm, "router": _plain_router,
            "adamw": _plain_adamw}[state["op"]](state)


def _activated(s):
    """The gate's factor a, its derivative, and the shape that broadcasts over [T, d]."""
    if s["gate"] is None:
        return 1.0, 0.0
    gate = s["gate"].float()
    gate = gate[:, None] if s["case"]["gate"] == "token" else gate
    if s["case"]["sigmoid"]:
        a = 1.0 / (1.0 + torch.exp(-gate))
        return a, a * (1.0 - a)
    return gate, 1.0


def _norm_fwd(s):
    x, p, rs_y, rs_r, n = s["x"].float(), s["y"].float(), None, None, None
    if s["w_post"] is not None:
        rs_y = torch.rsqrt(p.square().mean(1) + EPS)
        p = p * rs_y[:, None] * (s["w_post"] + s["off"])
    r = x + s["scale"] * _activated(s)[0] * p
    if s["w_pre"] is not None:
        rs_r = torch.rsqrt(r.square().mean(1) + EPS)
        n = r * rs_r[:, None] * (s["w_pre"] + s["off"])
    return r, n, rs_y, rs_r


def _norm_bwd(s, r, rs_y, rs_r):
    c, out = s["case"], {}
    t = s["dr"].float()
    if s["w_pre"] is not None:
        hat, dn = r.float() * rs_r[:, None], s["dn"].float()
        if c["learn"]:
            out["dw_pre"] = (dn * hat).sum(0)
        dn = dn * (s["w_pre"] + s["off"])
        t = t + rs_r[:, None] * (dn - hat * (dn * hat).mean(1, keepdim=True))
    out["dx"] = t.to(s["dr"].dtype)
    a, da = _activated(s)
    dp, p = s["scale"] * a * t, s["y"].float()
    if s["w_post"] is not None:
        hat = p * rs_y[:, None]
        p = hat * (s["w_post"] + s["off"])
        if c["learn"]:
            out["dw_post"] = (dp * hat).sum(0)
        dp = dp * (s["w_post"] + s["off"])
        dp = rs_y[:, None] * (dp - hat * (dp * hat).mean(1, keepdim=True))
    out["dy"] = dp.to(s["y"].dtype)
    if s["gate"] is not None:
        dg = s["scale"] * da * t * p
        dg = {"token": lambda: dg.sum(1), "channel": lambda: dg.sum(0),
              "element": lambda: dg}[c["gate"]]()
        out["dgate"] = dg.to(s["gate"].dtype)
    return out


def _plain_norm(s):
    c, out = s["case"], {}
    r, rs_y, rs_r = s["r"], s["rstd_y"], s["rstd_r"]
    if c["dir"] != "bwd":
        r, n, rs_y, rs_r = _norm_fwd(s)
        r = r.to(s["x"].dtype)
        out = {"r": r, "n": None if n is None else n.to(s["y"].dtype), "rstd_y": rs_y,
               "rstd_r": rs_r}
    if c["dir"] != "fwd":
        out.update(_norm_bwd(s, r, rs_y, rs_r))
    return out


def _plain_router(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"]
    top = l.amax(1, keepdim=True)
    ex = torch.exp(l - top)
    sum_ = ex.sum(1, keepdim=True)
    P = ex / sum_
    lse = (top + torch.log(sum_))[:, 0]
    f = s["counts"].float() / (T * k)
    pmean = P.mean(0)
    out = {"losses": torch.stack([E * (f * pmean).sum(), lse.square().mean()]), "lse": lse,
           "pmean": pmean}
    if c["dir"] == "fwd":
        return out
    d = P * ((AUX * E / T) * (f - (P * f).sum(1, keepdim=True)) + (2 * ZED / T) * lse[:, None])
    w, dw = s["w"], s["dw"]
    d.scatter_add_(1, s["ids"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    out["dlogits"] = d
    return out


def _bits(x):
    return x.view(torch.int32).long()


def _float(bits):
    return bits.to(torch.int32).view(torch.float32)


def _dither(local, step):
    return (local * DITHER_I + step * DITHER_T) & 0xFFFFFFFF


def _to8(x, local, step, root):
    """float8_e4m3 values of x / scale and the E8M0 bytes of the scales, x a whole number of
    blocks.  The largest of a block lands in [128, 256); a value x between two representable
    ones goes up where the dither passes its distance to the upper one."""
    mag = _bits(x.abs()).view(-1, BLOCK)
    byte = ((mag.amax(1) >> 23) - 7).clamp(min=8)
    b = byte[:, None]
    u = _dither(local, step).view(-1, BLOCK)
    u = (0xFFFFFFFF - u if root else u) >> 12
    low = _float((b - 6) << 23)                   # smallest normal value: 2^-6 scale
    a = _float(mag)
    below = a < low
    code = ((_bits(torch.where(below, a + low, a)) + u) >> 20) - ((b - 7) << 3)
    code = code - 8 * below.long()
    if root:                                      # sqrt(v) > 0 stays above zero
        code = torch.where((mag > 0) & (code < 1), torch.ones_like(code), code)
    code = code.reshape(-1) + 128 * (x < 0).long()
    return code.to(torch.uint8).view(torch.float8_e4m3fn), byte.to(torch.uint8)


def _scale(byte):
    return _float(byte.long() << 23).repeat_interleave(BLOCK)


def _plain_adamw(s):
    """All tensors at once: they lie in one buffer, each from a whole block on, zeros between."""
    c, b1, b2 = s["case"], BETAS[0], BETAS[1]
    s["step"] += 1
    t = s["step"]
    g = s["grad"].float()
    if c["clip"]:
        norm = g.double().square().sum().sqrt().float()
        s["norm"].copy_(norm)
        g = g * torch.clamp(c["clip"] / (norm + 1e-6), max=1.0)
    keep1, take1, keep2, take2, correct, eps, lr = torch.tensor(
        [b1, 1 - b1, b2, 1 - b2, 1 / math.sqrt(1 - b2 ** t), ADAM_EPS, LR / (1 - b1 ** t)],
        dtype=torch.float32).tolist()
    m, v = s["m"], s["v"]
    if c["bits"] == 8:
        m = m.float() * _scale(s["scales"][:, 0])
        v = (v.float() * _scale(s["scales"][:, 1])).square()
    m = keep1 * m + take1 * g
    v = keep2 * v + (take2 * g) * g
    root = v.sqrt()
    p = (s["param"] if s["master"] is None else s["master"]).float()
    p = (p.view(-1, BLOCK) * s["kept"]).view(-1) - lr * (m / (root * correct + eps))
    s["param"].copy_(p)
    if s["master"] is not None:
        s["master"].copy_(p)
    if c["bits"] == 8:
        m, s["scales"][:, 0] = _to8(m, s["local"], t, False)
        v, s["scales"][:, 1] = _to8(root, s["local"], t, True)
    s["m"].copy_(m)
    s["v"].copy_(v)
    return _adamw_out(s)


def _adamw_out(s):
    return {"param": s["param"], "master": s["master"], "m": s["m"], "v": s["v"],
            "scales": None if s["scales"] is None else s["scales"].view(torch.float8_e8m0fnu),
            "norm": s["norm"]}


# ------------------------------------------------------- the framework's calls

def _workspace(lib_size):
    return torch.empty(max(16, lib_size), dtype=torch.uint8, device=DEV)


def _own_norm(s):
    from expert_routing_grouped_moe_gb300 import lib
    c, out = s["case"], {}
    gate = dict(gate=s["gate"], gate_kind=c["gate"], gate_sigmoid=c["sigmoid"])
    if c["dir"] != "bwd":
        lib.moe_block_norm_fwd(s["x"], s["y"], s["r"], s["n"], w_post=s["w_post"],
                               w_pre=s["w_pre"], rstd_y=s["rstd_y"], rstd_r=s["rstd_r"],
                               scale=s["scale"], eps=EPS, w_offset=s["off"], **gate)
        out = {q: s[q] for q in ("r", "n", "rstd_y", "rstd_r")}
    if c["dir"] != "fwd":
        if s["ws"] is None:
            s["ws"] = _workspace(lib.moe_block_norm_workspace_size(c["T"], c["d"]))
        lib.moe_block_norm_bwd(s["dr"], s["dn"], s["r"], s["y"], s["dx"], s["dy"],
                               w_post=s["w_post"], w_pre=s["w_pre"], rstd_y=s["rstd_y"],
                               rstd_r=s["rstd_r"], dgate=s["dgate"], dw_post=s["dw_post"],
                               dw_pre=s["dw_pre"], ws=s["ws"], scale=s["scale"],
                               w_offset=s["off"], **gate)
        out.update({q: s[q] for q in ("dx", "dy", "dgate", "dw_post", "dw_pre")})
    return out


def _own_router(s):
    from expert_routing_grouped_moe_gb300 import lib
    c = s["case"]
    if s["ws"] is None:
        s["ws"] = _workspace(lib.moe_router_loss_workspace_size(c["T"], c["E"]))
    lib.moe_router_loss_fwd(s["logits"], s["counts"], c["k"], s["losses"], s["lse"], s["pmean"],
                            s["ws"])
    out = {q: s[q] for q in ("losses", "lse", "pmean")}
    if c["dir"] != "fwd":
        lib.moe_router_bwd(s["logits"], s["lse"], s["counts"], s["ids"], s["w"], s["dw"],
                           s["dlogits"], aux_coef=AUX, z_coef=ZED)
        out["dlogits"] = s["dlogits"]
    return out


def _own_adamw(s):
    from expert_routing_grouped_moe_gb300 import lib
    c = s["case"]
    if s["table"] is None:         # the optimizer's list of tensors, made once
        def row(o, n, wd):
            q, e = slice(o, o + n), slice(o // BLOCK, -(-(o + n) // BLOCK))
            return dict(param=s["param"][q], grad=s["grad"][q], m=s["m"][q], v=s["v"][q],
                        scales=None if s["scales"] is None else s["scales"][e],
                        master=None if s["master"] is None else s["master"][q], weight_decay=wd)
        s["table"] = lib.AdamWTable([row(*a) for a in zip(s["start"], s["sizes"], s["decay"])])
        s["ws"] = _workspace(lib.moe_adamw_workspace_size(s["table"]))
    s["step"] += 1
    lib.moe_adamw_step(s["table"], s["step"], lr=LR, betas=BETAS, eps=ADAM_EPS,
                       max_norm=c["clip"], grad_norm=s["norm"], ws=s["ws"])
    return _adamw_out(s)


# ------------------------------------------------------------- bytes and work

def work(case):
    c = case
    if c["op"] == "norm":
        n, xs, ys = c["T"] * c["d"], SIZE[c["x"]], SIZE[c["y"]]
        gate = {"none": 0, "token": 4 * c["T"], "channel": 4 * c["d"], "element": ys * n}[c["gate"]]
        weights = 4 * c["d"] * (c["post"] + c["pre"])
        saved = 4 * c["T"] * (c["post"] + c["pre"])
        fwd = n * (2 * xs + ys + ys * c["pre"]) + gate + weights + saved
        bwd = n * (2 * xs + xs * c["pre"] + 2 * ys + ys * c["pre"]) + 2 * gate + saved
        bwd += weights * (2 if c["learn"] else 1)
        return {"bytes": fwd * (c["dir"] != "bwd") + bwd * (c["dir"] != "fwd"),
                "flops": n * (14 * (c["dir"] != "bwd") + 30 * (c["dir"] != "fwd"))}
    if c["op"] == "router":
        n = c["T"] * c["E"]
        fwd = 4 * n + 4 * c["T"] + 8 * c["E"]
        bwd = 8 * n + 4 * c["T"] + 12 * c["T"] * c["k"] + 4 * c["E"]
        return {"bytes": fwd + bwd * (c["dir"] != "fwd"),
                "flops": n * (6 + 8 * (c["dir"] != "fwd"))}
    n = sum(_sizes(c))
    each = SIZE[c["grad"]] + SIZE[c["param"]] + (8 if c["master"] else SIZE[c["param"]])
    each += 16 if c["bits"] == 32 else 4 + 4 / BLOCK
    return {"bytes": int(n * each), "flops": 16 * n}


# ------------------------------------------------------------ 64-bit results

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "router": _exact_router, "adamw": _exact_adamw}[case["op"]](s)


def _exact_norm(s):
    """From the definition: r and n, and the gradients of <dr, r> + <dn, n> by the chain rule
    through the two quotients z / sqrt(mean z^2 + eps)."""
    c = s["case"]
    d = c["d"]
    wide = {q: v.double() for q, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    gate = wide.get("gate")
    if gate is None:
        a, slope = torch.ones((), dtype=torch.float64, device=DEV), None
    else:
        gate = gate.unsqueeze(1) if c["gate"] == "token" else gate
        a = torch.sigmoid(gate) if c["sigmoid"] else gate
        slope = torch.sigmoid(gate) * torch.sigmoid(-gate) if c["sigmoid"] else torch.ones_like(a)
    y = wide["y"]
    ry = ((y * y).sum(1, keepdim=True) / d + EPS) ** -0.5
    p = y * ry * wide["w_post"] if c["post"] else y
    r = wide["x"] + a * p * s["scale"]
    rr = ((r * r).sum(1, keepdim=True) / d + EPS) ** -0.5
    out = {}
    if c["dir"] != "bwd":
        out = {"r": r, "n": r * rr * wide["w_pre"] if c["pre"] else None,
               "rstd_y": ry[:, 0] if c["post"] else None, "rstd_r": rr[:, 0] if c["pre"] else None}
    else:
        r = wide["r"]                       # the backward's input: r as it was stored
        rr = wide["rstd_r"][:, None] if c["pre"] else rr
        ry = wide["rstd_y"][:, None] if c["post"] else ry
    if c["dir"] == "fwd":
        return out
    if c["dir"] == "both":                  # the backward reads r as it is stored
        r = r.to(s["x"].dtype).double()
    t = wide["dr"].clone()
    if c["pre"]:
        u = wide["dn"] * wide["w_pre"]
        t += rr * u - r * rr ** 3 * (u * r).sum(1, keepdim=True) / d
        if c["learn"]:
            out["dw_pre"] = torch.einsum("td,td->d", wide["dn"], r * rr)
    out["dx"] = t
    q = t * a * s["scale"]
    if c["post"]:
        u = q * wide["w_post"]
        out["dy"] = ry * u - y * ry ** 3 * (u * y).sum(1, keepdim=True) / d
        if c["learn"]:
            out["dw_post"] = torch.einsum("td,td->d", q, y * ry)
    else:
        out["dy"] = q
    if gate is not None:
        dg = t * (y * ry * wide["w_post"] if c["post"] else y) * s["scale"] * slope
        out["dgate"] = dg.sum(1) if c["gate"] == "token" else dg.sum(0) if c["gate"] == "channel" \
            else dg
    return out


def _exact_router(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"].double()
    lse = torch.logsumexp(l, 1)
    P = torch.exp(l - lse[:, None])
    f = s["counts"].double() / (T * k)
    out = {"losses": torch.stack([E * (P @ f).mean(), (lse ** 2).mean()]), "lse": lse,
           "pmean": P.sum(0) / T}
    if c["dir"] != "fwd":
        J = AUX * E / T * (f[None, :] - (P @ f)[:, None]) + 2 * ZED / T * lse[:, None]
        d = P * J
        w = torch.softmax(torch.gather(l, 1, s["ids"].long()), 1)
        dw = s["dw"].double()
        top = torch.zeros_like(d)
        top.scatter_(1, s["ids"].long(), w * dw - w * (w * dw).sum(1, keepdim=True))
        out["dlogits"] = d + top
    return out


def _exact_adamw(s):
    c, (b1, b2) = s["case"], BETAS
    t = s["step"] + 1
    eight = c["bits"] == 8
    g = s["grad"].double()
    out = {"norm": None}
    if c["clip"]:
        out["norm"] = torch.linalg.vector_norm(g).reshape(1)
        g = g * min(1.0, c["clip"] / (float(out["norm"]) + 1e-6))
    m, v = s["m"].double(), s["v"].double()
    if eight:
        unit = torch.exp2(s["scales"].double() - 127).repeat_interleave(BLOCK, 0)
        m, v = m * unit[:, 0], (v * unit[:, 1]) ** 2
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    wd = torch.cat([torch.full((n,), w, dtype=torch.float64, device=DEV)
                    for n, w in zip(s["padded"], s["decay"])])
    p = (s["param"] if s["master"] is None else s["master"]).double()
    p = p - LR * wd * p - LR * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + ADAM_EPS)
    out.update(param=p, master=p if c["master"] else None, m=m, v=v, scales=None)
    if eight:
        i = torch.cat([torch.arange(n, device=DEV) for n in s["padded"]])
        u = torch.remainder(i * DITHER_I + t * DITHER_T, 1 << 32)
        out["m"], em = _exact8(m, u)
        out["v"], er = _exact8(v.sqrt(), (1 << 32) - 1 - u)
        out["v"] = torch.where((v > 0) & (out["v"] == 0), torch.full_like(v, 2.0 ** -9), out["v"])
        out["scales"] = torch.stack([em, er], 1)
    return out


def _exact8(x, u):
    """x / scale on the grid of float8_e4m3, by floor(x / spacing + u): (values, scales)."""
    big = x.abs().view(-1, BLOCK).amax(1)
    e = torch.where(big > 0, torch.frexp(big).exponent - 1, -200).clamp(min=-112)
    scale = torch.exp2(e.double() - 7)
    z = x.abs() / scale.repeat_interleave(BLOCK)
    spacing = torch.exp2((torch.frexp(z).exponent - 1).clamp(min=-6).double() - 3)
    z = torch.floor(z / spacing + (u >> 12).double() / (1 << 20)) * spacing
    return torch.where(x < 0, -z, z), scale
