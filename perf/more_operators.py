"""Timed cases of the operators at the ends of a stack of MoE blocks and of its checkpoints.

Three operators, each with inputs as a program that fine-tunes or samples a
language model has them in hand:

* ``embed``    rows of a table for token ids, scaled, and the table's gradient
               (``lib.moe_embed_fwd`` / ``_bwd``)
                 out[t] = scale table[ids[t]],   dtable[v] = scale sum_{t: ids[t] = v} dout[t]
               the gradient dense (rows without tokens are zeros) or added to what is there
* ``logprob``  log probabilities of given tokens, entropy and the top alternatives of
               each row of logits x, and the gradient of x (``lib.moe_logprob_fwd`` /
               ``_bwd``, or ``_step`` where the outputs' gradients are known ahead)
                 z = x / temperature,  lse = log sum exp z,  logp_j = z[y_j] - lse,
                 H = -sum p log p,   dz = sum_j g_j (1[y_j] - p) - g_H p (log p + H) + g_l p
* ``ckpt``     activations kept in 8 bits: codes int8 with a power-of-two scale (E8M0)
               for each 32 values of a row, and their use in the backward pass
               (``lib.moe_ckpt_pack`` / ``_unpack`` / ``_unpack_swiglu``)
                 e least with max |x| <= 127 2^e,  code = rint(x / 2^e),  x' = code 2^e
               a layer's pre-activations come back with act = w silu(gate) up as a pair
               of bf16 values, hi = bf16(act), lo = bf16(act - hi)

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits, rounded once at the end; with ``own`` true it calls the framework.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32                     # values that share a scale in 8 bits
IGNORE = -100                  # a target that asks for nothing
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
IDS = {32: torch.int32, 64: torch.int64}


# ------------------------------------------------------------------- cases

def _embed(name, dir, T, V, d, table="bf16", rows="bf16", scale=1.0, add=False, pad=False, ids=64):
    """rows: type of out (fwd) or dout (bwd); table: type of the table or of its gradient."""
    c = {"op": "embed", "dir": dir, "T": T, "V": V, "d": d, "table": table, "rows": rows,
         "scale": scale, "add": add, "pad": pad, "ids": ids}
    return dict(c, name=name) if name else c


def _logprob(name, dir, T, V, x="bf16", m=1, top=0, entropy=False, temp=1.0, blocked=0.0,
             ignored=0.0, ids=64):
    c = {"op": "logprob", "dir": dir, "T": T, "V": V, "x": x, "m": m, "top": top,
         "entropy": entropy, "temp": temp, "blocked": blocked, "ignored": ignored, "ids": ids}
    return dict(c, name=name) if name else c


def _ckpt(name, kind, T, d, k=1, x="fp32", shared=False):
    """kind "layer": pre-activations of T tokens' k experts (and a shared one), d features
    each for gate and up; kind "rows": [T, d] rows."""
    c = {"op": "ckpt", "kind": kind, "T": T, "d": d, "k": k, "x": x, "shared": shared}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the row of one sampled token: latency only
        _embed("embed fwd 1x2048", "fwd", 1, 151936, 2048),
        # a large packed batch at the gpt-oss-shaped width, residual stream in 32 bits, scaled
        _embed("embed fwd 65536x2880 fp32", "fwd", 65536, 201088, 2880, rows="fp32",
               scale=math.sqrt(2880)),
        # the dense gradient that an optimizer reads, one step of the Qwen3-30B-A3B-shaped layer
        _embed("embed bwd 4096x2048", "bwd", 4096, 151936, 2048, table="fp32"),
        # a ragged batch with padding and an odd width, added to a tied head's gradient
        _embed("embed bwd add 30011x1001", "bwd", 30011, 50257, 1001, table="fp32", rows="bf16",
               add=True, pad=True, ids=32),
        # the 20 likeliest tokens while one sequence is sampled
        _logprob("logprob fwd 1x151936 top 20", "fwd", 1, 151936, top=20, temp=0.7),
        # constrained sampling scored and trained on: switched-off tokens, prompts left out, an
        # odd vocabulary in 32 bits
        _logprob("logprob both 777x50257 fp32", "both", 777, 50257, x="fp32", top=5, entropy=True,
                 temp=0.8, blocked=0.3, ignored=0.25, ids=32),
        # distillation: a teacher's 8 tokens for each position, entropy trained too
        _logprob("logprob both 1024x201088 m 8", "both", 1024, 201088, m=8, top=8, entropy=True),
        # fine-tuning: the loss's weights are known, so one call gives values and gradient
        _logprob("logprob step 4096x151936", "step", 4096, 151936, ignored=0.1),
        # the smallest layer
        _ckpt("ckpt layer 256x64", "layer", 256, 64, 2),
        # the Qwen3-30B-A3B-shaped layer's pre-activations, kept and used again
        _ckpt("ckpt layer 4096x768 k 8", "layer", 4096, 768, 8),
        # a ragged batch through odd-sized experts with a shared one
        _ckpt("ckpt layer 1037x1000 k 4 shared", "layer", 1037, 1000, 4, shared=True),
        # rows of the block side at the gpt-oss-shaped width
        _ckpt("ckpt rows 16384x2880 bf16", "rows", 16384, 2880, x="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case, no costlier than the largest listed one."""
    op = rng.choice(["embed", "embed", "logprob", "logprob", "ckpt"])
    if op == "embed":
        d = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 512), 2048, 2880])
        V = rng.choice([_log(rng, 1000, 200_000), 50257, 151936])
        V = min(V, 320_000_000 // d)
        T = max(1, min(_log(rng, 1, 131072), 65536 * 2880 // d))
        dir = rng.choice(["fwd", "bwd", "bwd"])
        return _embed("", dir, T, V, d, rng.choice(["bf16", "fp32"]), rng.choice(["bf16", "fp32"]),
                      rng.choice([1.0, math.sqrt(d)]), dir == "bwd" and rng.random() < 0.4,
                      dir == "bwd" and rng.random() < 0.3, rng.choice([32, 64]))
    if op == "logprob":
        x = rng.choice(["bf16", "bf16", "fp32"])
        V = rng.choice([_log(rng, 1000, 200_000), 8 * _log(rng, 125, 25000), 50257, 151936])
        T = max(1, min(_log(rng, 1, 65536), 4096 * 151936 // V // (2 if x == "fp32" else 1)))
        top = rng.choice([0, 0, 1, 5, 20])
        if top:
            T = max(1, T // 4)
        return _logprob("", rng.choice(["fwd", "both", "step"]), T, V, x,
                        rng.choice([1, 1, 1, 4, 8]), top, rng.random() < 0.5,
                        rng.choice([1.0, 1.0, 0.7]), rng.choice([0.0, 0.0, 0.3]),
                        rng.choice([0.0, 0.3]), rng.choice([32, 64]))
    if rng.random() < 0.6:
        k, f = rng.choice([1, 2, 4, 8]), rng.choice([8 * _log(rng, 8, 360), 768, 1000, 2880])
        T = max(1, min(_log(rng, 1, 32768), 30_000_000 // (k * f)))
        return _ckpt("", "layer", T, f, k, shared=rng.random() < 0.3)
    d = rng.choice([_log(rng, 64, 8192), 2048, 2880])
    return _ckpt("", "rows", max(1, min(_log(rng, 1, 65536), 60_000_000 // d)), d, 1,
                 rng.choice(["bf16", "fp32"]))


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(DEV)
    g.manual_seed(int(seed) * 7919 + 23)
    return {"embed": _prepare_embed, "logprob": _prepare_logprob,
            "ckpt": _prepare_ckpt}[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _zipf(g, V, *shape):
    """Ids whose frequency falls as 1 / rank, as words do."""
    u = torch.rand(*shape, generator=g, device=DEV, dtype=torch.float64)
    return (torch.exp(u * math.log(V + 1)) - 1).long().clamp(0, V - 1)


def _prepare_embed(c, g):
    T, V, d = c["T"], c["V"], c["d"]
    ids = _zipf(g, V, T)
    s = {"case": c, "op": "embed", "pad": V - 1 if c["pad"] else None, "ws": None}
    if c["pad"]:               # the ends of padded sequences
        ids[torch.arange(T, device=DEV) % 512 >= 400] = V - 1
    s["ids"] = ids.to(IDS[c["ids"]])
    if c["dir"] == "fwd":
        s["table"] = (0.02 * _randn(g, V, d)).to(TYPES[c["table"]])
        s["out"] = torch.empty(T, d, dtype=TYPES[c["rows"]], device=DEV)
    else:
        s["dout"] = (1e-3 * _randn(g, T, d)).to(TYPES[c["rows"]])
        s["dtable"] = (1e-3 * _randn(g, V, d)).to(TYPES[c["table"]]) if c["add"] else torch.empty(
            V, d, dtype=TYPES[c["table"]], device=DEV)
    return s


def _prepare_logprob(c, g):
    T, V, m, xt = c["T"], c["V"], c["m"], TYPES[c["x"]]
    # frequent tokens are likelier, and each row has a level of its own
    level = -torch.log(torch.arange(1, V + 1, device=DEV, dtype=torch.float32))
    x = _randn(g, T, V).mul_(2.0).add_(level).add_(4.0 * _randn(g, T, 1))
    if c["blocked"]:
        x.masked_fill_(torch.rand(V, generator=g, device=DEV) < c["blocked"], -math.inf)
    s = {"case": c, "op": "logprob", "logits": x.to(xt), "inv": 1.0 / c["temp"]}
    y = _zipf(g, V, T, m)
    y = torch.where(torch.isinf(torch.gather(x, 1, y)), x.argmax(1, keepdim=True), y)
    y[torch.rand(T, generator=g, device=DEV) < c["ignored"]] = IGNORE
    del x
    s["targets"] = (y if m > 1 else y[:, 0]).to(IDS[c["ids"]])
    f32 = dict(dtype=torch.float32, device=DEV)
    w = torch.softmax(_randn(g, T, m), 1) if m > 1 else torch.ones(T, 1, **f32)
    s["dlogp"] = (-w / T).reshape(s["targets"].shape).contiguous()
    s["dentropy"] = torch.full((T,), -0.01 / T, **f32) if c["entropy"] else None
    s["logp"], s["stats"] = torch.empty(s["targets"].shape, **f32), torch.empty(T, 2, **f32)
    s["lse"] = torch.empty(T, **f32)
    s["entropy"] = torch.empty(T, **f32) if c["entropy"] else None
    s["top_ids"] = torch.empty(T, c["top"], dtype=torch.int32, device=DEV) if c["top"] else None
    s["top_logp"] = torch.empty(T, c["top"], **f32) if c["top"] else None
    s["dlogits"] = None if c["dir"] == "fwd" else torch.empty_like(s["logits"])
    return s


def _prepare_ckpt(c, g):
    s = {"case": c, "op": "ckpt"}
    if c["kind"] == "rows":
        T, d = c["T"], c["d"]
        s["x"] = (_randn(g, T, d) * torch.exp(0.8 * _randn(g, d))).to(TYPES[c["x"]])
        s["y"] = torch.empty_like(s["x"])
        R, C = T, d
    else:
        K = c["k"] + c["shared"]
        R, f = c["T"] * K, c["d"]
        C = 32 * ((f + 15) // 16)
        # [gate 16 | up 16] chunks, the features past f zeros
        x = _randn(g, R, C) * torch.exp(0.5 * _randn(g, R, 1))
        x.view(R, -1, 2, 16).masked_fill_(
            torch.arange(C // 2, device=DEV).view(-1, 1, 16) >= f, 0.0)
        s["x"], s["y"] = x, torch.empty_like(x)
        s["order"] = torch.randperm(R, generator=g, device=DEV).to(torch.int32)
        s["w"] = torch.softmax(_randn(g, c["T"], c["k"]), 1)
        s["act"] = torch.empty(2, R, f, dtype=torch.bfloat16, device=DEV)
    s["codes"] = torch.empty(R, C, dtype=torch.int8, device=DEV)
    s["scales"] = torch.empty(R, -(-C // BLOCK), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------- plain forms

def run(state):
    if own:
        return {"embed": _own_embed, "logprob": _own_logprob, "ckpt": _own_ckpt}[state["op"]](state)
    return {"embed": _plain_embed, "logprob": _plain_logprob,
            "ckpt": _plain_ckpt}[state["op"]](state)


def _plain_embed(s):
    c = s["case"]
    if c["dir"] == "fwd":
        return {"out": (s["table"][s["ids"]].float() * c["scale"]).to(TYPES[c["rows"]])}
    rows, ids = s["dout"].float() * c["scale"], s["ids"]
    if s["pad"] is not None:
        rows = rows * (ids != s["pad"])[:, None]
    if c["add"]:
        total = s["dtable"].float()
    else:
        total = torch.zeros(c["V"], c["d"], device=DEV)
    total.index_add_(0, ids, rows)
    if c["add"]:
        s["dtable"].copy_(total)
        return {"dtable": s["dtable"]}
    return {"dtable": total.to(TYPES[c["table"]])}


def _plain_logprob(s):
    c, out = s["case"], {}
    x = s["logits"].float()
    z = x * s["inv"]
    y = s["targets"].long().view(c["T"], c["m"])
    asked = y != IGNORE
    y = torch.where(asked, y, 0)
    top = z.amax(1, keepdim=True)
    z = z - top
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    logp = torch.where(asked, torch.gather(z, 1, y) - log_total, 0.0)
    out["logp"], out["lse"] = logp.view(s["targets"].shape), (top + log_total)[:, 0]
    p = e / total
    if c["entropy"]:
        z = z.clamp(min=-1e4) - log_total
        entropy = -(p * z).sum(1, keepdim=True)
        out["entropy"] = entropy[:, 0]
    if c["top"]:
        # values in the order of whole numbers, the lower id first among equal ones
        key = (x + 0.0).view(torch.int32).long()
        key = torch.where(key < 0, key ^ 0x7FFFFFFF, key)
        key = key * 2 ** 32 + torch.arange(c["V"] - 1, -1, -1, device=DEV)
        ids = c["V"] - 1 - torch.topk(key, c["top"], dim=1).values % 2 ** 32
        del key
        value = torch.gather(x, 1, ids) * s["inv"] - top - log_total
        out["top_ids"] = torch.where(value == -math.inf, -1, ids).to(torch.int32)
        out["top_logp"] = value
    if c["dir"] != "fwd":
        g = torch.where(asked, s["dlogp"].view(c["T"], c["m"]), 0.0)
        d = -g.sum(1, keepdim=True) * p
        if c["entropy"]:
            d -= s["dentropy"][:, None] * p * (z + entropy)
        d.scatter_add_(1, y, g)
        out["dlogits"] = (d * s["inv"]).to(TYPES[c["x"]])
    return out


def _pow2(e):
    """2^e for whole e in -126 .. 127, exactly."""
    return ((e + 127) << 23).view(torch.float32)


def _plain_pack(x):
    """Codes [R, C] and scale bytes [R, blocks] of x [R, C]."""
    R, C = x.shape
    n = -(-C // BLOCK)
    x = torch.nn.functional.pad(x.float(), (0, n * BLOCK - C)).view(R, n, BLOCK)
    big = x.abs().amax(2)
    # exponent and leading bits of the largest, against 127 = 1.984375 * 2^6
    e = (((big.view(torch.int32) + 0x1FFFF) >> 23) - 133).clamp(min=-126)
    codes = torch.round(x * _pow2(-e)[:, :, None])
    return codes.view(R, n * BLOCK)[:, :C].to(torch.int8), (e + 127).to(torch.uint8)


def _plain_unpack(codes, scales):
    unit = _pow2(scales.to(torch.int32) - 127).repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
    return codes.float() * unit


def _weights(s):
    """The weight of each sorted row: its slot's, 1 for the shared expert's."""
    c = s["case"]
    w = torch.cat([s["w"], torch.ones(c["T"], 1, device=DEV)], 1) if c["shared"] else s["w"]
    return w.reshape(-1)[s["order"].long()]


def _plain_ckpt(s):
    c = s["case"]
    codes, scales = _plain_pack(s["x"])
    x = _plain_unpack(codes, scales)
    out = {"codes": codes, "scales": scales.view(torch.float8_e8m0fnu)}
    if c["kind"] == "rows":
        out["x"] = x.to(TYPES[c["x"]])
        return out
    h = x.view(x.shape[0], -1, 2, 16)
    gate = h[:, :, 0].reshape(x.shape[0], -1)[:, :c["d"]]
    up = h[:, :, 1].reshape(x.shape[0], -1)[:, :c["d"]]
    act = _weights(s)[:, None] * (gate / (1.0 + torch.exp(-gate))) * up
    high = act.to(torch.bfloat16)
    out.update(h=x, act=torch.stack([high, (act - high.float()).to(torch.bfloat16)]))
    return out


# ------------------------------------------------------- the framework's calls

def _own_embed(s):
    from expert_routing_grouped_moe_gb300 import lib
    c = s["case"]
    if c["dir"] == "fwd":
        lib.moe_embed_fwd(s["ids"], s["table"], s["out"], scale=c["scale"])
        return {"out": s["out"]}
    if s["ws"] is None:
        s["ws"] = torch.empty(max(16, lib.moe_embed_workspace_size(c["T"], c["V"], c["d"])),
                              dtype=torch.uint8, device=DEV)
    lib.moe_embed_bwd(s["ids"], s["dout"], s["dtable"], s["ws"], scale=c["scale"], pad_id=s["pad"],
                      accumulate=c["add"])
    return {"dtable": s["dtable"]}


def _own_logprob(s):
    from expert_routing_grouped_moe_gb300 import lib
    c = s["case"]
    want = dict(lse=s["lse"], entropy=s["entropy"], top_ids=s["top_ids"], top_logp=s["top_logp"],
                inv_temp=s["inv"], ignore_id=IGNORE)
    if c["dir"] == "step":
        lib.moe_logprob_step(s["logits"], s["targets"], s["logp"], s["stats"], s["dlogp"],
                             s["dlogits"], dentropy=s["dentropy"], **want)
    else:
        lib.moe_logprob_fwd(s["logits"], s["targets"], s["logp"], s["stats"], **want)
    if c["dir"] == "both":
        lib.moe_logprob_bwd(s["logits"], s["targets"], s["stats"], s["dlogp"], s["dlogits"],
                            entropy=s["entropy"], dentropy=s["dentropy"], inv_temp=s["inv"],
                            ignore_id=IGNORE)
    names = ["logp", "lse"] + ["entropy"] * c["entropy"]
    names += ["top_ids", "top_logp"] * (c["top"] > 0) + ["dlogits"] * (c["dir"] != "fwd")
    return {q: s[q] for q in names}


def _own_ckpt(s):
    from expert_routing_grouped_moe_gb300 import lib
    c = s["case"]
    lib.moe_ckpt_pack(s["x"], s["codes"], s["scales"])
    out = {"codes": s["codes"], "scales": s["scales"].view(torch.float8_e8m0fnu)}
    if c["kind"] == "rows":
        lib.moe_ckpt_unpack(s["codes"], s["scales"], s["y"])
        out["x"] = s["y"]
        return out
    lib.moe_ckpt_unpack_swiglu(s["codes"], s["scales"], s["order"], s["w"], c["shared"], s["y"],
                               s["act"])
    out.update(h=s["y"], act=s["act"])
    return out


# ------------------------------------------------------------- bytes and work

def work(case):
    c = case
    if c["op"] == "embed":
        n = c["T"] * c["d"]
        size, rows = SIZE[c["table"]], SIZE[c["rows"]]
        # distinct ids of T draws: id v has the share log(1 + 1 / (v + 1)) / log(V + 1)
        groups = [(lo, min(2 * lo, c["V"] + 1)) for lo in _doubling(c["V"])]
        share = [math.log(hi / lo) / (hi - lo) / math.log(c["V"] + 1) for lo, hi in groups]
        distinct = sum((hi - lo) * -math.expm1(-c["T"] * p) for (lo, hi), p in zip(groups, share))
        if c["dir"] == "fwd":
            return {"bytes": int(distinct * c["d"] * size + n * rows + c["T"] * c["ids"] / 8),
                    "flops": n}
        out = 2 * distinct * c["d"] if c["add"] else c["V"] * c["d"]
        read = 400 / 512 if c["pad"] else 1.0
        return {"bytes": int(n * rows * read + out * size + c["T"] * c["ids"] / 8), "flops": 2 * n}
    if c["op"] == "logprob":
        n, T = c["T"] * c["V"], c["T"]
        size = SIZE[c["x"]]
        small = T * (c["m"] * (c["ids"] / 8 + 4) + 12 + 4 * c["entropy"] + 8 * c["top"])
        passes = {"fwd": 1, "both": 3, "step": 2}[c["dir"]]
        if c["dir"] == "both" and not c["entropy"]:
            passes -= c["ignored"]   # rows without a target get zeros, without being read
        return {"bytes": int(n * size * passes + small),
                "flops": n * (4 + 2 * c["entropy"] + (c["dir"] != "fwd") * (3 + 2 * c["entropy"]))}
    if c["kind"] == "rows":
        n = c["T"] * c["d"]
        return {"bytes": 2 * n * SIZE[c["x"]] + 2 * n + 2 * n // BLOCK, "flops": 4 * n}
    R = c["T"] * (c["k"] + c["shared"])
    C = 32 * ((c["d"] + 15) // 16)
    return {"bytes": R * (10 * C + 2 * C // BLOCK + 4 * c["d"]) + 4 * R + 4 * c["T"] * c["k"],
            "flops": R * (4 * C + 8 * c["d"])}


def _doubling(V):
    return [2 ** i for i in range(V.bit_length()) if 2 ** i <= V]


# ------------------------------------------------------------ 64-bit results

def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "logprob": _exact_logprob, "ckpt": _exact_ckpt}[case["op"]](s)


def _exact_embed(s):
    """Rows picked and summed in 64 bits, the sums over tokens in the order of sorted ids."""
    c = s["case"]
    ids = s["ids"].long()
    if c["dir"] == "fwd":
        return {"out": torch.index_select(s["table"], 0, ids).double() * c["scale"]}
    if s["pad"] is not None:
        keep = ids != s["pad"]
        ids, dout = ids[keep], s["dout"][keep]
    else:
        dout = s["dout"]
    full = s["dtable"].double() if c["add"] else torch.zeros(c["V"], c["d"], dtype=torch.float64,
                                                             device=DEV)
    order = torch.argsort(ids, stable=True)
    seen, count = torch.unique_consecutive(ids[order], return_counts=True)
    sums = torch.segment_reduce(dout[order].double(), "sum", lengths=count, axis=0)
    full[seen] += c["scale"] * sums
    return {"dtable": full}


def _exact_logprob(s):
    """Row groups of at most 2^27 logits, so that 64 bits fit the card beside the inputs."""
    c = s["case"]
    per = max(1, 2 ** 27 // c["V"])
    parts = [_exact_rows(s, slice(i, i + per)) for i in range(0, c["T"], per)]
    return {q: None if parts[0][q] is None else torch.cat([p[q] for p in parts]) for q in parts[0]}


def _exact_rows(s, rows):
    c, out = s["case"], {}
    z = s["logits"][rows].double() / c["temp"]
    y = s["targets"][rows].long()
    y = y[:, None] if y.dim() == 1 else y
    lse = torch.logsumexp(z, 1, keepdim=True)
    lp = z - lse
    valid = (y >= 0).double()
    picked = torch.gather(lp, 1, y.clamp(min=0)).masked_fill(y < 0, 0.0)
    out["logp"] = picked if c["m"] > 1 else picked[:, 0]
    out["lse"] = lse[:, 0]
    p = torch.exp(lp)
    if c["entropy"]:
        plogp = torch.xlogy(p, p)
        out["entropy"] = -plogp.sum(1)
    if c["top"]:
        out["top_ids"] = None
        out["top_logp"] = torch.topk(lp, c["top"], 1).values
    if c["dir"] != "fwd":
        w = s["dlogp"][rows].double().reshape(y.shape) * valid
        d = torch.zeros_like(z)
        d.scatter_add_(1, y.clamp(min=0), w)
        d -= p * w.sum(1, keepdim=True)
        if c["entropy"]:
            d -= s["dentropy"][rows].double()[:, None] * (plogp + p * out["entropy"][:, None])
        out["dlogits"] = d / c["temp"]
    return out


def _exact_ckpt(s):
    """Codes by division in 64 bits, from the definition of the exponent."""
    c = s["case"]
    x = s["x"].double()
    R, C = x.shape
    block = torch.arange(C, device=DEV) // BLOCK
    big = torch.zeros(R, -(-C // BLOCK), dtype=torch.float64, device=DEV)
    big.scatter_reduce_(1, block.expand(R, C), x.abs(), "amax")
    e = torch.ceil(torch.log2(big.clamp(min=2.0 ** -150) / 127)).clamp(min=-126)
    e = torch.where(127 * torch.exp2(e) < big, e + 1, e)        # the logarithm's rounding
    e = torch.where((127 * torch.exp2(e - 1) >= big) & (e > -126), e - 1, e)
    unit = torch.exp2(e)[:, block]
    codes = torch.round(x / unit)
    value = codes * unit
    out = {"codes": None, "scales": torch.exp2(e)}
    if c["kind"] == "rows":
        out["x"] = value
        return out
    f = c["d"]
    col = torch.arange(f, device=DEV)
    gate = value[:, col // 16 * 32 + col % 16]
    up = value[:, col // 16 * 32 + 16 + col % 16]
    slot = s["order"].long() % (c["k"] + c["shared"])
    token = s["order"].long() // (c["k"] + c["shared"])
    w = torch.where(slot < c["k"], s["w"].double()[token, slot.clamp(max=c["k"] - 1)], 1.0)
    act = torch.sigmoid(gate) * gate * up * w[:, None]
    # the two halves together hold act; the second is what the first leaves over
    high = act.to(torch.bfloat16).double()
    out.update(h=value, act=torch.stack([high, act - high]))
    return out
