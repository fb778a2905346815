"""Oracle of the operators at the ends of a stack of blocks and of its checkpoints:
embedding, log probabilities, 8-bit activations.  NumPy in 64 bits, written from
the formulas; the 8-bit format is whole numbers and powers of two, which 64 bits
hold exactly.  Shares no code with the package."""
import numpy as np


# ------------------------------------------------------------------- embedding

def embed(ids, table, scale=1.0):
    """out [..., d]; ids outside the table give zeros."""
    V = table.shape[0]
    ok = (ids >= 0) & (ids < V)
    out = scale * table[np.where(ok, ids, 0)]
    out[~ok] = 0.0
    return out


def embed_grad(ids, dout, V, scale=1.0, pad=None, base=None):
    """(dtable, sums of the sizes of its terms, number of terms of each row)."""
    d = dout.shape[-1]
    total = np.zeros((V, d)) if base is None else base.astype(np.float64).copy()
    mag, n = np.abs(total), np.zeros(V, dtype=np.int64)
    for i, row in zip(ids.reshape(-1), dout.reshape(-1, d)):
        if 0 <= i < V and i != pad:
            total[i] += scale * row
            mag[i] += abs(scale) * np.abs(row)
            n[i] += 1
    return total, mag, n


# ----------------------------------------------------------- log probabilities

def logprob(x, y, inv_temp=1.0, ignore=-100, top=0):
    """x [T,V], y [T,m] -> dict of lse [T], logp [T,m], p, logs (log p) [T,V],
    entropy [T], top_ids and top_logp [T,top]."""
    T, V = x.shape
    z = inv_temp * x
    with np.errstate(invalid="ignore", divide="ignore"):
        M = z.max(1, keepdims=True)
        M0 = np.where(np.isneginf(M), 0.0, M)
        e = np.exp(z - M0)
        log_sum = np.log(e.sum(1, keepdims=True))
        lse = M0 + log_sum
        logs = np.where(np.isneginf(z), -np.inf, (z - M0) - log_sum)   # also where all is -inf
    p = np.where(np.isneginf(lse), 0.0, np.exp(np.where(np.isneginf(lse), 0.0, logs)))
    out = {"lse": lse[:, 0], "p": p, "logs": logs}
    plogp = np.where(p > 0, p * np.where(p > 0, logs, 0.0), p)   # p: zeros, or NaN
    out["entropy"] = -plogp.sum(1)
    out["plogp"] = plogp
    ok = (y >= 0) & (y < V) & (y != ignore)
    out["ok"] = ok
    out["logp"] = np.where(ok, np.take_along_axis(logs, np.where(ok, y, 0), 1), 0.0)
    ids, lp = np.full((T, top), -1, dtype=np.int32), np.full((T, top), -np.inf)
    for t in range(T):
        order = sorted((c for c in range(V) if x[t, c] > -np.inf), key=lambda c: (-x[t, c], c))[:top]
        ids[t, :len(order)] = order
        lp[t, :len(order)] = logs[t, order]
    out["top_ids"], out["top_logp"] = ids, lp
    return out


def logprob_grad(x, y, inv_temp=1.0, ignore=-100, dlogp=None, dentropy=None, dlse=None):
    """(dx [T,V], sums of the sizes of its terms)."""
    r = logprob(x, y, inv_temp, ignore)
    T, V = x.shape
    g = np.where(r["ok"], 0.0 if dlogp is None else dlogp, 0.0)
    a = np.zeros(T) if dlse is None else dlse
    h = np.zeros(T) if dentropy is None else dentropy
    live = (g != 0).any(1) | (a != 0) | (h != 0)
    d = r["p"] * (a - g.sum(1))[:, None] - h[:, None] * (r["plogp"] + r["p"] * r["entropy"][:, None])
    mag = r["p"] * (np.abs(a) + np.abs(g).sum(1))[:, None] + np.abs(h)[:, None] * (
        np.abs(r["plogp"]) + r["p"] * np.abs(r["entropy"])[:, None])
    for t in range(T):
        for j in range(y.shape[1]):
            if r["ok"][t, j] and not np.isneginf(r["lse"][t]):
                d[t, y[t, j]] += g[t, j]
                mag[t, y[t, j]] += abs(g[t, j])
    d[~live], mag[~live] = 0.0, 0.0
    return inv_temp * d, abs(inv_temp) * mag


# ------------------------------------------------------------- 8-bit checkpoints

BLOCK = 32


def ckpt_pack(x):
    """(codes [R,C] int8, scale bytes [R, blocks] uint8) of x [R,C], exactly."""
    R, C = x.shape
    n = -(-C // BLOCK)
    codes, bytes_ = np.zeros((R, C), dtype=np.int8), np.zeros((R, n), dtype=np.uint8)
    for b in range(n):
        v = x[:, b * BLOCK:(b + 1) * BLOCK].astype(np.float64)
        big = np.abs(v).max(1)
        fine = np.isfinite(v).all(1)
        e = np.full(R, -126)
        for r in range(R):
            while fine[r] and 127.0 * 2.0 ** e[r] < big[r] and e[r] < 121:
                e[r] += 1
        q = np.rint(np.where(fine[:, None], v, 0.0) / 2.0 ** e[:, None].astype(np.float64))
        codes[:, b * BLOCK:(b + 1) * BLOCK] = q.clip(-127, 127).astype(np.int8)
        bytes_[:, b] = np.where(fine, e + 127, 255)
    return codes, bytes_


def ckpt_value(codes, bytes_):
    unit = np.where(bytes_ == 255, np.nan, 2.0 ** (bytes_.astype(np.float64) - 127))
    return codes * np.repeat(unit, BLOCK, 1)[:, :codes.shape[1]]


def swiglu_from(h, f, w):
    """act [P,f] = w silu(gate) up of h [P,hs] in chunks [gate 16 | up 16]."""
    col = np.arange(f)
    gate, up = h[:, col // 16 * 32 + col % 16], h[:, col // 16 * 32 + 16 + col % 16]
    with np.errstate(over="ignore"):
        return w[:, None] * gate / (1.0 + np.exp(-gate)) * up, gate
