"""Oracle of the operators around the expert layer: norms with gate and residual
scale, router losses, AdamW.  NumPy in 64 bits, written from the formulas; the
8-bit optimizer step restates the stored format in fp32 operations, one rounding
each, because its results are defined to the bit.  Shares no code with the
package."""
import math

import numpy as np


# ------------------------------------------------------------- norms around a block

def _gate(gate, kind, sigmoid):
    """(a, a') broadcastable over [T, d]."""
    if kind == "none":
        return np.float64(1.0), np.float64(0.0)
    g = np.asarray(gate, dtype=np.float64)
    g = g[:, None] if kind == "token" else g
    if not sigmoid:
        return g, np.ones_like(g)
    with np.errstate(over="ignore"):
        a, b = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
    return a, a * b


def _rstd(z, eps):
    return 1.0 / np.sqrt(np.mean(z * z, axis=1, keepdims=True) + eps)


def block_norm_forward(x, y, w_post=None, w_pre=None, gate=None, kind="none", sigmoid=False,
                       scale=1.0, eps=1e-6, off=0.0):
    """dict with r, n, rstd_y, rstd_r and the sizes of their terms (mag_r, mag_n)."""
    out = {"rstd_y": None, "rstd_r": None, "n": None}
    x = np.zeros_like(y) if x is None else x
    r, mag = x, np.abs(x)
    if y is not None:
        p = y
        if w_post is not None:
            ry = _rstd(y, eps)
            out["rstd_y"] = ry[:, 0]
            p = y * ry * (w_post + off)
        add = scale * _gate(gate, kind, sigmoid)[0] * p
        r, mag = x + add, np.abs(x) + np.abs(add)
    out["r"], out["mag_r"] = r, mag
    if w_pre is not None:
        rr = _rstd(r, eps)
        out["rstd_r"] = rr[:, 0]
        out["n"] = r * rr * (w_pre + off)
        out["mag_n"] = mag * rr * np.abs(w_pre + off)
    return out


def block_norm_backward(dr, dn, r, y, w_post=None, w_pre=None, rstd_y=None, rstd_r=None, gate=None,
                        kind="none", sigmoid=False, scale=1.0, off=0.0):
    """dict with dx, dy, dgate, dw_post, dw_pre and, as mag_*, the sum of the
    sizes of the terms each value is made of."""
    out = {}
    shape = (r if r is not None else y).shape
    t = np.zeros(shape) if dr is None else dr.copy()
    mag = np.abs(t)
    if w_pre is not None:
        rr = rstd_r[:, None]
        hat, u = r * rr, dn * (w_pre + off)
        t = t + rr * (u - hat * np.mean(u * hat, axis=1, keepdims=True))
        mag = mag + rr * (np.abs(u) + np.abs(hat) * np.mean(np.abs(u * hat), axis=1, keepdims=True))
        out["dw_pre"] = np.sum(dn * hat, axis=0)
        out["mag_dw_pre"] = np.sum(np.abs(dn * hat), axis=0)
    out["dx"], out["mag_dx"] = t, mag
    if y is None:
        return out
    a, da = _gate(gate, kind, sigmoid)
    dp, mdp, p = scale * a * t, np.abs(scale * a) * mag, y
    if w_post is not None:
        ry = rstd_y[:, None]
        hat, w = y * ry, w_post + off
        p = hat * w
        out["dw_post"] = np.sum(dp * hat, axis=0)
        out["mag_dw_post"] = np.sum(mdp * np.abs(hat), axis=0)
        dy = ry * (dp * w - hat * np.mean(dp * p, axis=1, keepdims=True))
        mdy = ry * (mdp * np.abs(w) + np.abs(hat) * np.mean(mdp * np.abs(p), axis=1, keepdims=True))
    else:
        dy, mdy = dp, mdp
    out["dy"], out["mag_dy"] = dy, mdy
    if kind != "none":
        dg, mdg = scale * da * t * p, np.abs(scale * da) * mag * np.abs(p)
        axis = {"token": 1, "channel": 0, "element": None}[kind]
        out["dgate"] = dg if axis is None else dg.sum(axis)
        out["mag_dgate"] = mdg if axis is None else mdg.sum(axis)
    return out


# ---------------------------------------------------------------------- router

def _softmax(l):
    """(P, lse) of rows that may hold -inf; an empty row has P = 0, lse = -inf."""
    m = l.max(axis=1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore"):
        ex = np.exp(l - m)
        s = ex.sum(axis=1, keepdims=True)
        lse = (m + np.log(s))[:, 0]
    return ex / np.where(s == 0, 1.0, s), lse


def router_losses(logits, counts, k):
    """(losses [2], lse [T], pmean [E])."""
    T, E = logits.shape
    P, lse = _softmax(logits)
    pm = P.sum(axis=0) / T
    f = counts[:E] / (T * k)
    z = np.where(np.isneginf(lse), 0.0, lse)
    return np.array([E * np.sum(f * pm), np.sum(z * z) / T]), lse, pm


def router_backward(logits, counts, ids, weights, dweights, aux, z, k):
    """dlogits, and the sum of the sizes of its terms."""
    T, E = logits.shape
    P, lse = _softmax(logits)
    l0 = np.where(np.isneginf(lse), 0.0, lse)[:, None]
    f = counts[:E] / (T * k) if counts is not None else np.zeros(E)
    dot = (P * f).sum(axis=1, keepdims=True)
    d = P * (aux * E / T * (f - dot) + 2.0 * z / T * l0)
    mag = P * (abs(aux) * E / T * (f + dot) + 2.0 * abs(z) / T * np.abs(l0))
    if dweights is not None:
        live = ~np.isneginf(lse)
        c = weights * (dweights - (weights * dweights).sum(axis=1, keepdims=True))
        cm = weights * (np.abs(dweights) + np.abs(weights * dweights).sum(axis=1, keepdims=True))
        for t in np.nonzero(live)[0]:
            for j in range(ids.shape[1]):
                if 0 <= ids[t, j] < E:
                    d[t, ids[t, j]] += c[t, j]
                    mag[t, ids[t, j]] += cm[t, j]
    return d, mag


# ----------------------------------------------------------------------- AdamW

def adamw(p, g, m, v, step, lr, b1=0.9, b2=0.999, eps=1e-8, wd=0.0):
    """(p, m, v) after one step, in 64 bits."""
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    up = (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return p * (1 - lr * wd) - lr * up, m, v


ADAMW_BLOCK = 256
_T, _I = 2654435769, 1779033703   # floor(2^32 frac(golden ratio)), floor(2^32 frac(sqrt 2)), odd


def e4m3_value(codes):
    """Values of e4m3 bytes (1-4-3 bits, bias 7, no infinities)."""
    c = np.asarray(codes, dtype=np.int64)
    e, f = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, f * 2.0 ** -9, (8 + f) * np.exp2(e - 10.0))
    return np.where(c & 128, -mag, mag)


def _code(mag):
    """e4m3 magnitude code of values that lie on its grid."""
    grid = e4m3_value(np.arange(0x7F))
    return np.searchsorted(grid, mag)


def adamw_quantise(x, step, root):
    """(codes, scale bytes) of the fp32 values x: floor(x / (spacing scale) + u) on the e4m3
    grid, u the step's dither, the scale of each block of 256 from its largest value."""
    n = x.size
    blocks = -(-n // ADAMW_BLOCK)
    z = np.zeros(blocks * ADAMW_BLOCK)
    z[:n] = np.abs(x.astype(np.float64))
    top = z.reshape(blocks, -1).max(axis=1)
    e = np.floor(np.log2(np.where(top > 0, top, 2.0 ** -200)))
    byte = np.maximum(e + 127 - 7, 8)
    z = (z.reshape(blocks, -1) / np.exp2(byte - 127)[:, None]).reshape(-1)[:n]
    u = (np.arange(n, dtype=np.uint64) * np.uint64(_I) + np.uint64(step * _T % 2 ** 32)) % 2 ** 32
    u = (2 ** 32 - 1 - u) if root else u
    u = (u.astype(np.uint64) >> np.uint64(12)).astype(np.float64) * 2.0 ** -20
    spacing = np.exp2(np.maximum(np.floor(np.log2(np.maximum(z, 2.0 ** -40))), -6) - 3)
    code = _code(np.floor(z / spacing + u) * spacing)
    if root:
        code = np.where((z > 0) & (code == 0), 1, code)
    return (code + 128 * (x < 0)).astype(np.uint8), byte.astype(np.uint8)


def adamw_step32(p, g, m, v, codes, step, lr, b1, b2, eps, wd, coef=1.0, lr_mult=1.0):
    """One step in fp32 with every operation rounded by itself.  Moments: fp32 m and v,
    or codes = (m codes, root codes, scale bytes [blocks, 2]).  Returns p and the new
    moments in the same form."""
    f = np.float32
    if codes is not None:
        def value(c, byte):
            s = np.repeat(np.exp2(byte.astype(np.float64) - 127), ADAMW_BLOCK)[:c.size]
            return (e4m3_value(c) * s).astype(f)
        m = value(codes[0], codes[2][:, 0])
        v = value(codes[1], codes[2][:, 1])
        v = v * v
    lr = lr * lr_mult
    g = g.astype(f) * f(coef)
    m = f(b1) * m + f(1 - b1) * g
    v = f(b2) * v + (f(1 - b2) * g) * g
    root = np.sqrt(v)
    up = m / (root * f(1 / math.sqrt(1 - b2 ** step)) + f(eps))
    p = p.astype(f) * f(1 - lr * wd) - f(lr / (1 - b1 ** step)) * up
    if codes is None:
        return p, m, v
    cm, bm = adamw_quantise(m, step, False)
    cr, br = adamw_quantise(root, step, True)
    return p, cm, cr, np.stack([bm, br], axis=1)
