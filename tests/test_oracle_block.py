"""The oracle of the norms around a block, of the router's losses and of AdamW:
gradients against central differences in 64 bits, the losses and the optimizer
against what their definitions fix, the 8-bit state format against its own
grid (and torch's float8_e4m3fn and float8_e8m0fnu)."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo


def _diff(loss, z, h=1e-5):
    """Central differences of loss() in every entry of z (changed in place)."""
    g = np.zeros_like(z)
    for i in np.ndindex(z.shape):
        keep = z[i]
        z[i] = keep + h
        hi = loss()
        z[i] = keep - h
        lo = loss()
        z[i] = keep
        g[i] = (hi - lo) / (2 * h)
    return g


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("kind,sigmoid", [("none", False), ("token", False), ("token", True),
                                          ("channel", True), ("element", False),
                                          ("element", True)])
def test_norm_gradients_against_differences(post, pre, kind, sigmoid):
    rng = np.random.default_rng(3)
    T, d = 4, 5
    x, y, dr, dn = (rng.normal(size=(T, d)) for _ in range(4))
    wp = rng.normal(size=d) if post else None
    wq = rng.normal(size=d) if pre else None
    gate = {"none": None, "token": rng.normal(size=T), "channel": rng.normal(size=d),
            "element": rng.normal(size=(T, d))}[kind]
    kw = dict(gate=gate, kind=kind, sigmoid=sigmoid, scale=0.7, off=0.25)

    def loss():
        o = bo.block_norm_forward(x, y, wp, wq, eps=1e-3, **kw)
        return np.sum(o["r"] * dr) + (np.sum(o["n"] * dn) if pre else 0.0)

    f = bo.block_norm_forward(x, y, wp, wq, eps=1e-3, **kw)
    g = bo.block_norm_backward(dr, dn if pre else None, f["r"], y, wp, wq, f["rstd_y"],
                               f["rstd_r"], **kw)
    # differences of a smooth function with h = 1e-5: error about h^2 + 1e-16 / h
    tol = dict(rtol=1e-7, atol=1e-8)
    np.testing.assert_allclose(g["dx"], _diff(loss, x), **tol)
    np.testing.assert_allclose(g["dy"], _diff(loss, y), **tol)
    if post:
        np.testing.assert_allclose(g["dw_post"], _diff(loss, wp), **tol)
    if pre:
        np.testing.assert_allclose(g["dw_pre"], _diff(loss, wq), **tol)
    if kind != "none":
        np.testing.assert_allclose(g["dgate"], _diff(loss, gate), **tol)


def test_norm_of_x_alone_has_unit_mean_square():
    x = np.random.default_rng(1).normal(size=(3, 16)) * 5
    n = bo.block_norm_forward(x, None, w_pre=np.ones(16), eps=1e-12)["n"]
    np.testing.assert_allclose(np.mean(n * n, axis=1), 1.0, rtol=1e-10)


def test_router_gradient_against_differences():
    rng = np.random.default_rng(5)
    T, E, k, aux, z = 4, 6, 2, 0.3, 0.2
    l = rng.normal(size=(T, E))
    l[1, 2] = -np.inf                      # an expert that is switched off
    ids = np.argsort(-l, axis=1)[:, :k]
    counts = np.bincount(ids.reshape(-1), minlength=E)
    dw = rng.normal(size=(T, k))

    def weights():
        v = np.take_along_axis(l, ids, axis=1)
        e = np.exp(v - v.max(axis=1, keepdims=True))
        return e / e.sum(axis=1, keepdims=True)

    def loss():
        ls, _, _ = bo.router_losses(l, counts, k)
        return np.sum(weights() * dw) + aux * ls[0] + z * ls[1]

    g, _ = bo.router_backward(l, counts, ids, weights(), dw, aux, z, k)
    assert g[1, 2] == 0.0
    num = np.zeros_like(l)
    for t in range(T):
        for e in range(E):
            if np.isinf(l[t, e]):
                continue
            keep, h = l[t, e], 1e-5
            l[t, e] = keep + h
            hi = loss()
            l[t, e] = keep - h
            num[t, e] = (hi - loss()) / (2 * h)
            l[t, e] = keep
    np.testing.assert_allclose(g, num, rtol=1e-7, atol=1e-8)


def test_router_losses_even_load_and_empty_rows():
    l = np.zeros((8, 4))
    counts = np.array([4, 4, 4, 4])
    losses, lse, pm = bo.router_losses(l, counts, 2)
    np.testing.assert_allclose(losses, [1.0, np.log(4.0) ** 2])
    np.testing.assert_allclose(pm, 0.25)
    l[3] = -np.inf
    losses, lse, pm = bo.router_losses(l, counts, 2)
    assert np.isneginf(lse[3]) and np.isfinite(losses).all()
    np.testing.assert_allclose(losses[1], np.log(4.0) ** 2 * 7 / 8)
    g, _ = bo.router_backward(l, counts, np.zeros((8, 2), int), np.full((8, 2), .5),
                              np.ones((8, 2)), 1.0, 1.0, 2)
    assert np.all(g[3] == 0) and np.isfinite(g).all()


def test_adamw_first_step_is_the_sign_times_lr():
    g = np.array([3.0, -0.5, 1e-3])
    p, m, v = bo.adamw(np.ones(3), g, np.zeros(3), np.zeros(3), 1, lr=0.1, wd=0.5)
    np.testing.assert_allclose(p, 1 - 0.05 - 0.1 * np.sign(g), atol=1e-6)


def test_adamw_step32_is_adamw_within_fp32():
    rng = np.random.default_rng(2)
    p, g, m = (rng.normal(size=1000).astype(np.float32) for _ in range(3))
    v = (rng.normal(size=1000) ** 2).astype(np.float32)
    got = bo.adamw_step32(p, g, m, v, None, 7, 1e-2, 0.9, 0.999, 1e-8, 0.1)
    ref = bo.adamw(*(z.astype(np.float64) for z in (p, g, m, v)), 7, 1e-2, wd=0.1)
    for a, b in zip(got, ref):
        # at most 8 roundings on terms no larger than |p| + lr |m|/sqrt(v) ~ 10 here
        np.testing.assert_allclose(a, b, rtol=8 * 2.0 ** -24, atol=8 * 2.0 ** -24 * 10)


def test_e4m3_values_and_scales_are_torchs():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(bo.e4m3_value(codes), t)
    byte = torch.arange(8, 249, dtype=torch.int32).to(torch.uint8)
    s = byte.view(torch.float8_e8m0fnu).float().double().numpy()
    np.testing.assert_array_equal(s, np.exp2(byte.double().numpy() - 127))


def test_quantise_rounds_to_a_neighbour_and_is_even_over_steps():
    rng = np.random.default_rng(4)
    x = (rng.normal(size=700) * np.exp(3 * rng.normal(size=700))).astype(np.float32)
    x[5], x[300:310] = 0.0, 0.0
    mean = np.zeros(700)
    steps = 512
    for t in range(1, steps + 1):
        codes, byte = bo.adamw_quantise(x, t, False)
        assert not np.any((codes & 0x7F) > 0x78)          # no NaN, at most 256 scale
        s = np.repeat(np.exp2(byte.astype(float) - 127), 256)[:700]
        q = bo.e4m3_value(codes) * s
        step = np.maximum(np.abs(x) / 8, 2.0 ** -9 * s)    # spacing at or above x's binade
        assert np.all(np.abs(q - x) <= step)
        mean += q / steps
    # thresholds of a value over 512 steps: discrepancy of the golden ratio's
    # sequence, below (2 + log2 512) / 512 of a spacing, plus the 20-bit dither
    assert np.all(np.abs(mean - x) <= step * (11 / 512 + 2.0 ** -19))


def test_quantise_keeps_a_root_above_zero():
    x = np.zeros(256, dtype=np.float32)
    x[0], x[1] = 1.0, 1e-12
    codes, _ = bo.adamw_quantise(x, 1, True)
    assert codes[1] == 1 and codes[2] == 0
