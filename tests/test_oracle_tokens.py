"""The oracle of embedding, log probabilities and 8-bit checkpoints: central
differences, limits, and the format's definition."""
import numpy as np
import pytest

from oracle import token_oracle as to

RNG = np.random.default_rng


def test_embedding_gradient_is_the_transpose():
    """<embed(ids, W), dout> = <W, embed_grad(ids, dout)> for every W."""
    g = RNG(1)
    ids = g.integers(-1, 8, (5, 4))
    W, dout = g.standard_normal((7, 3)), g.standard_normal((5, 4, 3))
    dW, _, n = to.embed_grad(ids, dout, 7, 0.3)
    assert np.isclose((to.embed(ids, W, 0.3) * dout).sum(), (W * dW).sum())
    assert n.sum() == ((ids >= 0) & (ids < 7)).sum()
    pad, _, _ = to.embed_grad(ids, dout, 7, 0.3, pad=2)
    assert not pad[2].any() and np.array_equal(np.delete(pad, 2, 0), np.delete(dW, 2, 0))


@pytest.mark.parametrize("m,inv", [(1, 1.0), (3, 0.7), (4, 2.5)])
def test_logprob_gradient_by_central_differences(m, inv):
    g = RNG(m)
    x = g.standard_normal((3, 9))
    x[1, 4] = -np.inf
    y = g.integers(0, 9, (3, m))
    y[0, 0] = -100
    y[2, -1] = y[2, 0]
    y[y == 4] = 5
    dlogp, dh, dl = g.standard_normal((3, m)), g.standard_normal(3), g.standard_normal(3)

    def loss(x):
        r = to.logprob(x, y, inv)
        return (r["logp"] * np.where(y >= 0, dlogp, 0)).sum() + (r["entropy"] * dh).sum() + (
            r["lse"] * dl).sum()
    d, _ = to.logprob_grad(x, y, inv, dlogp=dlogp, dentropy=dh, dlse=dl)
    step = 1e-5
    for t in range(3):
        for c in range(9):
            if np.isinf(x[t, c]):
                assert d[t, c] == 0
                continue
            a, b = x.copy(), x.copy()
            a[t, c] += step
            b[t, c] -= step
            assert abs((loss(a) - loss(b)) / (2 * step) - d[t, c]) < 1e-8


def test_logprob_limits():
    x = np.array([[-np.inf] * 4, [0.0] * 4, [-3.0e38] * 4, [5.0, -np.inf, 5.0, 4.0]])
    r = to.logprob(x, np.array([[1], [2], [3], [0]]), top=3)
    assert r["lse"][0] == -np.inf and r["logp"][0, 0] == -np.inf and r["entropy"][0] == 0
    assert np.allclose(r["logp"][1:3, 0], -np.log(4)) and np.allclose(r["entropy"][1:3], np.log(4))
    assert r["top_ids"].tolist() == [[-1, -1, -1], [0, 1, 2], [0, 1, 2], [0, 2, 3]]
    d, _ = to.logprob_grad(x, np.array([[1], [2], [3], [0]]), dlogp=np.ones((4, 1)))
    assert not d[0].any() and np.allclose(d[1:].sum(1), 0)


def test_checkpoint_format():
    """The scale is the least power of two that fits, the code the nearest integer."""
    g = RNG(3)
    x = g.standard_normal((50, 71)) * np.exp(8 * g.standard_normal((50, 1)))
    x[0], x[1, :32] = 0.0, 127.0
    x[2, :32], x[3, 0], x[4, 40] = np.nextafter(np.float32(127), np.float32(200)), np.inf, np.nan
    codes, b = to.ckpt_pack(x)
    v = to.ckpt_value(codes, b)
    assert b[0].tolist() == [1, 1, 1] and not codes[0].any()
    assert b[1, 0] == 127 and b[2, 0] == 128 and b[3, 0] == 255 and b[4, 1] == 255
    assert np.isnan(v[3, :32]).all() and np.isnan(v[4, 32:64]).all()
    fine = np.isfinite(v)
    unit = np.repeat(2.0 ** (b.astype(float) - 127), 32, 1)[:, :71]
    assert (np.abs(x - v)[fine] <= unit[fine] / 2).all()
    big = np.stack([np.abs(x[:, i:i + 32]).max(1) for i in (0, 32, 64)], 1)
    ok = (b > 1) & (b < 255)
    least = 2.0 ** (b[ok].astype(float) - 127)
    assert (127 * least >= big[ok]).all() and (127 * least / 2 < big[ok]).all()
