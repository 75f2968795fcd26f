"""Pins of the oracle's formulas around the linear layers: gradients against
differences, hand-worked values, the dropout's rate."""

import numpy as np

from oracle import model


def _difference(f, x, d, h=1e-5):
    """Central difference of f along direction d: error about h^2 times the
    third derivative and 2^-53 |f| / h, both far below the tolerances here."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_layernorm_by_hand():
    y, mu, r = model.layernorm(np.array([[1.0, 3.0, 5.0, 7.0]]), np.array([1.0, 2.0, 1.0, 1.0]), np.array([0.0, 1.0, 0.0, 0.0]), 0.0)
    s = 5 ** 0.5
    assert mu[0] == 4.0 and np.isclose(r[0], 1 / s)
    assert np.allclose(y, [[-3 / s, 1 - 2 / s, 1 / s, 3 / s]])


def test_layernorm_gradients_are_those_of_differences():
    g = np.random.default_rng(0)
    x, dy, w, b = g.normal(size=(5, 7)), g.normal(size=(5, 7)), g.normal(size=7), g.normal(size=7)
    dx, dw, db = model.layernorm_bwd(dy, x, w, 1e-3)
    out = lambda x, w, b: (model.layernorm(x, w, b, 1e-3)[0] * dy).sum()  # noqa: E731
    for _ in range(4):
        d, e = g.normal(size=x.shape), g.normal(size=7)
        assert np.isclose(_difference(lambda v: out(v, w, b), x, d), (dx * d).sum(), rtol=1e-7, atol=1e-8)
        assert np.isclose(_difference(lambda v: out(x, v, b), w, e), (dw * e).sum(), rtol=1e-7, atol=1e-8)
        assert np.isclose(_difference(lambda v: out(x, w, v), b, e), (db * e).sum(), rtol=1e-7, atol=1e-8)


def test_cross_entropy_gradient_is_that_of_differences():
    g = np.random.default_rng(1)
    x, w, t = g.normal(size=(6, 4)), g.normal(size=(9, 4)), np.array([0, 8, -100, 3, 9, -1])
    losses, lse, p = model.cross_entropy(x, w, t, -100)
    assert (losses[[2, 4, 5]] == 0).all() and (p[[2, 4, 5]] == 0).all()  # left out: ignored, and not words
    up = g.normal(size=6)
    total = lambda x, w: (model.cross_entropy(x, w, t, -100)[0] * up).sum()  # noqa: E731
    dz = p * up[:, None]
    for _ in range(4):
        d, e = g.normal(size=x.shape), g.normal(size=w.shape)
        assert np.isclose(_difference(lambda v: total(v, w), x, d), (dz @ w * d).sum(), rtol=1e-7, atol=1e-8)
        assert np.isclose(_difference(lambda v: total(x, v), w, e), (dz.T @ x * e).sum(), rtol=1e-7, atol=1e-8)


def test_cross_entropy_by_hand():
    losses, lse, p = model.cross_entropy(np.array([[1.0]]), np.log(np.array([[1.0], [3.0]])), np.array([1]), -100)
    assert np.isclose(lse[0], np.log(4)) and np.isclose(losses[0], np.log(4 / 3)) and np.allclose(p, [[0.25, -0.25]])


def test_embedding_gradient():
    dy = np.arange(8.0).reshape(4, 2)
    dw = model.embedding_bwd(dy, np.array([2, 0, 2, 7]), 4, None, 0.5)
    assert np.allclose(dw, [[1, 1.5], [0, 0], [2, 3], [0, 0]])
    assert (model.embedding_bwd(dy, np.array([2, 0, 2, 7]), 4, 2, 0.5)[2] == 0).all()


def test_dropout_rate_scale_and_streams():
    for p in (0.1, 0.5, 0.73):
        kept, scale = model.dropout_keep((400, 333), p, 3, 9 << 16, 4)
        n, q = kept.size, round(65536 * p) / 65536
        # six standard deviations of n draws
        assert abs((~kept).mean() - q) < 6 * (q * (1 - q) / n) ** 0.5
        assert abs(float(scale) * (1 - q) - 1) <= 2 ** -24
    a, b = (model.dropout_keep((64, 64), 0.5, 3, tag, 4)[0] for tag in (1 << 16, 2 << 16))
    assert (a != b).any() and (a != model.dropout_keep((64, 64), 0.5, 3, 1 << 16, 5)[0]).any()
    x = np.full((3, 5), np.nan, np.float32)
    assert (model.dropout(x, 1.0, 0, 0, 0) == 0).all()
    assert np.isnan(model.dropout(x, 0.0, 0, 0, 0)).all()
