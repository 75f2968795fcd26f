"""Pins of the AdamW oracle: a hand-worked step, the 8-bit format's grid,
ties, scales and draws, and the binary32 moments against the formula."""

import numpy as np
import pytest

from oracle import adamw


def test_first_step_by_hand():
    # m-hat = g, v-hat = g^2: the first step is lr sign(g) away from the decayed p
    p, m, v = adamw.step([2.0], [0.5], [0.0], [0.0], 0.1, 0.9, 0.999, 0.0, 0.01, 1)
    assert p[0] == pytest.approx(2.0 - 0.1 * 0.01 * 2.0 - 0.1, rel=1e-12)
    assert m[0] == pytest.approx(0.05) and v[0] == pytest.approx(0.00025)


def test_moments_follow_the_formula():
    rng = np.random.default_rng(1)
    g, m = rng.standard_normal((2, 1000)).astype(np.float32)
    v = rng.random(1000).astype(np.float32)
    m1, v1, r1 = adamw.moments(g, m, v, 0.9, 0.999)
    _, m2, v2 = adamw.step(g, g, m, v, 0, 0.9, 0.999, 1, 0, 1)
    # three roundings of terms no larger than |0.9 m| + |0.1 g|
    assert np.all(np.abs(m1 - m2) <= 4 * 2.0 ** -24 * (0.9 * np.abs(m) + 0.1 * np.abs(g)))
    assert np.all(np.abs(v1 - v2) <= 6 * 2.0 ** -24 * v2)
    assert np.allclose(r1, np.sqrt(v2), rtol=4e-7)


def test_scale_and_grid():
    x = np.zeros(600, np.float32)
    x[:8] = [1.0, -0.999, 0.5, 1 / 16, 2.0 ** -13, 2.0 ** -16, 2.0 ** -17.5, 2.0 ** -30]
    x[300] = 1e-45
    codes, s = adamw.encode(x)
    assert s.tolist() == [2.0 ** -7, np.float32(2.0 ** -126), np.float32(2.0 ** -126)]
    d = adamw.decode(codes, s)
    # 1 = 128 units exactly; -0.999 -> -1 (spacing 8 units below 128); powers of two exact down to
    # 2^-9 units = 2^-16; 2^-17.5 is less than half of that
    assert d[:8].tolist() == [1.0, -1.0, 0.5, 1 / 16, 2.0 ** -13, 2.0 ** -16, 0.0, 0.0]
    pos, _ = adamw.encode(np.abs(x), positive=True)
    assert pos[6] == pos[7] == 1 and pos[8] == 0 and pos[300] == 1


def test_nearest_is_exhaustively_nearest():
    rng = np.random.default_rng(2)
    x = np.exp(rng.uniform(-12, 0, 256 * 40)).astype(np.float32)
    codes, s = adamw.encode(x)
    d = adamw.decode(codes, s).astype(np.float64)
    grid = adamw._grid()[None, :] * np.repeat(s.astype(np.float64), 256)[:, None]
    best = np.abs(grid - x.astype(np.float64)[:, None]).min(axis=1)
    unit = np.repeat(s.astype(np.float64), 256)
    assert np.all(np.abs(d - x) <= best + unit * 2.0 ** -29)


def test_stochastic_codes_are_unbiased_and_adjacent():
    n = 256 * 400
    x = np.full(n, 0.7, np.float32)
    x[::256] = 1.0
    lo, hi = adamw.draws(n, 3, 0x1000, 17)
    assert 0.49 < lo.mean() / 65536 < 0.51 and 0.49 < hi.mean() / 65536 < 0.51
    assert abs(np.corrcoef(lo, hi)[0, 1]) < 0.02
    for h in (lo, hi):
        codes, s = adamw.encode(x, h)
        d = adamw.decode(codes, s)
        inner = d[x < 1]
        assert set(np.unique(inner).tolist()) == {0.6875, 0.75}
        assert abs(inner.mean() - 0.7) < 5 * 0.0625 * 0.5 / np.sqrt(n)
    # subnormal codes too: 2.5 units of the smallest step
    x[x < 1] = 2.5 * 2.0 ** -16
    codes, s = adamw.encode(x, lo)
    inner = adamw.decode(codes, s)[x < 1]
    assert set(np.unique(inner).tolist()) == {2 * 2.0 ** -16, 3 * 2.0 ** -16}


def test_norm():
    assert adamw.norm([[3.0], [], [[0.0, 4.0]]]) == 5.0
