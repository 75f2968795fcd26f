"""Pins of the int8 oracle: hand-worked lines, both orientations, unbiased
stochastic rounding, and the product against a loop."""

import numpy as np
import pytest

from oracle import int8


def test_hand_worked_lines():
    x = np.array([[127.0, -63.5, 0.5, 1.5, 2.5, -0.5, 0.0, -126.6],
                  [0.0] * 8,
                  [1e-44] + [0.0] * 7])
    c, s = int8.quantize(x)
    assert s[0] == 1.0 and s[1] == s[2] == np.float32(2.0 ** -126)
    assert c[0].tolist() == [127, -64, 0, 2, 2, 0, 0, -127]  # ties to even
    assert not c[1].any() and not c[2].any()  # 1e-44 is far below half of 2^-126


def test_orientations_and_bounds():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((37, 53)).astype(np.float32)
    for axis in (0, 1):
        c, s = int8.quantize(x, axis)
        ref = x if axis else x.T
        assert c.shape == ref.shape and np.abs(c).max() == 127
        # half a step of the line's grid, plus the binary32 roundings of s, inv and y
        assert np.all(np.abs(int8.dequantize(c, s) - ref) <= (0.5 + 127 * 4 * 2.0 ** -24) * s[:, None])


def test_stochastic_rounding_is_unbiased():
    x = np.full((200, 1000), 0.3, np.float32)
    x[:, 0] = 127.0  # scale 1
    c, s = int8.quantize(x, rounding="sr", seed=9, tag=0x3000, step=4)
    mean = c[:, 1:].mean()
    n = 200 * 999
    assert abs(mean - 0.3) < 5 * np.sqrt(0.3 * 0.7 / n)
    assert set(np.unique(c[:, 1:])) == {0, 1}


@pytest.mark.parametrize("k", [1, 5, 130])
def test_product_against_a_loop(k):
    rng = np.random.default_rng(k)
    a, b = (int8.quantize(rng.standard_normal((n, k))) for n in (3, 4))
    got = int8.gemm(a, b)
    for i in range(3):
        for j in range(4):
            acc = sum(int(a[0][i, t]) * int(b[0][j, t]) for t in range(k))
            assert got[i, j] == pytest.approx(acc * float(a[1][i]) * float(b[1][j]), rel=1e-15)
