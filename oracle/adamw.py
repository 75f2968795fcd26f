"""AdamW reference: the step, its 8-bit state format and the gradient norm.
Test infrastructure: only the tests use the oracle.

AdamW is Loshchilov & Hutter's ("Decoupled Weight Decay Regularization"):
m' = b1 m + (1 - b1) g, v' = b2 v + (1 - b2) g^2, bias corrections 1 - b^t and
p' = p - lr wd p - lr m-hat / (sqrt(v-hat) + eps).  :func:`step` is that
formula in float64; :func:`moments` takes the moments' binary32 steps, whose
results the 8-bit states encode.

8-bit states: E4M3 codes of m and of sqrt(v) in blocks of 256 elements with a
scale 2**(floor(log2 amax) - 7), at least 2**-126, so that scaled magnitudes
lie below 256.  Codes go to the nearest value, ties to the even code, or
stochastically: with d the 20 fraction bits that binary32 has beyond E4M3's
three (of y + 2**-6 below 2**-6, where the grid is 2**-9), the code goes up iff
d + 16 h >= 2**20 for the 16-bit draw h.  Draws: element e takes word e & 3 of
the 32-bit layout (philox.words) with role 6, the low half for m and the high
half for sqrt(v).  A positive sqrt(v) never gets code 0.  A value that is not
finite gets the code of NaN and has no part in its block's scale.
"""

import numpy as np

from . import formats, philox

BLOCK = 256
ROLE_MOMENTS, ROLE_PARAM = 6, 7


def step(p, g, m, v, lr, b1, b2, eps, wd, t):
    """(p', m', v') in float64."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    mh, vh = m / (1 - b1 ** t), v / (1 - b2 ** t)
    return p - lr * wd * p - lr * mh / (np.sqrt(vh) + eps), m, v


def moments(g, m, v, b1, b2):
    """(m', v', sqrt(v')) in binary32, every operation rounded."""
    f = np.float32
    g, m, v = (np.asarray(a, f) for a in (g, m, v))
    m1 = f(b1) * m + f(1 - b1) * g
    v1 = f(b2) * v + (f(1 - b2) * g) * g
    return m1, v1, np.sqrt(v1)


def scales(x):
    """One power-of-two scale per block of 256 (the last may be short)."""
    n = len(x)
    a = np.abs(np.pad(np.asarray(x, np.float64), (0, -n % BLOCK))).reshape(-1, BLOCK).max(axis=1)
    _, e = np.frexp(a)                         # a = f 2**e, f in [0.5, 1)
    e = np.where(a > 0, e - 1 - 7, -126)
    return np.ldexp(1.0, np.maximum(e, -126)).astype(np.float32)


def _grid():
    return formats.e4m3_decode(np.arange(0x7F, dtype=np.uint8)).astype(np.float64)


def encode(x, h=None, positive=False):
    """(codes uint8, scales float32) of x, nearest or with 16-bit draws h."""
    x = np.asarray(x, np.float32)
    nan = ~np.isfinite(x)
    x = np.where(nan, np.float32(0), x)
    s = scales(x)
    y = np.abs(x).astype(np.float64) / np.repeat(s.astype(np.float64), BLOCK)[:len(x)]
    grid = _grid()
    if h is None:
        # binary32 rounds y + 2**-6 on its way to the subnormal grid
        y = np.where(y < 2.0 ** -6, (y + 2.0 ** -6).astype(np.float32).astype(np.float64) - 2.0 ** -6, y)
        lo = np.searchsorted(grid, y, side="right") - 1
        hi = np.minimum(lo + 1, len(grid) - 1)
        up, down = grid[hi] - y, y - grid[lo]
        c = np.where((up < down) | ((up == down) & (lo % 2 == 1)), hi, lo)
    else:
        z = np.where(y < 2.0 ** -6, y + 2.0 ** -6, y).astype(np.float32)
        lo = np.searchsorted(grid, z.astype(np.float64), side="right") - 1
        frac = (z.astype(np.float64) - grid[lo]) / (grid[lo + 1] - grid[lo])
        d = np.round(frac * 2 ** 20).astype(np.int64)         # exact: 20 bits
        c = lo + (d + 16 * np.asarray(h, np.int64) >= 2 ** 20)
        c = np.where(y < 2.0 ** -6, c - 8, c)
    c = np.where(nan, 0x7F, c).astype(np.uint8)
    if positive:
        return np.where((x != 0) & (c == 0), 1, c).astype(np.uint8), s
    return (c | np.where(x < 0, 0x80, 0)).astype(np.uint8), s


def decode(codes, s):
    """The binary32 values of codes with their blocks' scales."""
    codes = np.asarray(codes, np.uint8)
    nan = codes & 0x7F == 0x7F
    v = formats.e4m3_decode(np.where(nan, 0, codes & 0x7F)) * np.where(codes & 0x80, -1.0, 1.0)
    with np.errstate(invalid="ignore"):  # a scale that is not finite
        v = v * np.repeat(np.asarray(s, np.float64), BLOCK)[:len(codes)]
    return np.where(nan, np.nan, v).astype(np.float32)


def draws(n, seed, tag, t, role=ROLE_MOMENTS):
    """(low, high) halves of the n elements' 32-bit draws."""
    w = philox.words(np.arange(n, dtype=np.uint64), seed, philox.with_role(tag, role), t).astype(np.int64)
    return w & 0xFFFF, w >> 16


def norm(grads):
    return float(np.sqrt(sum((np.asarray(g, np.float64) ** 2).sum() for g in grads)))
