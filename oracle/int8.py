"""int8 reference: the quantiser with one scale per line and the product.
Test infrastructure: only the tests use the oracle.

The pages define no 8-bit integer format; the plainest symmetric reading is
taken.  With a the largest magnitude of a line (a row, or a column for the
quantised transpose), in binary32 steps (RN: to nearest):
  s = max(RN(a / 127), 2**-126), inv = RN(1 / s), y = RN(x inv),
  code = y to the nearest integer (ties to even), or floor(y) + [u < y -
  floor(y)] with the 16-bit Philox draw of the element's row-major position
  in the matrix (role 0), clamped to +-127.
numpy's float32 division and product are correctly rounded, and y - floor(y)
is taken in float32 as well (exact unless y is a tiny negative number, whose
difference to its floor rounds to one).
"""

import numpy as np

from . import philox

PITCH = 128


def quantize(x, axis=1, rounding="rne", seed=0, tag=0, step=0):
    """(codes int8 [outer, K], scales float32 [outer]) of matrix x with K along
    ``axis`` (1: rows; 0: columns, the codes are then the transpose)."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    amax = np.abs(x).max(axis=axis)
    scale = np.maximum(amax / np.float32(127), np.float32(2.0 ** -126)).astype(np.float32)
    inv = (np.float32(1) / scale).astype(np.float32)
    y = x * (inv[:, None] if axis else inv[None, :])
    if rounding == "sr":
        e = np.arange(rows * cols, dtype=np.uint64)
        u = philox.uniform_from_halves(philox.halves(e, seed, philox.with_role(tag, philox.ROLE_RESID), step))
        low = np.floor(y)
        c = low + (u.reshape(rows, cols) < (y - low))
    else:
        c = np.rint(y)
    c = np.clip(c, -127, 127).astype(np.int8)
    return (c if axis else np.ascontiguousarray(c.T)), scale


def dequantize(codes, scales):
    return codes.astype(np.float64) * np.asarray(scales, np.float64)[:, None]


def gemm(a, b):
    """C = A-hat B-hat^T of (codes, scales) pairs, in float64 (integer sums exact)."""
    c = a[0].astype(np.float64) @ b[0].astype(np.float64).T
    return c * np.asarray(a[1], np.float64)[:, None] * np.asarray(b[1], np.float64)[None, :]
