"""References of what stands around the linear layers: layer norm, dropout, the
embedding and the loss over a vocabulary.  Test infrastructure: only the tests
use the oracle.

The pages train language models and say nothing of these parts, so the
textbook formulas are taken, in float64.  Dropout is defined to the last bit:
element e of a matrix (its row-major position) takes the 16-bit Philox draw
h(e) of role 8, is dropped where h < t with t = rint(65536 p), and otherwise
becomes x * RN32(65536 / (65536 - t)) in binary32, to which the residual is
added in binary32.
"""

import numpy as np

from . import philox

ROLE_DROPOUT = 8


def layernorm(x, w, b, eps):
    """(y, mean, 1 / sd) of the rows of x."""
    mu = x.mean(axis=1, keepdims=True)
    r = 1.0 / np.sqrt(((x - mu) ** 2).mean(axis=1, keepdims=True) + eps)
    return (x - mu) * r * w + b, mu[:, 0], r[:, 0]


def layernorm_bwd(dy, x, w, eps):
    """(dx, dw, db)."""
    _, mu, r = layernorm(x, 1.0, 0.0, eps)
    h = (x - mu[:, None]) * r[:, None]
    g = dy * w
    dx = r[:, None] * (g - g.mean(axis=1, keepdims=True) - h * (g * h).mean(axis=1, keepdims=True))
    return dx, (dy * h).sum(axis=0), dy.sum(axis=0)


def dropout_keep(shape, p, seed, tag, step):
    """(kept, scale): which elements stay, and the binary32 factor of those."""
    t = int(np.rint(65536.0 * p))
    e = np.arange(int(np.prod(shape)), dtype=np.uint64)
    h = philox.halves(e, seed, philox.with_role(tag, ROLE_DROPOUT), step)
    scale = np.float32(65536.0 / (65536 - t)) if t < 65536 else np.float32(0)
    return (np.asarray(h).astype(np.int64) >= t).reshape(shape), scale


def dropout(x, p, seed, tag, step, residual=None):
    """float32 matrix (before the rounding to another type)."""
    kept, scale = dropout_keep(x.shape, p, seed, tag, step)
    with np.errstate(over="ignore", invalid="ignore"):
        y = np.where(kept, np.asarray(x, np.float32) * scale, np.float32(0))
        return y if residual is None else y + np.asarray(residual, np.float32)


def embedding_bwd(dy, ids, vocab, padding, scale):
    dw = np.zeros((vocab, dy.shape[1]))
    use = (ids >= 0) & (ids < vocab) & (ids != (-1 if padding is None else padding))
    np.add.at(dw, ids[use], dy[use])
    return dw * scale


def cross_entropy(x, w, targets, ignore):
    """(losses, lse, P for a gradient of 1 of each loss): P = softmax - onehot,
    zero rows where a token has no target."""
    use = (targets != ignore) & (targets >= 0) & (targets < w.shape[0])
    z = np.where(use[:, None], x, 0.0) @ w.T
    top = z.max(axis=1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(axis=1))
    at = np.where(use, targets, 0)
    rows = np.arange(len(targets))
    losses = np.where(use, lse - z[rows, at], 0.0)
    p = np.exp(z - lse[:, None])
    p[rows, at] -= 1.0
    return losses, lse, p * use[:, None]
