"""Host-side checks of the entry points around the linear layers (no GPU work):
argument errors are synchronous, sizes are right, layers refuse bad operands."""

import copy
import ctypes
import pickle

import pytest
import torch

from spectral_split_quantized_amd import metis
from spectral_split_quantized_amd.layer import Dropout, Embedding, LayerNorm, LinearCrossEntropy, set_step

D = 4096            # aligned stand-in, never dereferenced
ODD = 4097
BIG = 1 << 40


def _norm(X=D, xt=0, rows=8, cols=16, ldx=16, w=D, b=D, wt=1, eps=1e-5, Y=D, yt=0, ldy=16, mean=D, rstd=D):
    return metis.load().metis_layernorm_fwd(X, xt, rows, cols, ldx, w, b, wt, eps, Y, yt, ldy, mean, rstd, None)


def test_layernorm_argument_errors():
    for bad in (dict(X=None), dict(Y=None), dict(xt=2), dict(yt=-1), dict(wt=3), dict(rows=-1), dict(cols=0), dict(ldx=15),
                dict(ldy=15), dict(cols=1 << 31, ldx=1 << 31, ldy=1 << 31), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(mean=None), dict(rstd=None), dict(mean=D + 2), dict(X=ODD), dict(Y=ODD), dict(w=D + 2),
                dict(b=D + 2)):
        assert _norm(**bad) == metis.E_INVALID, bad
    assert _norm(rows=0, X=None, Y=None) == metis.OK


def _norm_bwd(dY=D, yt=0, lddy=16, X=D, xt=0, rows=8, cols=16, ldx=16, w=D, wt=1, mean=D, rstd=D, dX=D, lddx=16, dw=D, db=D, ws=D,
              n=BIG):
    return metis.load().metis_layernorm_bwd(dY, yt, lddy, X, xt, rows, cols, ldx, w, wt, mean, rstd, dX, lddx, dw, db, ws, n, None)


def test_layernorm_bwd_argument_errors():
    for bad in (dict(dY=None), dict(X=None), dict(xt=2), dict(yt=2), dict(wt=2), dict(cols=0), dict(lddy=15), dict(ldx=15),
                dict(lddx=15), dict(mean=None), dict(rstd=None), dict(dw=D + 2), dict(db=D + 2), dict(ws=D + 16), dict(dX=ODD)):
        assert _norm_bwd(**bad) == metis.E_INVALID, bad
    assert _norm_bwd(n=16) == metis.E_WORKSPACE and _norm_bwd(ws=None) == metis.E_WORKSPACE
    assert _norm_bwd(dX=None, dw=None, db=None, ws=None, n=0) == metis.OK  # nothing wanted
    size = metis.load().metis_layernorm_bwd_workspace
    assert size(0, 4) == 256 and size(1, 1) >= 8
    for rows, cols in ((1, 7), (16384, 768), (3, 4096), (100000, 20000), (1 << 30, 1 << 20)):
        assert size(rows, cols) >= 8 * cols


def _drop(X=D, dt=0, rows=8, cols=16, ldx=16, res=None, ldr=0, p=0.1, step=0, count=None, Y=D, ldy=16):
    return metis.load().metis_dropout(X, dt, rows, cols, ldx, res, ldr, p, 0, 0, step, count, Y, ldy, None)


def test_dropout_argument_errors():
    for bad in (dict(X=None), dict(Y=None), dict(dt=2), dict(rows=-1), dict(cols=0), dict(ldx=15), dict(ldy=15), dict(res=D, ldr=15),
                dict(res=ODD, ldr=16), dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(step=-1), dict(count=D + 4)):
        assert _drop(**bad) == metis.E_INVALID, bad
    assert _drop(rows=1 << 40, cols=1 << 30, ldx=1 << 30, ldy=1 << 30) == metis.E_UNSUPPORTED
    assert _drop(rows=0, X=None, Y=None) == metis.OK


def _embed(W=D, wt=0, vocab=10, cols=16, ldw=16, ids=D, bits=64, tokens=4, Y=D, yt=0, ldy=16):
    return metis.load().metis_embedding_fwd(W, wt, vocab, cols, ldw, ids, bits, tokens, 1.0, Y, yt, ldy, None)


def _embed_bwd(dY=D, yt=0, tokens=4, cols=16, lddy=16, ids=D, bits=64, vocab=10, padding=-1, dW=D, wt=0, lddw=16, ws=D, n=BIG):
    return metis.load().metis_embedding_bwd(dY, yt, tokens, cols, lddy, ids, bits, vocab, padding, 1.0, dW, wt, lddw, ws, n, None)


def test_embedding_argument_errors():
    for bad in (dict(W=None), dict(Y=None), dict(ids=None), dict(wt=2), dict(yt=2), dict(bits=16), dict(vocab=0), dict(cols=0),
                dict(tokens=-1), dict(ldw=15), dict(ldy=15), dict(ids=D + 4), dict(W=ODD)):
        assert _embed(**bad) == metis.E_INVALID, bad
    assert _embed(vocab=1 << 31) == metis.E_UNSUPPORTED and _embed(tokens=1 << 31) == metis.E_UNSUPPORTED
    assert _embed(tokens=0, ids=None, Y=None) == metis.OK
    for bad in (dict(dY=None), dict(dW=None), dict(ids=None), dict(yt=2), dict(wt=2), dict(bits=8), dict(vocab=0), dict(padding=10),
                dict(lddy=15), dict(lddw=15), dict(ws=D + 128)):
        assert _embed_bwd(**bad) == metis.E_INVALID, bad
    assert _embed_bwd(n=16) == metis.E_WORKSPACE and _embed_bwd(ws=None) == metis.E_WORKSPACE
    size = metis.load().metis_embedding_bwd_workspace
    assert size(0, 8) == 256
    for tokens, cols in ((1, 1), (17, 5), (16384, 4096), (1 << 20, 64)):
        assert size(tokens, cols) >= 16 * tokens + (tokens + 15) // 16 * 8 * cols


def _loss(**over):
    f = dict(x=D, w=D, targets=D, tokens=8, vocab=10, cols=64, ldx=64, ldw=64, ignore_index=-100, x_dtype=0, w_dtype=0, target_bits=64)
    f.update(over)
    return metis._Loss(**f)


def _ce(l, losses=D, lse=D, mean=1, total=D, ws=D, n=BIG):
    return metis.load().metis_cross_entropy_fwd(ctypes.byref(l), losses, lse, mean, total, ws, n, None)


def _ce_bwd(l, lse=D, grad=D, each=0, count=None, dX=D, lddx=64, dW=D, lddw=64, ws=D, n=BIG):
    return metis.load().metis_cross_entropy_bwd(ctypes.byref(l), lse, grad, each, count, dX, lddx, dW, lddw, ws, n, None)


def test_cross_entropy_argument_errors():
    lib = metis.load()
    assert lib.metis_cross_entropy_fwd(None, D, D, 1, D, D, BIG, None) == metis.E_INVALID
    for bad in (dict(x=None), dict(w=None), dict(targets=None), dict(vocab=0), dict(cols=0), dict(tokens=-1), dict(ldx=63),
                dict(ldw=63), dict(x_dtype=2), dict(w_dtype=2), dict(target_bits=8), dict(targets=D + 4), dict(x=ODD), dict(w=ODD)):
        assert _ce(_loss(**bad)) == metis.E_INVALID and _ce_bwd(_loss(**bad)) == metis.E_INVALID, bad
    for bad in (dict(tokens=(1 << 22) + 1), dict(cols=(1 << 22) + 1, ldx=(1 << 22) + 1, ldw=(1 << 22) + 1), dict(vocab=1 << 31)):
        assert _ce(_loss(**bad)) == metis.E_UNSUPPORTED and _ce_bwd(_loss(**bad)) == metis.E_UNSUPPORTED, bad
    for bad in (dict(lse=None), dict(lse=D + 2), dict(losses=D + 2), dict(total=D + 2), dict(mean=2), dict(ws=D + 16)):
        assert _ce(_loss(), **bad) == metis.E_INVALID, bad
    for bad in (dict(lse=None), dict(grad=None), dict(grad=D + 2), dict(count=D + 2), dict(each=2), dict(lddx=63), dict(lddw=63),
                dict(dX=ODD), dict(dW=ODD), dict(ws=D + 16)):
        assert _ce_bwd(_loss(), **bad) == metis.E_INVALID, bad
    assert _ce(_loss(), n=16) == metis.E_WORKSPACE and _ce(_loss(), ws=None) == metis.E_WORKSPACE
    assert _ce_bwd(_loss(), n=16) == metis.E_WORKSPACE and _ce_bwd(_loss(), ws=None) == metis.E_WORKSPACE
    assert _ce(_loss(tokens=0, x=None, targets=None), lse=None, losses=None, total=None, ws=None, n=0) == metis.OK
    assert _ce_bwd(_loss(), dX=None, dW=None, ws=None, n=0) == metis.OK


def test_cross_entropy_workspace_does_not_grow_with_the_vocabulary():
    size = lambda backward, **f: metis.load().metis_cross_entropy_workspace(ctypes.byref(_loss(**f)), backward)  # noqa: E731
    big = dict(tokens=8192, cols=4096, ldx=4096, ldw=4096)
    at = [size(1, vocab=v, **big) for v in (1 << 17, 1 << 20, 1 << 30)]
    assert max(at) <= 1.1 * min(at)
    assert at[0] < 8192 * (1 << 17) * 4  # the logits in binary32
    for tokens in (1, 63, 64, 1000):
        for dtype in (0, 1):
            for vocab in (1, 255, 50257):
                for cols in (1, 64, 769):
                    f = dict(tokens=tokens, vocab=vocab, cols=cols, ldx=cols, ldw=cols, x_dtype=dtype, w_dtype=dtype)
                    assert size(0, **f) >= 256 and size(1, **f) >= tokens * cols * 4


def test_layers_refuse_what_they_cannot_hold():
    with pytest.raises(ValueError):
        LayerNorm(8, weight=torch.ones(7), device="cpu")
    with pytest.raises(ValueError):
        LayerNorm(8, weight=torch.ones(8), bias=torch.zeros(8, dtype=torch.bfloat16), device="cpu")
    with pytest.raises(ValueError):
        LayerNorm(8, affine=False, bias=torch.zeros(8), device="cpu")
    with pytest.raises(ValueError):
        LayerNorm(8, device="cpu")(torch.zeros(3, 7))
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises(ValueError):
            Dropout(p, device="cpu")
    drop = Dropout(0.5, device="cpu")
    with pytest.raises(ValueError):
        drop(torch.zeros(2, 3), torch.zeros(3, 2))
    with pytest.raises(ValueError):
        drop(torch.zeros(2, 3), torch.zeros(2, 3, dtype=torch.bfloat16))
    for pad in (-1, 10):
        with pytest.raises(ValueError):
            Embedding(10, 4, padding_idx=pad, device="cpu")
    with pytest.raises(ValueError):
        Embedding(10, 4, weight=torch.zeros(4, 10), device="cpu")
    with pytest.raises(ValueError):
        LinearCrossEntropy(4, 10, reduction="max", device="cpu")
    head = LinearCrossEntropy(4, 10, device="cpu")
    with pytest.raises(ValueError):
        head(torch.zeros(2, 5), torch.zeros(2, dtype=torch.long))
    with pytest.raises(ValueError):
        head(torch.zeros(2, 4), torch.zeros(3, dtype=torch.long))


def test_bindings_refuse_other_types_and_layouts():
    x = torch.zeros(4, 8)
    for bad in (x.half(), x.t(), x.double(), x[:, ::2]):
        with pytest.raises((ValueError, TypeError)):
            metis.layernorm(bad)
        with pytest.raises((ValueError, TypeError)):
            metis.dropout(bad, 0.1)
        with pytest.raises((ValueError, TypeError)):
            metis.embedding(bad, torch.zeros(2, dtype=torch.long))
    with pytest.raises(ValueError):
        metis.layernorm(x, torch.ones(8), torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        metis.embedding(x, torch.zeros(2, dtype=torch.int16))
    with pytest.raises(ValueError):
        metis.embedding_bwd(x, torch.zeros(3, dtype=torch.long), 5)
    with pytest.raises(ValueError):
        metis.cross_entropy(x, torch.zeros(5, 8), torch.zeros(3, dtype=torch.long))
    with pytest.raises(ValueError):
        metis.cross_entropy(x, torch.zeros(5, 7), torch.zeros(4, dtype=torch.long))
    with pytest.raises(ValueError):  # no CPU path
        metis.layernorm(x)
    with pytest.raises(ValueError):
        metis.dropout(x, 0.1)
    with pytest.raises(ValueError):
        metis.dropout(x, 0.1, step_count=torch.zeros(1))


def test_dropout_without_effect_and_its_step():
    drop = Dropout(0.0, device="cpu")
    x, r = torch.randn(3, 4), torch.randn(3, 4)
    assert drop(x) is x and torch.equal(drop(x, r), x + r)
    drop = Dropout(0.5, seed=7, layer=2, device="cpu").eval()
    assert drop(x) is x
    model = torch.nn.Sequential(drop, LayerNorm(4, device="cpu"))
    set_step(model, 12)
    assert drop.step == 12
    for other in (copy.deepcopy(drop), pickle.loads(pickle.dumps(drop))):
        assert other.step == 12 and other.p == 0.5 and other.tag == drop.tag


def test_weights_can_be_shared():
    e = Embedding(10, 4, device="cpu")
    head = LinearCrossEntropy(4, 10, weight=e.weight, device="cpu")
    assert head.weight is e.weight
    assert set(dict(LayerNorm(4, device="cpu").named_parameters())) == {"weight", "bias"}
    assert not list(LayerNorm(4, affine=False, device="cpu").parameters())


def test_cross_entropy_workspace_over_tokens_and_types():
    """A piece's probabilities and its part of the weight are bounded, for few tokens and for many, in either type."""
    up = lambda n: (n + 63) // 64 * 64  # noqa: E731
    for tokens in (1, 64, 8192, 1 << 17, 1 << 20):
        for cols in (64, 769, 4096, 1 << 20):
            for xt, wt in ((0, 0), (1, 1), (0, 1), (1, 0)):
                f = dict(tokens=tokens, cols=cols, ldx=cols, ldw=cols, x_dtype=xt, w_dtype=wt)
                size = lambda backward, vocab: metis.load().metis_cross_entropy_workspace(ctypes.byref(_loss(vocab=vocab, **f)), backward)  # noqa: E731
                both = 2 if xt or wt else 1
                rows = up(tokens) * up(cols)
                x, w, p = 2 * (xt + 1) * rows, 2 * (wt + 1) * max(1 << 29, 256 * up(cols)), 2 * both * max(1 << 28, 4096 * up(tokens))
                dx = 0 if xt else 4 * tokens * cols
                at = [size(1, v) for v in (1 << 20, 1 << 23, (1 << 31) - 1)]
                x2 = 2 * x  # as it is, and weighed by the tokens' gradients
                # sums in parts of K: 32 at most, few where whole sums fill the chip
                part = 4 * tokens * cols * (32 if tokens * cols < 1 << 25 else 8)
                assert max(at) <= 1.02 * (x2 + w + p + dx + part) + (1 << 20), (f, at)
                # forward: planes of x, of a piece of w, and the statistics, 8 bytes for 64 words
                assert size(0, 1 << 23) <= x + w + ((1 << 23) // 64 * 8 + 8) * tokens + (1 << 20), f


def test_embedding_gradient_of_too_many_tokens_is_refused_before_any_work():
    limit = (1 << 28) - (1 << 18)
    assert _embed_bwd(tokens=limit, cols=1, lddy=1, lddw=1, n=1 << 60) == metis.E_UNSUPPORTED
    assert _embed_bwd(tokens=limit, cols=1, lddy=1, lddw=1, n=16) == metis.E_UNSUPPORTED
    assert _embed_bwd(tokens=limit - 1, cols=1, lddy=1, lddw=1, n=16) == metis.E_WORKSPACE
