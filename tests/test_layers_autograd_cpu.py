"""Uses of the layers around the linear ones that they refuse before any GPU
work, so that nothing is left out in silence."""

import pytest
import torch
import torch.autograd.forward_ad as fwAD

from spectral_split_quantized_amd import metis
from spectral_split_quantized_amd.layer import Dropout, Embedding, LayerNorm, LinearCrossEntropy

N, C, V = 3, 4, 5


def _runs():
    ids = torch.tensor([0, 1, 2])
    ln, drop = LayerNorm(C, device="cpu"), Dropout(0.5, device="cpu")
    head, em = LinearCrossEntropy(C, V, device="cpu"), Embedding(V, C, device="cpu")
    return {"norm": ln, "dropout": drop, "residual": lambda x: drop(torch.zeros(N, C), x), "loss": lambda x: head(x, ids)}, em, ids


@pytest.mark.parametrize("name", ["norm", "dropout", "residual", "loss", "embedding"])
def test_forward_mode_is_refused(name):
    runs, em, ids = _runs()
    with fwAD.dual_level():
        if name == "embedding":
            from spectral_split_quantized_amd import layer
            dual = fwAD.make_dual(em.weight.detach(), torch.ones(V, C))
            run = lambda: layer._layers().embedding(dual, ids, 1.0, -1, -1)  # noqa: E731
        else:
            dual = fwAD.make_dual(torch.zeros(N, C), torch.ones(N, C))
            run = lambda: runs[name](dual)  # noqa: E731
        with pytest.raises(NotImplementedError, match="forward-mode"):
            run()


def test_forward_mode_of_a_parameter_is_refused():
    ln = LayerNorm(C, device="cpu")
    with fwAD.dual_level(), pytest.raises(NotImplementedError, match="forward-mode"):
        torch.func.functional_call(ln, {"bias": fwAD.make_dual(torch.zeros(C), torch.ones(C))}, torch.zeros(N, C))


@pytest.mark.parametrize("name", ["norm", "dropout", "residual", "loss", "embedding"])
def test_tracing_is_refused(name):
    """A trace would record the outputs' allocation and nothing that fills it."""
    from torch.fx.experimental.proxy_tensor import make_fx
    runs, em, ids = _runs()
    run, x = (em, ids) if name == "embedding" else (runs[name], torch.zeros(N, C))
    with torch.no_grad():
        with pytest.raises(NotImplementedError, match="traced"):
            torch.jit.trace(run, x)
        for mode in ("real", "fake"):
            with pytest.raises(NotImplementedError, match="traced"):
                make_fx(run, tracing_mode=mode)(x)


def test_bindings_refuse_negated_views():
    """They read memory, where such a view's values have the other sign."""
    x = torch.ones(N, C)
    neg, ids, vec = torch._neg_view(x), torch.tensor([0, 1, 2]), torch.ones(N)
    for call in (lambda: metis.layernorm(neg), lambda: metis.layernorm(x, torch._neg_view(torch.ones(C))), lambda: metis.dropout(neg, 0.5),
                 lambda: metis.dropout(x, 0.5, residual=neg), lambda: metis.embedding(neg, ids), lambda: metis.embedding_bwd(neg, ids, 5),
                 lambda: metis.cross_entropy(neg, x, ids), lambda: metis.cross_entropy(x, neg, ids),
                 lambda: metis.layernorm_bwd(x, x, torch._neg_view(vec), vec), lambda: metis.layernorm_bwd(neg, x, vec, vec),
                 lambda: metis.cross_entropy_bwd(x, x, ids, torch._neg_view(vec), vec),
                 lambda: metis.cross_entropy_bwd(x, x, ids, vec, torch._neg_view(vec)), lambda: metis.int8_quantize(neg, metis.AXIS0)):
        with pytest.raises(ValueError, match="negated"):
            call()


def test_captures_of_the_8_bit_layer_do_not_need_the_extension(monkeypatch):
    """Where _layers.so has not been built it has no living graphs either."""
    from spectral_split_quantized_amd import layer

    def missing():
        raise ImportError("_layers.so cannot be loaded")

    monkeypatch.setattr(layer, "_ext", None)
    monkeypatch.setattr(layer, "_layers", missing)
    w, other = torch.nn.Parameter(torch.ones(2)), torch.nn.Parameter(torch.ones(2))

    class Node:
        pass

    node, lin = Node(), layer.Int8Linear(C, C, device="cpu")
    layer._watch(node, lin, [w], capturing=False)
    layer._watch(Node(), None, [other], capturing=True)
    with pytest.raises(RuntimeError, match="alive"):
        layer._watch(Node(), None, [w], capturing=True)
    with pytest.raises(RuntimeError, match="alive"):
        layer._watch(Node(), lin, [other], capturing=True)


def test_a_captured_dropout_needs_its_step_on_the_gpu(monkeypatch):
    """A layer that was left on the CPU would give every replay the same mask."""
    from spectral_split_quantized_amd import layer
    drop = Dropout(0.5, device="cpu")
    monkeypatch.setattr(layer, "_capturing", lambda t: True)
    with pytest.raises(RuntimeError, match="move the layer"):
        drop(torch.zeros(N, C))
    assert drop.eval()(torch.zeros(N, C)).shape == (N, C)
