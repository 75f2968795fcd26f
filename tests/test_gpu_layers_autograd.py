"""What autograd asks of the layers around the linear ones beyond a plain
backward pass."""

import pytest
import torch
import torch.autograd.forward_ad as fwAD

from spectral_split_quantized_amd import metis
from spectral_split_quantized_amd.layer import Dropout, Embedding, LayerNorm, LinearCrossEntropy, MetisLinear, set_step

from gpu_helpers import say

pytestmark = pytest.mark.gpu

N, C, V = 20, 64, 51


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X; none is visible")
    metis.load()
    torch.cuda.set_device(0)
    metis.init_device()


def _layers(seed=0):
    """(name, call of one tensor, that tensor) of each layer; the embedding's is its weight."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N, C, generator=g, device="cuda", requires_grad=True)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda")
    ln, em, head, drop = LayerNorm(C), Embedding(V, C), LinearCrossEntropy(C, V, reduction="none"), Dropout(0.5)
    set_step(drop, 0)
    return [("norm", ln, x), ("dropout", drop, x), ("embedding", lambda w: em(ids), em.weight), ("loss", lambda q: head(q, ids), x)]


def test_a_sparse_gradient_is_taken():
    """Autograd lets a sparse gradient of a strided output through."""
    for name, run, leaf in _layers():
        if name == "loss":
            continue  # (its output has no second dimension to gather from)
        say("sparse gradient: %s" % name)
        at = torch.arange(N, device="cuda")[:, None] % C
        got = torch.autograd.grad(torch.gather(run(leaf), 1, at, sparse_grad=True).sum(), leaf)[0]
        want = torch.autograd.grad(torch.gather(run(leaf), 1, at).sum(), leaf)[0]
        assert torch.equal(got, want)
        rows = torch.tensor([3, 0, 3], device="cuda")
        got = torch.autograd.grad(torch.nn.functional.embedding(rows, run(leaf), sparse=True).square().sum(), leaf)[0]
        want = torch.autograd.grad(torch.nn.functional.embedding(rows, run(leaf)).square().sum(), leaf)[0]
        assert torch.equal(got, want)  # (no row is named more than twice, and two values have one sum)
    metis.status_sync()


@pytest.mark.parametrize("name", ["norm", "loss"])
def test_second_derivatives_raise_whatever_the_gradient_from_above(name):
    """The gradients of a norm and of the loss depend on the inputs: a penalty
    on them is not left out in silence where the gradient from above is a
    constant."""
    say("second derivatives: %s" % name)
    run, leaf = {n: (r, x) for n, r, x in _layers()}[name]
    want = torch.autograd.grad(run(leaf).sum(), leaf)[0]
    y = run(leaf)
    (first,) = torch.autograd.grad(y.sum(), leaf, create_graph=True)
    assert torch.equal(first, want)
    with pytest.raises(RuntimeError, match="differentiate"):
        (y.sum() + first.square().sum()).backward()
    with pytest.raises(RuntimeError, match="differentiate"):
        torch.autograd.grad(first.sum(), leaf)
    leaf.grad = None
    run(leaf).sum().backward(create_graph=True)  # a graph that is not used is no error
    assert torch.equal(leaf.grad.detach(), want)
    leaf.grad = None


@pytest.mark.parametrize("name", ["dropout", "embedding"])
def test_gradients_that_depend_on_the_one_from_above_alone(name):
    """Those of dropout and of the embedding are linear: with a constant from
    above they are constants."""
    say("first derivatives with a graph: %s" % name)
    run, leaf = {n: (r, x) for n, r, x in _layers()}[name]
    (first,) = torch.autograd.grad(run(leaf).sum(), leaf, create_graph=True)
    assert not first.requires_grad and torch.equal(first, torch.autograd.grad(run(leaf).sum(), leaf)[0])
    up = torch.ones_like(run(leaf)).requires_grad_(True)
    (first,) = torch.autograd.grad(run(leaf), leaf, up, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate"):
        first.sum().backward()


def test_forward_mode_through_a_backward_pass_raises():
    for name, run, leaf in _layers():
        say("forward mode in a backward pass: %s" % name)
        y = run(leaf)
        with fwAD.dual_level():
            up = fwAD.make_dual(torch.ones_like(y), torch.ones_like(y))
            with pytest.raises(RuntimeError, match="forward-mode"):
                torch.autograd.grad(y, leaf, up)


@pytest.mark.filterwarnings("ignore:Dynamo")
@pytest.mark.parametrize("backend", ["eager", "aot_eager"])
def test_compiled_callers_break_the_graph_and_are_right(backend):
    """torch.compile leaves the layers' calls out of its graphs."""
    torch._dynamo.reset()
    for name, run, leaf in _layers():
        say("compiled caller: %s, %s" % (name, backend))
        leaf.grad = None
        want = run(leaf) * 2
        want.sum().backward()
        grad, leaf.grad = leaf.grad, None
        got = torch.compile(lambda q: run(q) * 2, backend=backend)(leaf)
        got.sum().backward()
        assert torch.equal(got, want) and torch.equal(leaf.grad, grad)


def test_a_backward_pass_cannot_be_recorded():
    from torch.fx.experimental.proxy_tensor import make_fx
    for name, run, leaf in _layers():
        say("recording a backward pass: %s" % name)
        y = run(leaf)
        with pytest.raises(Exception, match="traced"):
            make_fx(lambda up: torch.autograd.grad(y, leaf, up)[0])(torch.ones_like(y))


def _negated(t):
    """-t as a view that is negated when it is read, and contiguous as it lies."""
    v = torch._neg_view(t)
    assert v.is_neg() and v.is_contiguous()
    return v


def test_negated_views_are_taken_with_their_sign():
    """Of inputs, parameters and gradients."""
    g = torch.Generator(device="cuda").manual_seed(3)
    up = torch.randn(N, C, generator=g, device="cuda")
    for name, run, leaf in _layers():
        say("negated views: %s" % name)
        with torch.no_grad():
            want = run(-leaf) if name != "embedding" else -run(leaf)
            head = LinearCrossEntropy(C, V, weight=torch.nn.Parameter(_negated(leaf.detach()))) if name == "embedding" else None
        if head is None:
            assert torch.equal(run(_negated(leaf)), want)
            (got,) = torch.autograd.grad(run(_negated(leaf)).sum(), leaf)
            q = -leaf.detach()
            assert torch.equal(got, -torch.autograd.grad(run(q.requires_grad_(True)).sum(), q)[0])
        else:
            x = torch.randn(N, C, generator=g, device="cuda")
            t = torch.arange(N, device="cuda")
            assert torch.equal(head(x, t), LinearCrossEntropy(C, V, weight=-leaf.detach())(x, t))
            em = Embedding(V, C, weight=torch.nn.Parameter(_negated(leaf.detach())))
            assert torch.equal(em(t), -em.weight.detach().neg()[t])
        y = run(leaf)
        u = up if y.dim() > 1 else up[:, 0].contiguous()
        (got,) = torch.autograd.grad(y, leaf, _negated(u))
        assert torch.equal(got, torch.autograd.grad(run(leaf), leaf, -u)[0])
    x = torch.randn(N, C, generator=g, device="cuda")
    w, b = torch.randn(2, C, generator=g, device="cuda")
    ln = LayerNorm(C, weight=torch.nn.Parameter(_negated(w)), bias=torch.nn.Parameter(_negated(b)))
    assert torch.equal(ln(x), LayerNorm(C, weight=-w, bias=-b)(x))
    drop = Dropout(0.5)
    assert torch.equal(drop(x, _negated(x)), drop(x, -x))


def test_layers_around_the_split_linear_layer():
    """Embedding, dropout, norm, MetisLinear, dropout with the residual, norm and loss in one graph: the gradients are the
    library's calls', in a step that sketches and in one that reuses the factors."""
    say("embedding, dropout, norm, MetisLinear, dropout, norm, loss: one graph")
    vocab, cols, tokens = 301, 96, 128
    g = torch.Generator(device="cuda").manual_seed(9)
    em = Embedding(vocab, cols, scale=cols ** 0.5, weight=torch.randn(vocab, cols, generator=g, device="cuda") * 0.05)
    lin = MetisLinear(cols, cols, 8, s=8, l_k=32, refresh=8, weight=torch.randn(cols, cols, generator=g, device="cuda") * cols ** -0.5)
    drop1, drop2, norm1, norm2 = Dropout(0.1, layer=1), Dropout(0.2, layer=2), LayerNorm(cols), LayerNorm(cols)
    head = LinearCrossEntropy(cols, vocab, weight=em.weight)
    model = torch.nn.ModuleList([em, lin, drop1, drop2, norm1, norm2, head])
    ids = torch.randint(0, vocab, (4, tokens // 4), generator=g, device="cuda")
    t = ids.roll(-1, -1).clone()
    t[:, -1] = -100
    both, w, flat, ft = metis.AXIS0 | metis.AXIS1, em.weight.detach(), ids.reshape(-1), t.reshape(-1)
    f = {n: metis.Factors(r, cols, 8) for n, r in (("X", tokens), ("W", cols), ("D", tokens))}
    for step in (0, 1):
        set_step(model, step)
        model.zero_grad()
        h = drop1(em(ids))
        loss = head(norm2(drop2(lin(norm1(h)), h)), t)
        loss.backward()
        prepared = lambda m, n: metis.prepare_operand(m, lin.cfg, n != "W", lin.tags[n], step, f[n], both)  # noqa: E731,B023
        h1 = metis.dropout(metis.embedding(w, flat, em.scale), 0.1, tag=drop1.tag, step=step)
        n1, mu1, r1 = metis.layernorm(h1, norm1.weight, norm1.bias)
        qx, qw = prepared(n1, "X"), prepared(lin.weight.detach(), "W")
        h2 = metis.dropout(metis.gemm_fwd(qx, qw), 0.2, h1, 0, drop2.tag, step)
        n2, mu2, r2 = metis.layernorm(h2, norm2.weight, norm2.bias)
        _, lse, total = metis.cross_entropy(n2, w, ft)
        assert torch.equal(loss.detach(), total[0])
        d, dw = metis.cross_entropy_bwd(n2, w, ft, lse, torch.ones((), device="cuda"), total[1])
        d, a, b = metis.layernorm_bwd(d, h2, mu2, r2, norm2.weight)
        assert torch.equal(norm2.weight.grad, a) and torch.equal(norm2.bias.grad, b)
        dx, dlin = metis.gemm_bwd(prepared(metis.dropout(d, 0.2, tag=drop2.tag, step=step), "D"), qw, qx)
        assert torch.equal(lin.weight.grad, dlin)
        d1, a, b = metis.layernorm_bwd(dx, h1, mu1, r1, norm1.weight)
        assert torch.equal(norm1.weight.grad, a) and torch.equal(norm1.bias.grad, b)
        d = metis.dropout(d + d1, 0.1, tag=drop1.tag, step=step)
        assert torch.equal(em.weight.grad, dw + metis.embedding_bwd(d, flat, vocab, None, em.scale))
    metis.status_sync()


@pytest.mark.parametrize("reentrant", [False, True])
def test_recomputed_activations_give_the_same_gradients(reentrant):
    from torch.utils.checkpoint import checkpoint
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(N, C, generator=g, device="cuda", requires_grad=True)
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    ln, drop, head = LayerNorm(C), Dropout(0.3, seed=4), LinearCrossEntropy(C, V)
    set_step(drop, 7)
    say("recomputed activations, reentrant %s" % reentrant)
    block = lambda q: head(drop(ln(q), q), t)  # noqa: E731
    leaves = [x, ln.weight, ln.bias, head.weight]
    block(x).backward()
    want = [p.grad for p in leaves]
    for p in leaves:
        p.grad = None
    checkpoint(block, x, use_reentrant=reentrant).backward()
    assert all(torch.equal(p.grad, w) for p, w in zip(leaves, want))


def test_transforms_over_batches_and_functions_raise():
    for name, run, leaf in _layers():
        say("transforms: %s" % name)
        q = leaf.detach()
        if name != "embedding":  # (its call here closes over the weight)
            for transform in (lambda: torch.func.vmap(run)(q.expand(3, *q.shape)), lambda: torch.func.grad(lambda v: run(v).sum())(q),
                              lambda: torch.func.jvp(run, (q,), (q,))):
                with pytest.raises((RuntimeError, NotImplementedError, ValueError)):
                    transform()
        y = run(leaf)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(y, leaf, torch.ones(2, *y.shape, device="cuda"), is_grads_batched=True)
