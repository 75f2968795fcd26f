"""What autograd asks of the layers around the linear ones beyond a plain
backward pass."""

import pytest
import torch

from spectral_split_quantized_amd import metis
from spectral_split_quantized_amd.layer import Dropout, Embedding, LayerNorm, LinearCrossEntropy, set_step

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
