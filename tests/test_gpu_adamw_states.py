"""GPU tests of the optimizer's states: step counts of their own, stored
values that are not finite, values kept beside a new maximum.

Moments, codes and scales are defined to the last bit and compared for
equality, with oracle/adamw.py or with an optimizer whose counts are host
integers."""

import numpy as np
import pytest
import torch

from spectral_split_quantized_amd import metis, optim

from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X; none is visible")
    metis.load()
    torch.cuda.set_device(0)


def _params(seed, sizes):
    g = torch.Generator().manual_seed(seed)
    return [torch.nn.Parameter(torch.randn(s, generator=g).cuda()) for s in sizes], g


@pytest.mark.parametrize("bits", [32, 8])
def test_counts_that_differ_in_a_captured_step(bits):
    """A parameter that had no gradient in some steps, loaded into an optimizer
    whose counts are on the GPU: eager and replayed steps equal those of host
    counts, stochastic draws included."""
    say("adamw, counts that differ, %d bits" % bits)
    ps, g = _params(1, ((50, 90), (4100,), (700,)))
    twins = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    eager = optim.AdamW(twins, lr=1e-2, state_bits=bits, min_8bit_size=1, seed=8)
    for t in range(5):
        for i, p in enumerate(twins):
            p.grad = None if i == 1 and t % 2 else torch.randn(p.shape, generator=g).cuda()
        eager.step()
    opt = optim.AdamW(ps, lr=1e-2, state_bits=bits, min_8bit_size=1, capturable=True, seed=8)
    opt.load_state_dict(eager.state_dict())
    assert [int(opt.state[p]["step"]) for p in ps] == [5, 3, 5]
    for a, b in zip(ps, twins):
        a.data.copy_(b.data)
        a.grad = torch.zeros_like(a)

    def feed():
        for a, b in zip(ps, twins):
            b.grad = torch.randn(a.shape, generator=g).cuda()
            a.grad.copy_(b.grad)

    def check():
        torch.cuda.synchronize()
        eager.step()
        for a, b in zip(ps, twins):
            for k in opt.state[a]:
                if k != "step":
                    assert torch.equal(opt.state[a][k].view(torch.uint8), eager.state[b][k].view(torch.uint8)), k
            # the bias corrections by squaring and by pow agree to binary64 rounding
            assert torch.allclose(a, b, rtol=2.0 ** -22, atol=2.0 ** -24 * 1e-2)

    feed()
    opt.step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for _ in range(3):
        feed()
        graph.replay()
        check()
    assert [int(opt.state[p]["step"]) for p in ps] == [9, 7, 9]
    metis.status_sync()
