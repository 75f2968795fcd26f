"""The loss over a vocabulary at the ends of its ranges."""

import pytest
import torch

from spectral_split_quantized_amd import metis

from gpu_helpers import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X; none is visible")
    metis.load()
    torch.cuda.set_device(0)
    metis.init_device()


@pytest.mark.parametrize("xt,wt", [(BF, BF), (F, F), (BF, F), (F, BF)])
def test_few_tokens_over_several_pieces(xt, wt):
    """A piece holds at most 2^29 values of the weight: 131072 words of 4096 values."""
    say("cross entropy of few tokens in two pieces %s %s" % (xt, wt))
    g = torch.Generator(device="cuda").manual_seed(21)
    n, v, d = 5, 140001, 4096
    x = torch.randn(n, d, generator=g, device="cuda").to(xt)
    w = (torch.randn(v, d, generator=g, device="cuda") * 2 / d ** 0.5).to(wt)
    t = torch.tensor([v - 1, 131071, 131072, -100, 17], device="cuda")
    use = t != -100
    at = torch.where(use, t, 0)
    losses, lse, total = metis.cross_entropy(x, w, t)
    z, size = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
    rlse = torch.logsumexp(z, 1)
    # logits: sums of d products, and two planes a binary32 value (3 2^-22); log-sum-exp: 64 values, then a 64th of the
    # blocks of 64 words one after the other, then six joins; exponentials and logarithm
    dl = (size * (d * U + (3 * 2.0 ** -22 if F in (xt, wt) else 0))).amax(1) + (64 + v / 4096 + 16) * 2 * U + 16 * U * size.amax(1)
    rl = torch.where(use, rlse - z.gather(1, at[:, None])[:, 0], 0.0)
    assert ((losses - rl).abs() <= 2 * dl * use + U * rl.abs()).all()
    dx, dw = metis.cross_entropy_bwd(x, w, t, lse, torch.ones((), device="cuda"), total[1])
    p = torch.exp(z - rlse[:, None])
    p[torch.arange(n), at] -= 1
    p *= use[:, None] / 4
    sx, sw = p.abs() @ w.double().abs(), p.abs().T @ x.double().abs()
    own = 2 * (2 * dl.amax() + 16 * U * (1 + size.amax())).item()  # P's own error: exponentials of logits less lse

    def rel(out, other):
        # P: a pair (2^-22) for a binary32 gradient, else rounded to binary16; the other operand: bf16 as it is, binary32 a
        # pair, or rounded to binary16 where the gradient is bf16
        return own + (2.0 ** -22 if out == F else 2.0 ** -11) + (0 if other == BF else 2.0 ** -21 if out == F else 2.0 ** -11)

    # what lies 2^-40 below the largest probability, or the largest value of the other operand, may be lost
    low = 2.0 ** -39
    want = p @ w.double()
    tol = sx * (rel(xt, wt) + v * U) + low * (0.25 * w.double().abs().sum(0) + w.double().abs().max() * p.abs().sum(1, keepdim=True))
    assert ((dx - want).abs() <= tol + torch.finfo(xt).eps / 2 * (want.abs() + tol)).all()
    want = p.T @ x.double()
    tol = sw * (rel(wt, xt) + n * U) + low * (0.25 * x.double().abs().sum(0) + x.double().abs().max() * p.abs().sum(0)[:, None])
    assert ((dw - want).abs() <= tol + torch.finfo(wt).eps / 2 * (want.abs() + tol)).all()
    assert not dx[3].any()
    metis.status_sync()
