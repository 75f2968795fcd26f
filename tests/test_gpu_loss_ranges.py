"""The loss over a vocabulary at the ends of its ranges."""

import numpy as np
import pytest
import torch

from spectral_split_quantized_amd import metis
from spectral_split_quantized_amd.layer import LinearCrossEntropy

from gpu_helpers import say
from test_gpu_model import _loss_limits, f64, near

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


@pytest.mark.parametrize("tokens,vocab,cols", [(70, 200, 96), (3, 70, 7), (520, 2100, 320), (300, 5000, 64)])
@pytest.mark.parametrize("xt,wt", [(BF, BF), (F, F), (BF, F), (F, BF)])
def test_gradients_of_losses_far_apart(tokens, vocab, cols, xt, wt):
    """Each token's probabilities have a scale of their own: a token's gradient
    keeps its bits however large another token's is."""
    say("cross entropy %d x %d x %d with gradients from 2^-70 to 2^70 %s %s" % (tokens, vocab, cols, xt, wt))
    g = torch.Generator(device="cuda").manual_seed(tokens + cols)
    x = torch.randn(tokens, cols, generator=g, device="cuda").to(xt)
    w = (torch.randn(vocab, cols, generator=g, device="cuda") * 2 / cols ** 0.5).to(wt)
    t = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    t[2::7] = -100
    up = torch.randn(tokens, generator=g, device="cuda") * torch.exp2(torch.linspace(-70, 70, tokens, device="cuda").round())
    up[5::11] = 0
    x[2::14] = float("nan")  # (left out)
    losses, lse, _ = metis.cross_entropy(x, w, t)
    dx, dw = metis.cross_entropy_bwd(x, w, t, lse, up)
    assert all(torch.equal(a, b) for a, b in zip(metis.cross_entropy_bwd(x, w, t, lse, up), (dx, dw)))
    assert torch.equal(metis.cross_entropy_bwd(x, w, t, lse, up, want_dw=False)[0], dx)
    assert torch.equal(metis.cross_entropy_bwd(x, w, t, lse, up, want_dx=False)[1], dw)
    T = t.cpu().numpy()
    use = T != -100
    X, W, G = np.where(use[:, None], f64(x), 0), f64(w), f64(up)[:, None]
    # P and its limits for gradients of one, then each row by its token's
    P1, dP1 = _loss_limits(X, W, T, np.ones(tokens), xt, wt)[4:]
    P, dP = P1 * G, dP1 * np.abs(G)
    # the other operand: bf16 as it is, binary32 a pair, or rounded to binary16 where the gradient is bf16; and then P's
    # high part alone
    pair = F in (xt, wt)
    ox, ow = (0 if xt == BF else 2.0 ** -21 if wt == F else 2.0 ** -11), (0 if wt == BF else 2.0 ** -21 if xt == F else 2.0 ** -11)
    ex, ew = (2.0 ** -11 if pair and xt == BF else 0), (2.0 ** -11 if pair and wt == BF else 0)
    size = np.abs(P) + dP
    near(dx, P @ W, dP @ np.abs(W) + size @ np.abs(W) * (vocab * U + ow + ex) + 2.0 ** -39 * np.abs(W).max() * size.sum(1, keepdims=True), "dx")
    assert not dx[5::11].any() and not dx[2::7].any()
    # dw: x carries the inverse of P's scale, under a common one, and is off by 2^-39 of its largest value there at most; a
    # scale is within a factor of two of its gradient
    worst = (np.abs(X).max(1) * np.abs(G[:, 0])).max()
    unit = (np.abs(P1) + dP1).sum(0)[:, None]
    near(dw, P.T @ X, dP.T @ np.abs(X) + size.T @ np.abs(X) * (tokens * U + ox + ew) + 2.0 ** -38 * unit * worst, "dw")
    metis.status_sync()


def test_the_layer_weighs_each_token():
    say("loss of each token, weighted over 30 orders of magnitude")
    g = torch.Generator(device="cuda").manual_seed(23)
    head = LinearCrossEntropy(64, 90, reduction="none")
    x = torch.randn(70, 64, generator=g, device="cuda", requires_grad=True)
    t = torch.randint(0, 90, (70,), generator=g, device="cuda")
    each = torch.autograd.grad(head(x, t), x, torch.ones(70, device="cuda"))[0]
    weights = torch.exp2(-torch.arange(70, device="cuda").float())
    got = torch.autograd.grad(head(x, t), x, weights)[0]
    assert torch.equal(got, each * weights[:, None])  # powers of two, and no other token's part
