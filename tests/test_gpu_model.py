"""GPU parity of the operators around the linear layers with the float64
oracle.  Tolerances count roundings: u = 2^-24 is binary32's half step, and an
output's own rounding is finfo(t).eps / 2 of its value."""

import numpy as np
import pytest
import torch

from oracle import model
from spectral_split_quantized_amd import metis
from spectral_split_quantized_amd.layer import Dropout, Embedding, Int8Linear, LayerNorm, LinearCrossEntropy, set_step
from spectral_split_quantized_amd.optim import AdamW

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


def f64(t):
    return t.detach().double().cpu().numpy()


def half(t):
    return torch.finfo(t).eps / 2


def near(got, want, tol, what):
    """|got - want| within tol plus the rounding to got's type."""
    g = f64(got)
    assert g.shape == want.shape, what
    # a value that rounds across a step of its type: half a step of the larger
    limit = tol + half(got.dtype) * (np.abs(want) + tol) + 2.0 ** -133
    bad = ~(np.abs(g - want) <= limit)
    assert not bad.any(), "%s: %d outside, worst %.3g of its limit" % (what, bad.sum(), np.nanmax(np.abs(g - want) / limit))


def strided(t, gap):
    """The same values as rows with a gap behind each, and the memory behind."""
    rows, cols = t.shape
    room = torch.full((rows, cols + gap), 77.0, dtype=t.dtype, device=t.device)
    room[:, :cols] = t
    return room[:, :cols], room


# -------------------------------------------------------------- layer norm --

NORMS = [(1, 1), (3, 2), (5, 7), (2, 63), (9, 64), (17, 65), (4, 512), (33, 513), (600, 768), (7, 1000), (5, 1024), (6, 1030), (3, 2048),
         (5, 2050), (70, 4096), (3, 4100), (2, 8192), (3, 8200), (2, 16384), (5, 16390), (70, 20001)]


@pytest.mark.parametrize("rows,cols", NORMS)
@pytest.mark.parametrize("xt,yt,wt", [(BF, BF, F), (F, F, F), (F, BF, F), (BF, BF, BF)])
def test_layernorm_matches_the_oracle(rows, cols, xt, yt, wt):
    say("layer norm %d x %d %s %s %s" % (rows, cols, xt, yt, wt))
    g = torch.Generator(device="cuda").manual_seed(rows * 31 + cols)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gap = {0: 0, 1: 8, 2: 3}[(rows + cols) % 3]
    x, _ = strided((rnd(rows, cols) * 2 + 3 * rnd(rows, 1)).to(xt), gap)
    w, b, dy = (1 + rnd(cols)).to(wt), rnd(cols).to(wt), rnd(rows, cols).to(yt)
    eps = 1e-3
    yv, room = strided(torch.zeros(rows, cols, dtype=yt, device="cuda"), gap)
    y, mean, rstd = metis.layernorm(x, w, b, eps, Y=yv)
    dx, dw, db = metis.layernorm_bwd(dy, x, mean, rstd, w)
    metis.status_sync()
    X, W, B, DY = f64(x), f64(w), f64(b), f64(dy)
    ry, rm, rr = model.layernorm(X, W, B, eps)
    rdx, rdw, rdb = model.layernorm_bwd(DY, X, W, eps)
    assert gap == 0 or bool((room[:, cols:] == 77).all())
    # mean: at most 32 values a thread one after the other (or cols / 1024),
    # then a tree of ten and sixteen partial sums
    depth = max(32, cols / 1024) + 30
    dm = depth * U * np.abs(X).mean(axis=1) + U * np.abs(rm)
    near(mean, rm, dm, "mean")
    # 1 / sd: the variance moves by twice the mean's error times the centred
    # values (whose mean magnitude is below sd) and by its own sum
    dr = rr * (2 * dm * rr + (depth + 8) * U)
    near(rstd, rr, dr, "rstd")
    h = (X - rm[:, None]) * rr[:, None]
    dh = (dm * rr)[:, None] + np.abs(h) * (dr / rr)[:, None] + 4 * U * (np.abs(h) + np.abs(X) * rr[:, None])
    near(y, ry, dh * np.abs(W) + 3 * U * (np.abs(h * W) + np.abs(B)), "y")
    gr = np.abs(DY * W)
    mg, mq = gr.mean(axis=1, keepdims=True), (gr * np.abs(h)).mean(axis=1, keepdims=True)
    dq = (gr * dh).mean(axis=1, keepdims=True) + (depth + 4) * U * mq
    tol = rr[:, None] * ((depth + 4) * U * mg + np.abs(h) * dq + dh * mq + 6 * U * (gr + mg + np.abs(h) * mq)) + np.abs(rdx) * (dr / rr)[:, None]
    near(dx, rdx, tol, "dx")
    # sums over rows: at most rows values one after the other
    near(dw, rdw, (np.abs(DY) * dh).sum(axis=0) + (rows + 4) * U * (np.abs(DY * h)).sum(axis=0), "dw")
    near(db, rdb, rows * U * np.abs(DY).sum(axis=0), "db")
    again = metis.layernorm_bwd(dy, x, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))


def test_layernorm_parts_and_places():
    say("layer norm: parts, in place, without parameters, no rows")
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(40, 96, generator=g, device="cuda")
    w, dy = torch.randn(96, generator=g, device="cuda"), torch.randn(40, 96, generator=g, device="cuda")
    y, mean, rstd = metis.layernorm(x, w)
    dx, dw, db = metis.layernorm_bwd(dy, x, mean, rstd, w)
    for want in ((True, False, False), (False, True, False), (False, False, True), (False, True, True)):
        got = metis.layernorm_bwd(dy, x, mean, rstd, w, *want)
        assert all((a is None) == (not n) and (a is None or torch.equal(a, b)) for a, b, n in zip(got, (dx, dw, db), want))
    z = x.clone()
    assert torch.equal(metis.layernorm(z, w, Y=z)[0], y) and torch.equal(z, y)
    ones = torch.ones(96, device="cuda")
    assert torch.equal(metis.layernorm(x)[0], metis.layernorm(x, ones, torch.zeros(96, device="cuda"))[0])
    assert torch.equal(metis.layernorm(x, stats=False)[0], metis.layernorm(x)[0])
    e = torch.empty(0, 96, device="cuda")
    none = torch.empty(0, device="cuda")
    dx, dw, db = metis.layernorm_bwd(e, e, none, none, w)
    assert dx.shape == (0, 96) and not dw.any() and not db.any()
    long = torch.randn(3, 20000, generator=g, device="cuda")  # dx over dy where the row does not fit registers
    dl = torch.randn(3, 20000, generator=g, device="cuda")
    _, m, r = metis.layernorm(long)
    want = metis.layernorm_bwd(dl, long, m, r)
    lib = metis.load()
    ws = torch.empty(lib.metis_layernorm_bwd_workspace(3, 20000), dtype=torch.uint8, device="cuda")
    dw, db, over = (torch.empty(20000, device="cuda") for _ in range(2)), None, dl.clone()
    dw, db = dw
    assert lib.metis_layernorm_bwd(over.data_ptr(), 1, 20000, long.data_ptr(), 1, 3, 20000, 20000, None, 1, m.data_ptr(), r.data_ptr(),
                                   over.data_ptr(), 20000, dw.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel(),
                                   torch.cuda.current_stream().cuda_stream) == metis.OK
    assert all(torch.equal(a, b) for a, b in zip((over, dw, db), want))


def test_layernorm_rows_do_not_meet():
    say("layer norm: a row of NaN, a constant row, large values")
    x = torch.randn(6, 130, device="cuda")
    clean = metis.layernorm(x)[0]
    x[2], x[4] = float("nan"), 5.0
    y = metis.layernorm(x)[0]
    assert y[2].isnan().all() and (y[4] == 0).all()
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], clean[keep])
    big = x[:1] * 1e15  # squares overflow nothing below 2^128
    assert torch.isfinite(metis.layernorm(big)[0]).all()


# ----------------------------------------------------------------- dropout --

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 8), (5, 33), (64, 64), (101, 770), (1, 4099), (700, 1024)])
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout_is_the_oracles_to_the_bit(rows, cols, dt, p):
    say("dropout %d x %d %s %g" % (rows, cols, dt, p))
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(dt)
    res = torch.randn(rows, cols, generator=g, device="cuda").to(dt)
    x.view(-1)[:: 5] = float("inf")
    tag = metis.make_tag(3, metis.OPERAND_X)
    for r in (None, res):
        want = model.dropout(x.float().cpu().numpy(), p, 2 ** 40 + 7, tag, 11, None if r is None else r.float().cpu().numpy())
        want = torch.from_numpy(want).to(dt)
        for gap in (0, 8, 3):
            xs, rs = strided(x, gap)[0], None if r is None else strided(r, 2 * gap)[0]
            ys, room = strided(torch.zeros_like(x), gap)
            metis.dropout(xs, p, rs, 2 ** 40 + 7, tag, 11, Y=ys)
            assert torch.equal(ys.cpu().nan_to_num(9), want.nan_to_num(9))
            assert gap == 0 or bool((room[:, cols:] == 77).all())
            metis.dropout(xs, p, rs, 2 ** 40 + 7, tag, 11, Y=xs)  # in place
            assert torch.equal(xs.cpu().nan_to_num(9), want.nan_to_num(9))
    metis.status_sync()


def test_dropout_step_on_the_gpu_and_far_elements():
    say("dropout: steps, elements past 2^32 counters' blocks")
    x = torch.randn(50, 40, device="cuda")
    count = torch.zeros((), dtype=torch.int64, device="cuda")
    for step in (0, 5, 2 ** 31 + 9, 4):
        count.fill_(-1 if step == 4 else step)
        assert torch.equal(metis.dropout(x, 0.3, seed=1, step=4, step_count=count), metis.dropout(x, 0.3, seed=1, step=step))
    # rows far apart in memory: 3 rows whose offsets pass 2^32 bytes
    room = torch.zeros(2 * (1 << 30) + 4096, dtype=BF, device="cuda")
    far = torch.as_strided(room, (3, 64), (1 << 30, 1))
    far.copy_(torch.randn(3, 64, device="cuda"))
    assert torch.equal(metis.dropout(far, 0.5, seed=2), metis.dropout(far.contiguous(), 0.5, seed=2))
    y, _, _ = metis.layernorm(far)
    assert torch.equal(y, metis.layernorm(far.contiguous())[0])


# --------------------------------------------------------------- embedding --

@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 1), (3, 5, 7), (16, 3, 8), (17, 600, 65), (1000, 10, 64), (1023, 300000, 8), (1024, 511, 8), (1024, 512, 12), (1025, 70000, 20), (5000, 513, 770),
                                               (300, 300000, 8), (3000, 300000, 8), (40000, 50257, 16)])
@pytest.mark.parametrize("wt,yt,bits", [(BF, BF, 64), (F, F, 32), (F, BF, 64), (BF, F, 32)])
def test_embedding_matches_the_oracle(tokens, vocab, cols, wt, yt, bits):
    say("embedding %d of %d x %d %s %s %d" % (tokens, vocab, cols, wt, yt, bits))
    g = torch.Generator(device="cuda").manual_seed(tokens + cols)
    w, wroom = strided(torch.randn(vocab, cols, generator=g, device="cuda").to(wt), 8 if cols % 3 else 0)
    ids = (torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64) ** 3 * vocab).long().clamp(max=vocab - 1)
    ids = ids.to(torch.int32 if bits == 32 else torch.int64)
    scale = 0.3
    y = metis.embedding(w, ids, scale, out_dtype=yt)
    assert torch.equal(y, (w[ids.long()].float() * scale).to(yt))
    dy = torch.randn(tokens, cols, generator=g, device="cuda").to(yt)
    for padding in (None, int(ids[0])):
        dw = metis.embedding_bwd(dy, ids, vocab, padding, scale, w_dtype=wt)
        want = model.embedding_bwd(f64(dy), ids.cpu().numpy(), vocab, padding, scale)
        size = model.embedding_bwd(np.abs(f64(dy)), ids.cpu().numpy(), vocab, padding, scale)
        # a token's rows in pieces of 16, the pieces one after the other
        most = int(torch.bincount(ids.long()).max())
        near(dw, want, (min(most, 16) + most / 16 + 3) * U * size, "dw")
        assert not dw[torch.from_numpy(size.sum(axis=1) == 0).cuda()].any()
        assert torch.equal(dw, metis.embedding_bwd(dy, ids, vocab, padding, scale, w_dtype=wt))
    metis.status_sync()


def test_embedding_of_no_tokens_one_token_and_numbers_outside():
    say("embedding: no tokens, all alike, outside the vocabulary")
    w = torch.randn(11, 24, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert metis.embedding(w, none).shape == (0, 24)
    assert not metis.embedding_bwd(torch.empty(0, 24, device="cuda"), none, 11).any()
    dy = torch.randn(3000, 24, device="cuda")
    same = torch.full((3000,), 10, device="cuda")
    dw = metis.embedding_bwd(dy, same, 11)
    near(dw[10], f64(dy).sum(axis=0), (16 + 3000 / 16 + 3) * U * np.abs(f64(dy)).sum(axis=0), "one row")
    assert not dw[:10].any()
    metis.status_sync()
    for dt in (torch.int32, torch.int64):
        bad = torch.tensor([3, -1, 11, 2 ** 31 - 1, 4] + ([2 ** 40, -2 ** 40] if dt == torch.int64 else []), dtype=dt, device="cuda")
        y = metis.embedding(w, bad)
        with pytest.raises(metis.MetisError):
            metis.status_sync()
        ok = torch.tensor([0, 4], device="cuda")
        assert torch.equal(y[ok], w[[3, 4]]) and not y[1:4].any() and not y[5:].any()
        d = torch.randn(len(bad), 24, device="cuda")
        dw = metis.embedding_bwd(d, bad, 11)
        with pytest.raises(metis.MetisError):
            metis.status_sync()
        assert torch.equal(dw[[3, 4]], d[ok]) and not dw[[0, 1, 2, 5, 6, 7, 8, 9, 10]].any()


# -------------------------------------------------------------------- loss --

def _loss_limits(X, W, T, up, xt, wt):
    """Reference values and their limits."""
    use = (T >= 0) & (T < len(W))
    losses, lse, p = model.cross_entropy(X, W, T, -100)
    pair = F in (xt, wt)
    # logits: sums of cols products.  binary16 has 11 significant bits, so the
    # high part of a binary32 operand is off by 2^-11 of it at most, and the low
    # part, the rest rounded, by 2^-11 of the rest: the pair by 2^-22.  A product
    # of two pairs is off by that twice and by low times low, 2^-11 2^-11, left
    # out: 3 2^-22.  Below its normal range binary16 is off by 2^-25, where the
    # operand's largest value is 2^14 or more: 2^-39 of that.
    XU = np.where(use[:, None], X, 0)
    size = np.abs(XU) @ np.abs(W).T
    small = 2.0 ** -39 * 2 * X.shape[1] * np.abs(XU).max() * np.abs(W).max()
    dl = size * (X.shape[1] * U + (3 * 2.0 ** -22 if pair else 0)) + small
    at = np.where(use, T, 0)
    # log-sum-exp: the worst logit error, the sums' depth (64 values, then
    # blocks of 64 words in four parts), exponentials and logarithm
    dlse = dl.max(axis=1) + (64 + len(W) / 256 + 16) * 2 * U + 8 * U * (np.abs(lse) + size.max(axis=1))
    dloss = dlse + dl[np.arange(len(T)), at] + U * np.abs(lse)
    soft = np.abs(np.where(np.arange(len(W)) == at[:, None], p + 1, p)) * use[:, None]
    step = 2.0 ** -22 if pair else 2.0 ** -11  # P as a pair, or rounded to binary16
    G = np.abs(up)[:, None]
    dp = G * (soft * (dl + dlse[:, None] + 16 * U * (1 + size)) + 4 * U * (soft + np.abs(p))) + (step + 2 * U) * np.abs(p) * G + 2.0 ** -39 * G.max()
    return losses, lse, dloss, dlse, p * up[:, None], dp * use[:, None]


LOSSES = [(1, 1, 1), (1, 2, 64), (3, 70, 7), (5, 64, 128), (64, 65, 64), (65, 300, 100), (130, 1000, 192), (37, 5000, 768), (300, 259, 33),
          (1030, 515, 64), (2, 9000, 65), (520, 2100, 320)]


@pytest.mark.parametrize("tokens,vocab,cols", LOSSES)
@pytest.mark.parametrize("xt,wt,bits", [(BF, BF, 64), (F, F, 32), (F, BF, 64), (BF, F, 64)])
def test_cross_entropy_matches_the_oracle(tokens, vocab, cols, xt, wt, bits):
    say("cross entropy %d x %d x %d %s %s" % (tokens, vocab, cols, xt, wt))
    g = torch.Generator(device="cuda").manual_seed(tokens + vocab + cols)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gap = {0: 0, 1: 64, 2: 3}[(tokens + vocab) % 3]
    x, _ = strided(rnd(tokens, cols).to(xt), gap)
    w, _ = strided((rnd(vocab, cols) * 2 / cols ** 0.5).to(wt), gap)
    t = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    t[2::5] = -100
    up = rnd(tokens)
    t32 = t.to(torch.int32 if bits == 32 else torch.int64)
    losses, lse, total = metis.cross_entropy(x, w, t32)
    X, W, T = f64(x), f64(w), t.cpu().numpy()
    use = T != -100
    rl, rlse, dloss, dlse, P, dP = _loss_limits(X, W, T, f64(up), xt, wt)
    near(losses, rl, dloss * use, "losses")
    near(lse, rlse, dlse, "lse") if use.all() else near(lse[t >= 0], rlse[use], dlse[use], "lse")
    assert total[1].item() == use.sum()
    near(total[0], np.array(rl.sum() / max(use.sum(), 1)), (dloss * use).sum() / max(use.sum(), 1) + 2 * U * abs(rl.mean()), "mean")
    summed = metis.cross_entropy(x, w, t32, mean=False)[2]
    near(summed[0], np.array(rl.sum()), (dloss * use).sum() + 2 * U * abs(rl.sum()), "sum")

    def grads(dx, dw, P, dP, what):
        # the gradients' other operand: bf16 as it is; binary32 as a pair (2^-22,
        # and as much for low times low), or rounded to binary16 (2^-11) where
        # the gradient itself is bf16; 2^-39 of the largest value is added for
        # what lies below binary16's normal range
        ow = 0.0 if wt == BF else (2.0 ** -21 if xt == F else 2.0 ** -11)
        ox = 0.0 if xt == BF else (2.0 ** -21 if wt == F else 2.0 ** -11)
        sx = np.abs(P) + dP
        dP = dP + 2.0 ** -39 * np.abs(P).max()
        extra = 2.0 ** -11 if F in (xt, wt) else 0.0  # the high part of P alone, for a bf16 gradient
        near(dx, P @ W, dP @ np.abs(W) + 2.0 ** -39 * np.abs(W).max() * sx.sum(1, keepdims=True) + sx @ np.abs(W) * (vocab * U + ow + (extra if xt == BF else 0)), what + " dx")
        XX = np.where(use[:, None], X, 0)
        near(dw, P.T @ XX, dP.T @ np.abs(XX) + 2.0 ** -39 * np.abs(XX).max() * sx.sum(0)[:, None] + sx.T @ np.abs(XX) * (tokens * U + ox + (extra if wt == BF else 0)), what + " dw")

    dx, dw = metis.cross_entropy_bwd(x, w, t32, lse, up)
    grads(dx, dw, P, dP, "each")
    one = torch.tensor(0.7, device="cuda")
    P1, dP1 = _loss_limits(X, W, T, np.full(tokens, 0.7 / max(use.sum(), 1)), xt, wt)[4:]
    got = metis.cross_entropy_bwd(x, w, t32, lse, one, total[1])
    grads(*got, P1, dP1 + 4 * U * np.abs(P1), "mean")
    again = metis.cross_entropy_bwd(x, w, t32, lse, one, total[1])
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert torch.equal(metis.cross_entropy_bwd(x, w, t32, lse, one, total[1], want_dw=False)[0], got[0])
    assert torch.equal(metis.cross_entropy_bwd(x, w, t32, lse, one, total[1], want_dx=False)[1], got[1])
    metis.status_sync()


def test_cross_entropy_in_several_pieces():
    say("cross entropy over pieces of the vocabulary")
    g = torch.Generator(device="cuda").manual_seed(4)
    n, v, d = 4096, 140001, 64  # three pieces of 65536 words and less
    x = torch.randn(n, d, generator=g, device="cuda").to(BF)
    w = (torch.randn(v, d, generator=g, device="cuda") * 0.3).to(BF)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[0], t[1], t[2] = v - 1, 65535, 65536
    losses, lse, total = metis.cross_entropy(x, w, t)
    z = x.double() @ w.double().T
    rlse = torch.logsumexp(z, 1)
    rl = rlse - z.gather(1, t[:, None])[:, 0]
    dl = (x.double().abs() @ w.double().abs().T).amax(1) * d * U
    assert ((losses - rl).abs() <= 2 * dl + (64 + v / 256 + 16) * 2 * U + 16 * U * z.abs().amax()).all()
    p = torch.exp(z - rlse[:, None])
    p[torch.arange(n), t] -= 1
    p /= n
    one = torch.ones((), device="cuda")
    dx, dw = metis.cross_entropy_bwd(x, w, t, lse, one, total[1])
    sx, sw = p.abs() @ w.double().abs(), p.abs().T @ x.double().abs()
    rel = 2.0 ** -11 + 64 * 2.0 ** -20  # P's rounding, and its own error (logits here below 64 in size)
    assert ((dx - p @ w.double()).abs() <= sx * (rel + v / 8 * U) + 2.0 ** -8 * (p @ w.double()).abs()).all()
    assert ((dw - p.T @ x.double()).abs() <= sw * (rel + n * U) + 2.0 ** -8 * (p.T @ x.double()).abs()).all()


@pytest.mark.parametrize("xs,ws,us", [(0, 0, 0), (60, -60, 0), (-70, 69, 40), (-120, 118, -90), (40, -41, 100)])
@pytest.mark.parametrize("xt,wt", [(BF, BF), (F, F), (F, BF)])
def test_cross_entropy_over_the_exponents(xt, wt, xs, ws, us):
    """Operands and gradients of any size, in rows of sizes far apart: the planes' scale follows the largest value."""
    say("cross entropy of x 2^%d, w 2^%d, gradients 2^%d %s %s" % (xs, ws, us, xt, wt))
    tokens, vocab, cols = 70, 200, 96
    g = torch.Generator(device="cuda").manual_seed(xs + 200)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (rnd(tokens, cols) * 2.0 ** xs).to(xt)
    x[1::7] *= 2.0 ** -12
    w = (rnd(vocab, cols) * 2.0 ** ws / cols ** 0.5).to(wt)
    w[3::5] *= 2.0 ** -10
    w[4] = 0
    t = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    t[5] = -100
    x[5] = float("nan")
    up = rnd(tokens) * 2.0 ** us
    up[::9] *= 2.0 ** -9
    X, W, T = np.nan_to_num(f64(x)), f64(w), t.cpu().numpy()
    use = T != -100
    rl, rlse, dloss, dlse, P, dP = _loss_limits(X, W, T, f64(up), xt, wt)
    losses, lse, _ = metis.cross_entropy(x, w, t)
    near(losses, np.where(use, rl, 0), dloss * use, "losses")
    dx, dw = metis.cross_entropy_bwd(x, w, t, lse, up)
    XX = np.where(use[:, None], X, 0)
    P, dP = np.where(use[:, None], P, 0), np.where(use[:, None], dP, 0)
    ow = 2.0 ** -21 if wt == F else 0.0
    ox = 0.0 if xt == BF else 2.0 ** -21 if wt == F else 2.0 ** -11
    extra = 2.0 ** -11 if F in (xt, wt) and wt == BF else 0.0  # the high part of P alone
    sx = np.abs(P) + dP
    dP = dP + 2.0 ** -39 * np.abs(P).max()
    near(dx, P @ W, dP @ np.abs(W) + sx @ np.abs(W) * (vocab * U + ow) + 2.0 ** -39 * np.abs(W).max() * sx.sum(1, keepdims=True), "dx")
    want, tol = P.T @ XX, dP.T @ np.abs(XX) + sx.T @ np.abs(XX) * (tokens * U + ox + extra) + 2.0 ** -39 * np.abs(XX).max() * sx.sum(0)[:, None]
    # gradients of 2^100 times an x of 2^40 lie beyond the type's largest value, 2^128: infinities of their sign
    beyond = np.abs(want) - tol >= 2.0 ** 128
    got = f64(dw)
    assert (got[beyond] == np.sign(want[beyond]) * np.inf).all()
    sure = np.abs(want) + tol < torch.finfo(wt).max
    assert sure.all() or us + xs >= 120
    near(dw[torch.from_numpy(sure).cuda()], want[sure], tol[sure], "dw")
    metis.status_sync()


def test_cross_entropy_leaves_tokens_out():
    say("cross entropy: ignored tokens with anything in their rows, targets outside, none left, no tokens")
    g = torch.Generator(device="cuda").manual_seed(6)
    for dt in (BF, F):
        x = torch.randn(70, 64, generator=g, device="cuda").to(dt)
        w = torch.randn(90, 64, generator=g, device="cuda").to(dt)
        t = torch.randint(0, 90, (70,), generator=g, device="cuda")
        t[5], t[60] = -100, -100
        one = torch.ones((), device="cuda")
        losses, lse, total = metis.cross_entropy(x, w, t)
        dx, dw = metis.cross_entropy_bwd(x, w, t, lse, one, total[1])
        y = x.clone()
        y[5], y[60] = float("nan"), float("inf")
        y[5, 1], y[60, 2] = 1e30, -1e30
        l2, lse2, total2 = metis.cross_entropy(y, w, t)
        dx2, dw2 = metis.cross_entropy_bwd(y, w, t, lse2, one, total2[1])
        assert torch.equal(losses, l2) and torch.equal(total, total2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
        assert not dx[5].any() and losses[5] == 0
        metis.status_sync()
        bad = t.clone()
        bad[5], bad[60] = 90, -7  # not words: left out as well, and reported
        l3, lse3, total3 = metis.cross_entropy(x, w, bad)
        with pytest.raises(metis.MetisError):
            metis.status_sync()
        assert torch.equal(losses, l3) and torch.equal(total, total3)
        assert all(torch.equal(a, b) for a, b in zip(metis.cross_entropy_bwd(x, w, bad, lse3, one, total3[1]), (dx, dw)))
        none = torch.full_like(t, -100)
        losses, lse, total = metis.cross_entropy(x, w, none)
        assert not losses.any() and total.tolist() == [0.0, 0.0]
        assert not any(q.any() for q in metis.cross_entropy_bwd(x, w, none, lse, one, total[1]))
        losses, lse, total = metis.cross_entropy(x[:0], w, t[:0])
        assert losses.shape == (0,) and total.tolist() == [0.0, 0.0]
        dx, dw = metis.cross_entropy_bwd(x[:0], w, t[:0], lse, one, total[1])
        assert dx.shape == (0, 64) and dw.shape == (90, 64) and not dw.any()


def test_cross_entropy_of_extreme_logits():
    say("cross entropy: large logits, equal logits")
    w = torch.zeros(130, 64, device="cuda", dtype=BF)
    w[:, 0] = torch.arange(130, device="cuda") % 7
    x = torch.zeros(3, 64, device="cuda", dtype=BF)
    x[0, 0], x[1, 0] = 3000.0, -3000.0
    t = torch.tensor([6, 0, 5], device="cuda")
    losses, lse, _ = metis.cross_entropy(x, w, t)
    counts = [len(range(6, 130, 7)), len(range(0, 130, 7)), 130]
    assert np.allclose(f64(losses), np.log(counts), atol=18000 * 4 * U)
    dx, _ = metis.cross_entropy_bwd(x, w, t, lse, torch.ones(3, device="cuda"))
    assert torch.isfinite(dx).all()


# ------------------------------------------------------------------ layers --

def _block(vocab, cols, seed=0, dtype=F):
    """Embedding, dropout, norm, 8-bit linear, dropout with the residual, norm, loss (the embedding's weight)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    e = Embedding(vocab, cols, scale=cols ** 0.5, weight=(torch.randn(vocab, cols, generator=g, device="cuda") * 0.05).to(dtype))
    lin = Int8Linear(cols, cols, rounding="rne", weight=torch.randn(cols, cols, generator=g, device="cuda") * cols ** -0.5)

    class Block(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.embed, self.lin = e, lin
            self.drop1, self.drop2 = Dropout(0.1, seed=seed, layer=1), Dropout(0.2, seed=seed, layer=2)
            self.norm1, self.norm2 = LayerNorm(cols), LayerNorm(cols)
            self.head = LinearCrossEntropy(cols, vocab, weight=e.weight)

        def forward(self, ids, targets):
            h = self.drop1(self.embed(ids))
            h = self.drop2(self.lin(self.norm1(h)), h)
            return self.head(self.norm2(h), targets)
    return Block()


def _text(vocab, seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, vocab, shape, generator=g, device="cuda")
    t = ids.roll(-1, -1).clone()
    t[..., -1] = -100
    return ids, t


def test_layers_run_together_and_their_gradients_are_the_calls():
    say("embedding, dropout, norm, int8 linear, dropout, norm, loss: one graph")
    m = _block(301, 96)
    ids, t = _text(301, 1, 4, 33)
    set_step(m, 3)
    loss = m(ids, t)
    loss.backward()
    got = {k: p.grad.clone() for k, p in m.named_parameters()}
    # the same by the library's calls
    w, flat, ft = m.embed.weight.detach(), ids.reshape(-1), t.reshape(-1)
    e = metis.embedding(w, flat, m.embed.scale)
    h1 = metis.dropout(e, 0.1, seed=0, tag=m.drop1.tag, step=3)
    n1, mu1, r1 = metis.layernorm(h1, m.norm1.weight, m.norm1.bias)
    q = metis.int8_quantize(n1, metis.AXIS0 | metis.AXIS1)
    qw = metis.int8_quantize(m.lin.weight.detach(), metis.AXIS0 | metis.AXIS1)
    h2 = metis.dropout(metis.int8_gemm(q.ax1, qw.ax0), 0.2, h1, 0, m.drop2.tag, 3)
    n2, mu2, r2 = metis.layernorm(h2, m.norm2.weight, m.norm2.bias)
    _, lse, total = metis.cross_entropy(n2, w, ft)
    assert torch.equal(loss.detach(), total[0])
    d, dw = metis.cross_entropy_bwd(n2, w, ft, lse, torch.ones((), device="cuda"), total[1])
    d, a, b = metis.layernorm_bwd(d, h2, mu2, r2, m.norm2.weight)
    assert torch.equal(got["norm2.weight"], a) and torch.equal(got["norm2.bias"], b)
    qd = metis.int8_quantize(metis.dropout(d, 0.2, seed=0, tag=m.drop2.tag, step=3), metis.AXIS0 | metis.AXIS1)
    assert torch.equal(got["lin.weight"], metis.int8_gemm(q.ax0, qd.ax0))
    d1, a, b = metis.layernorm_bwd(metis.int8_gemm(qd.ax1, qw.ax1), h1, mu1, r1, m.norm1.weight)
    assert torch.equal(got["norm1.weight"], a) and torch.equal(got["norm1.bias"], b)
    d = metis.dropout(d + d1, 0.1, seed=0, tag=m.drop1.tag, step=3)
    assert torch.equal(got["embed.weight"], dw + metis.embedding_bwd(d, flat, 301, None, m.embed.scale))
    metis.status_sync()


def test_layers_train_with_the_optimizer():
    say("a few steps of the block with AdamW")
    m = _block(301, 96)
    opt = AdamW(m.parameters(), lr=1e-3, max_norm=1.0)
    ids, t = _text(301, 2, 4, 33)
    for step in range(3):
        set_step(m, step)
        opt.zero_grad()
        m(ids, t).backward()
        before = [p.detach().clone() for p in m.parameters()]
        opt.step()
        assert all(torch.isfinite(p).all() and not torch.equal(p, q) for p, q in zip(m.parameters(), before))
    metis.status_sync()


def test_layers_in_a_graph_take_each_replays_step_and_inputs():
    say("captured passes of the block")
    m = _block(301, 96)
    ids, t = _text(301, 3, 4, 33)
    set_step(m, 1)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        m(ids, t).backward()
    torch.cuda.synchronize()
    m.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = m(ids, t)
        loss.backward()
    grads = {k: p.grad for k, p in m.named_parameters()}
    for step, seed in ((5, 7), (6, 7), (5, 8)):
        new, nt = _text(301, seed, 4, 33)
        ids.copy_(new)
        t.copy_(nt)
        set_step(m, step)
        graph.replay()
        torch.cuda.synchronize()
        other = _block(301, 96)
        set_step(other, step)
        want = other(new, nt)
        want.backward()
        assert torch.equal(want.detach(), loss)
        assert all(torch.equal(p.grad, grads[k]) for k, p in other.named_parameters())
    metis.status_sync()


def test_capture_next_to_a_living_eager_graph_is_refused():
    say("captures next to eager graphs of the same leaves")
    m = _block(51, 64)
    ids, t = _text(51, 3, 2, 20)
    keep = m(ids, t)
    x = torch.randn(4, 64, device="cuda", requires_grad=True)
    held = [m.norm1(x), m.drop1(x), m.embed(ids), m.head(x, t[0, :4])]
    torch.cuda.synchronize()
    for run in (lambda: m(ids, t), lambda: m.norm1(x), lambda: m.drop1(x), lambda: m.embed(ids), lambda: m.head(x, t[0, :4]),
                lambda: LayerNorm(64)(x)):
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError, match="alive"):
            with torch.cuda.graph(graph):
                run()
    del keep, held
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    say("tables, rows and vocabularies past 2^32 bytes")
    g = torch.Generator(device="cuda").manual_seed(12)
    rows, cols = 140000, 16384  # 4.6 GB of bf16, 2.3e9 values
    big = torch.zeros(rows, cols, dtype=BF, device="cuda")
    some = torch.tensor([0, 65535, 131071, 131072, 139999], device="cuda")
    big[some] = torch.randn(5, cols, generator=g, device="cuda").to(BF)
    part = big[some]
    ids = some[[4, 0, 3, 4, 2, 1]]
    assert torch.equal(metis.embedding(big, ids), big[ids])
    dy = torch.randn(6, cols, generator=g, device="cuda").to(BF)
    dw = metis.embedding_bwd(dy, ids, rows)
    near(dw[139999], f64(dy[0]) + f64(dy[3]), 4 * U * (np.abs(f64(dy[0])) + np.abs(f64(dy[3]))), "the last row")
    assert torch.equal(dw[131072], dy[2]) and torch.equal(dw[0], dy[1]) and not dw[139998].any() and not dw[131070].any()
    del dw
    y, mean, rstd = metis.layernorm(big)
    assert torch.equal(y[some], metis.layernorm(part)[0])
    dx = metis.layernorm_bwd(big, big, mean, rstd, want_dweight=False, want_dbias=False)[0]
    assert torch.equal(dx[some], metis.layernorm_bwd(part, part, mean[some], rstd[some], want_dweight=False, want_dbias=False)[0])
    del dx
    # the draws of a value follow from its place: those of the first rows again, and every row's share
    y = metis.dropout(big.fill_(1), 0.25, seed=3, Y=y)
    assert torch.equal(y[:100], metis.dropout(big[:100], 0.25, seed=3))
    kept = (y[some] != 0).double().mean(1)
    assert ((kept - 0.75).abs() < 6 * (0.25 * 0.75 / cols) ** 0.5).all()
    assert not torch.equal(y[131072 + 65536 // 16384], y[65536 // 16384])
    del y
    big.normal_(generator=g)
    x = torch.randn(3, cols, generator=g, device="cuda").to(BF) / cols ** 0.5
    t = torch.tensor([139999, 0, 131073], device="cuda")
    losses, lse, _ = metis.cross_entropy(x, big, t)
    z = torch.cat([x.double() @ big[i:i + 10000].double().T for i in range(0, rows, 10000)], 1)
    want = torch.logsumexp(z, 1) - z.gather(1, t[:, None])[:, 0]
    # each logit is a sum of 16384 products, |x| |w| below 128 in all
    assert ((losses - want).abs() <= 128 * cols * U + 1e-4).all()
    up = torch.ones(3, device="cuda")
    dx, dw = metis.cross_entropy_bwd(x, big, t, lse, up)
    p = torch.softmax(z, 1)
    p[torch.arange(3), t] -= 1
    for v in (0, 1, 131071, 131073, 139999):
        row = p[:, v] @ x.double()
        size = p[:, v].abs() @ x.double().abs()
        # P: rounded to binary16, and off by what the logits and the log-sum-exp are
        assert ((dw[v].double() - row).abs() <= 2.0 ** -8 * row.abs() + size * (2.0 ** -11 + 3 * 128 * cols * U)).all(), v
    metis.status_sync()


def test_embedding_gradient_of_numbers_of_28_bits():
    say("embedding: token numbers of 28 bits")
    g = torch.Generator(device="cuda").manual_seed(16)
    vocab = (1 << 27) + 5
    for tokens in (1000, 5000):
        ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        ids[::3] = ids[0]
        ids[1], ids[2], ids[4] = vocab - 1, 1 << 18, vocab - 1
        dy = torch.randn(tokens, 1, generator=g, device="cuda")
        dw = metis.embedding_bwd(dy, ids, vocab)
        want = torch.zeros(vocab, 1, dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double())
        size = torch.zeros(vocab, 1, dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double().abs())
        assert ((dw.double() - want).abs() <= (16 + tokens / 3 / 16 + 3) * U * size).all()
    metis.status_sync()


def test_more_words_than_rows_of_probabilities_may_hold():
    say("cross entropy over 9000001 words")
    g = torch.Generator(device="cuda").manual_seed(13)
    n, v = 3, 9000001
    x = torch.randn(n, 2, generator=g, device="cuda").to(BF)
    w = torch.randn(v, 2, generator=g, device="cuda").to(BF)
    t = torch.tensor([v - 1, 1 << 22, 17], device="cuda")
    losses, lse, _ = metis.cross_entropy(x, w, t)
    z = x.double() @ w.double().T
    rlse = torch.logsumexp(z, 1)
    assert ((lse - rlse).abs() <= (64 + v / 4096 + 16) * 2 * U + 32 * U).all()  # sums of 64, 1 / 64 of the blocks in a row, then joined
    dx, dw = metis.cross_entropy_bwd(x, w, t, lse, torch.ones(n, device="cuda"))
    p = torch.exp(z - rlse[:, None])
    p[torch.arange(n), t] -= 1
    want, size = p @ w.double(), p.abs() @ w.double().abs()
    # P rounded to binary16 (or off by 2^-25 of what 2^15 stands for), sums over words in parts and pieces
    tiny = 2.0 ** -39 * w.double().abs().sum(0)
    assert ((dx - want).abs() <= 2.0 ** -8 * want.abs() + size * (2.0 ** -11 + 1e-3) + tiny).all()
    want, size = p.T @ x.double(), p.abs().T @ x.double().abs()
    assert ((dw - want).abs() <= 2.0 ** -8 * want.abs() + size * (2.0 ** -11 + 1e-3) + 2.0 ** -39 * x.double().abs().sum(0)).all()
    metis.status_sync()


@pytest.mark.parametrize("dt", [BF, F])
def test_each_layer_in_a_graph_replayed_between_eager_work(dt):
    say("each layer captured alone, replayed with eager passes between, %s" % dt)
    g = torch.Generator(device="cuda").manual_seed(14)
    n, c, v = 70, 96, 301
    ln, em = LayerNorm(c), Embedding(v, c, padding_idx=3, out_dtype=dt)
    drop = Dropout(0.3, seed=5)
    heads = [LinearCrossEntropy(c, v, reduction=r, dtype=dt) for r in ("none", "sum", "mean")]
    set_step(drop, 0)
    x = torch.randn(n, c, generator=g, device="cuda").to(dt).requires_grad_(True)
    res = torch.randn(n, c, generator=g, device="cuda").to(dt).requires_grad_(True)
    ids = torch.randint(0, v, (n,), generator=g, device="cuda")
    runs = [(lambda: ln(x), [x, ln.weight, ln.bias]), (lambda: drop(x, res), [x, res]), (lambda: em(ids), [em.weight])]
    runs += [(lambda h=h: h(x, ids), [x, h.weight]) for h in heads]
    for run, leaves in runs:
        y = run()
        up = torch.randn(y.shape, generator=g, device="cuda").to(y.dtype)
        torch.autograd.grad(y, leaves, up)
        del y
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = run()
            grads = torch.autograd.grad(y, leaves, up)
        y = y.detach()
        for step in (1, 2, 3):
            with torch.no_grad():
                x.copy_(torch.randn(n, c, generator=g, device="cuda"))
                ids.copy_(torch.randint(0, v, (n,), generator=g, device="cuda"))
                ids[step::7] = -100 if leaves[-1] is not em.weight else 3
                up.copy_(torch.randn(up.shape, generator=g, device="cuda"))
            set_step(drop, step)
            graph.replay()
            torch.cuda.synchronize()
            kept = [y.clone()] + [q.clone() for q in grads]
            want = run()
            eager = torch.autograd.grad(want, leaves, up)
            assert all(torch.equal(a, b) for a, b in zip(kept, [want.detach(), *eager]))
            del want
    with pytest.raises(metis.MetisError):  # the embedding's first pass met the numbers -100 that dropout's passes left
        metis.status_sync()
    metis.status_sync()


def test_what_autograd_may_ask_of_the_layers():
    say("layers: a graph kept and used again, inputs changed in place, second derivatives, a loss scaled in place")
    n, c, v = 20, 64, 51
    ln, em, head, drop = LayerNorm(c), Embedding(v, c), LinearCrossEntropy(c, v), Dropout(0.5)
    x = torch.randn(n, c, device="cuda", requires_grad=True)
    ids = torch.randint(0, v, (n,), device="cuda")
    for run, leaves in ((lambda: ln(x), [x, ln.weight]), (lambda: drop(x), [x]), (lambda: em(ids), [em.weight]), (lambda: head(x, ids), [x, head.weight])):
        y = run()
        up = torch.ones_like(y)
        a = torch.autograd.grad(y, leaves, up, retain_graph=True)
        b = torch.autograd.grad(y, leaves, up)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    for run in (lambda: ln(x), lambda: em(ids), lambda: head(x, ids)):
        y = run()
        y.sum().backward()
        with pytest.raises(RuntimeError):
            y.sum().backward()  # what the pass kept is gone
    y = ln(x * 1)
    up = torch.ones_like(y, requires_grad=True)
    (first,) = torch.autograd.grad(y, x, up, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate"):
        first.sum().backward()
    for run in (lambda q: ln(q), lambda q: head(q, ids)):
        q = x * 1
        y = run(q)
        q += 1
        with pytest.raises(RuntimeError, match="modified"):
            y.sum().backward()
    # a loss divided in place, as by the number of micro-batches
    x.grad = None
    want = torch.autograd.grad(head(x, ids) / 4, [x, head.weight])
    loss = head(x, ids)
    loss /= 4
    assert all(torch.equal(p, q) for p, q in zip(torch.autograd.grad(loss, [x, head.weight]), want))
    metis.status_sync()


def test_two_streams_at_once():
    say("the loss and the embedding on two streams at once")
    g = torch.Generator(device="cuda").manual_seed(15)
    x = [torch.randn(700, 128, generator=g, device="cuda").to(dt) for dt in (BF, F)]
    w = [torch.randn(5000, 128, generator=g, device="cuda").to(dt) for dt in (BF, F)]
    t = torch.randint(0, 5000, (700,), generator=g, device="cuda")
    one = torch.ones((), device="cuda")

    def run(i):
        losses, lse, total = metis.cross_entropy(x[i], w[i], t)
        dx, dw = metis.cross_entropy_bwd(x[i], w[i], t, lse, one, total[1])
        return [losses, total, dx, dw, metis.embedding_bwd(x[i], t, 5000)]
    want = [run(0), run(1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(i))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for once in got[i] for a, b in zip(once, want[i]))
    metis.status_sync()


def test_layers_on_another_stream_and_without_gradients():
    say("layers on a stream of their own, no_grad, inference_mode, eval")
    m = _block(51, 64)
    ids, t = _text(51, 3, 2, 20)
    set_step(m, 2)
    want = m(ids, t).detach()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = m(ids, t).detach()
    s.synchronize()
    assert torch.equal(got, want)
    with torch.no_grad():
        assert torch.equal(m(ids, t), want)
    with torch.inference_mode():
        assert torch.equal(m(ids, t), want)
    m.eval()
    with torch.no_grad():
        h = metis.embedding(m.embed.weight, ids.reshape(-1), m.embed.scale)
        assert torch.equal(m.drop1(m.embed(ids)).reshape(-1, 64), h)


def test_layer_shapes_types_and_frozen_parts():
    say("layers: shapes, types, parts without gradients")
    for dt in (BF, F):
        x = torch.randn(2, 3, 70, device="cuda").to(dt).requires_grad_(True)
        ln = LayerNorm(70)
        ln.bias.requires_grad_(False)
        y = ln(x)
        assert y.shape == x.shape and y.dtype == dt
        y.backward(torch.ones_like(y))
        assert x.grad.shape == x.shape and x.grad.dtype == dt and ln.weight.grad.dtype == F and ln.bias.grad is None
        x.grad = None
        z = LayerNorm(70, affine=False)(x.transpose(0, 1))
        z.backward(torch.ones_like(z).transpose(0, 1).contiguous().transpose(0, 1))
        assert x.grad.shape == x.shape
        e = Embedding(9, 70, out_dtype=dt)
        assert e(torch.tensor([[1, 2], [3, 4]], device="cuda", dtype=torch.int32)).shape == (2, 2, 70)
        head = LinearCrossEntropy(70, 9, weight=e.weight, reduction="none")
        t = torch.tensor([[1, 2, -100], [0, 8, 3]], device="cuda")
        losses = head(x, t)
        assert losses.shape == t.shape and losses[0, 2] == 0
        x.grad = None
        losses.sum().backward()  # the gradient of a sum is an expanded one
        a = x.grad.clone()
        x.grad = None
        LinearCrossEntropy(70, 9, weight=e.weight, reduction="sum")(x, t).backward()
        assert torch.equal(a, x.grad) and x.grad.dtype == dt and not a[0, 2].any()
        x.grad = None
        drop = Dropout(0.5, seed=3)
        d = drop(x)
        d.backward(torch.ones_like(d))
        assert torch.equal(d.detach() == 0, x.grad == 0)
    metis.status_sync()
