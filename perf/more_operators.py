"""What stands around a language model's linear layers: cases, plain forms and exact values.

Operators: layer norm, dropout from a counter-based generator (with the
residual added), the embedding lookup, and the softmax cross entropy over a
vocabulary of the product of hidden states with an output weight; each with
its gradients.

``own`` selects the side: False runs the plain torch forms below, True the
library's layers.
"""

import math

import numpy as np
import torch

own = False

MASK32 = 0xFFFFFFFF
EPS = 1e-5               # of the norm
IGNORE = -100            # the target of a token without a loss
STEP, LAYER = 5, 3       # select the dropout's draws
OPERAND_X, ROLE_DROP = 2, 8


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # serving: the norm before a projection of an 8-billion-parameter model, a decode batch
        {"name": "norm_tokens", "op": "norm", "rows": 8, "cols": 4096, "dtype": "bf16", "train": False},
        # a training step's norm in a small model
        {"name": "norm_small", "op": "norm", "rows": 8192, "cols": 768, "dtype": "f32", "train": True},
        # and in the 8-billion-parameter one, 16384 tokens
        {"name": "norm_large", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16", "train": True},
        # dropout behind a small model's embedding, a ragged batch
        {"name": "drop_small", "op": "drop", "rows": 1001, "cols": 770, "dtype": "f32", "p": 0.1, "residual": False},
        # dropout of a block's output and the residual stream
        {"name": "drop_residual", "op": "drop", "rows": 16384, "cols": 4096, "dtype": "bf16", "p": 0.1, "residual": True},
        # serving: the embedding of a decode batch
        {"name": "embed_tokens", "op": "embed", "tokens": 48, "vocab": 50257, "cols": 768, "dtype": "bf16", "train": False},
        # a training step's embedding in a small model
        {"name": "embed_small", "op": "embed", "tokens": 8192, "vocab": 50257, "cols": 768, "dtype": "f32", "train": True},
        # and in the 8-billion-parameter one
        {"name": "embed_large", "op": "embed", "tokens": 16384, "vocab": 128256, "cols": 4096, "dtype": "bf16", "train": True},
        # the loss of a short text, for scoring
        {"name": "loss_tokens", "op": "loss", "tokens": 37, "vocab": 50257, "cols": 768, "dtype": "bf16", "train": False},
        # a training step with float32 weights, an odd vocabulary and odd features
        {"name": "loss_ragged", "op": "loss", "tokens": 1001, "vocab": 10007, "cols": 1001, "dtype": "f32", "train": True},
        # a training step of a small model
        {"name": "loss_small", "op": "loss", "tokens": 8192, "vocab": 50257, "cols": 768, "dtype": "bf16", "train": True},
        # and of the 8-billion-parameter one
        {"name": "loss_large", "op": "loss", "tokens": 8192, "vocab": 128256, "cols": 4096, "dtype": "bf16", "train": True},
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm; one in three is made a multiple of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.34 and v > 64:
        v -= v % 64
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["norm", "drop", "embed", "loss", "loss"])
    case = {"op": op, "dtype": rng.choice(["bf16", "f32"])}
    if op == "norm":
        case.update(rows=_log(rng, 1, 16384), cols=_log(rng, 16, 4096), train=rng.choice([True, True, False]))
    elif op == "drop":
        case.update(rows=_log(rng, 1, 16384), cols=_log(rng, 16, 4096), p=rng.choice([0.05, 0.1, 0.25, 0.5]),
                    residual=rng.choice([True, False]))
    elif op == "embed":
        case.update(tokens=_log(rng, 1, 16384), vocab=_log(rng, 256, 128256), cols=_log(rng, 16, 4096),
                    train=rng.choice([True, True, False]))
    else:
        case.update(tokens=_log(rng, 1, 8192), vocab=_log(rng, 256, 128256), cols=_log(rng, 64, 4096),
                    train=rng.choice([True, True, False]))
    return case


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _hidden(g, rows, cols, dtype):
    """Gaussian values with a mean of their own and a few strong channels, as a residual stream has them."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= 1 + 20 * (torch.rand(cols, generator=g, device="cuda") < 0.005)
    x += 0.3 * torch.randn(rows, 1, generator=g, device="cuda")
    return x.to(dtype)


def _words(g, tokens, vocab):
    """Token numbers of a text: the k-th most frequent about as often as 1 / k, spread over the vocabulary."""
    u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(vocab)).long().clamp(1, vocab) - 1
    return rank * 7919 % vocab


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], _dtype(case)
    s = {"case": case, "seed": seed % 1000}
    rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    if op == "norm":
        s["x"] = _hidden(g, case["rows"], case["cols"], dt)
        s["w"], s["b"] = 1 + 0.1 * rnd(case["cols"]), 0.1 * rnd(case["cols"])
    elif op == "drop":
        s["x"] = _hidden(g, case["rows"], case["cols"], dt)
        s["res"] = _hidden(g, case["rows"], case["cols"], dt) if case["residual"] else None
    elif op == "embed":
        s["w"] = (rnd(case["vocab"], case["cols"]) * 0.02).to(dt)
        s["ids"], s["scale"] = _words(g, case["tokens"], case["vocab"]), case["cols"] ** 0.5
    else:
        n, cols = case["tokens"], case["cols"]
        s["w"] = (rnd(case["vocab"], cols) * 0.02).to(dt)
        s["t"] = _words(g, n, case["vocab"])
        # hidden states that lean towards their target's row, as a trained model's do; every tenth token has no target
        lean = s["w"][s["t"]].float()
        s["x"] = (rnd(n, cols) + 6 * lean / lean.norm(dim=1, keepdim=True)).to(dt)
        s["t"] = s["t"].masked_fill(torch.arange(n, device="cuda") % 10 == 9, IGNORE)
    if case.get("train", op == "drop") and op != "loss":
        rows = case["tokens"] if op == "embed" else case["rows"]
        s["dy"] = (rnd(rows, case["cols"]) * 1e-3).to(dt)
    if own:
        from spectral_split_quantized_amd import layer, metis
        metis.init_device()
        if op == "norm":
            s["layer"] = layer.LayerNorm(case["cols"], eps=EPS, weight=s["w"], bias=s["b"])
        elif op == "drop":
            s["layer"] = layer.Dropout(case["p"], seed=s["seed"], layer=LAYER)
            s["layer"].step = STEP
        elif op == "embed":
            s["layer"] = layer.Embedding(case["vocab"], case["cols"], scale=s["scale"], weight=s["w"])
        else:
            s["layer"] = layer.LinearCrossEntropy(case["cols"], case["vocab"], weight=s["w"], ignore_index=IGNORE,
                                                  reduction="mean" if case["train"] else "none")
        if case.get("train", True):
            for k in ("x", "res"):
                if s.get(k) is not None:
                    s[k].requires_grad_(True)
    return s


# ------------------------------------------------------------- plain forms --

def _mulhilo(a, const):
    """High and low words of the 64-bit product of 32-bit words held in int64."""
    lo, hi = (a & 0xFFFF) * const, (a >> 16) * const
    return ((hi + (lo >> 16)) >> 16) & MASK32, ((hi << 16) + lo) & MASK32


def _philox(q, tag, step, seed):
    """The four words of the Philox4x32-10 blocks of counters (q lo, q hi, tag, step)."""
    c0, c1 = q & MASK32, q >> 32
    c2, c3 = torch.full_like(q, tag), torch.full_like(q, step)
    k0, k1 = seed & MASK32, seed >> 32
    for _ in range(10):  # the generator's ten rounds
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    return c0, c1, c2, c3


TAG = LAYER << 16 | OPERAND_X << 12 | ROLE_DROP << 8


def _halves(shape, seed):
    """The 16-bit draws of a matrix's elements in row-major order."""
    n = shape[0] * shape[1]
    words = torch.stack(_philox(torch.arange((n + 7) // 8, device="cuda"), TAG, STEP, seed), 1)
    return torch.stack((words & 0xFFFF, words >> 16), 2).reshape(-1)[:n].reshape(shape)


def _norm(s):
    dt, w, b = s["x"].dtype, s["w"], s["b"]
    x = s["x"].float()
    centred = x - x.mean(1, keepdim=True)
    r = 1 / torch.sqrt(centred.square().mean(1, keepdim=True) + EPS)
    hat = centred * r
    out = {"y": (hat * w + b).to(dt)}
    if s["case"]["train"]:
        dy = s["dy"].float()
        g = dy * w
        out["dx"] = (r * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))).to(dt)
        out["dw"], out["db"] = (dy * hat).sum(0), dy.sum(0)
    return out


def _drop(s):
    dt, t = s["x"].dtype, round(65536 * s["case"]["p"])
    keep = _halves(s["x"].shape, s["seed"]) >= t
    scale = 65536 / (65536 - t)
    y = torch.where(keep, s["x"].float() * scale, 0.0)
    if s["res"] is not None:
        y = y + s["res"].float()
    out = {"y": y.to(dt), "dx": torch.where(keep, s["dy"].float() * scale, 0.0).to(dt)}
    if s["res"] is not None:
        out["dres"] = s["dy"]
    return out


def _embed(s):
    w, ids = s["w"], s["ids"]
    out = {"y": (w[ids].float() * s["scale"]).to(w.dtype)}
    if s["case"]["train"]:
        dw = torch.zeros(w.shape, device="cuda").index_add_(0, ids, s["dy"].float())
        out["dw"] = (dw * s["scale"]).to(w.dtype)
    return out


def _loss(s):
    w, x, t = s["w"].float(), s["x"].float(), s["t"]
    valid = t != IGNORE
    count = valid.sum()
    at = torch.where(valid, t, 0)[:, None]
    z = x @ w.T
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    each = torch.where(valid, (lse - z.gather(1, at))[:, 0], 0.0)
    if not s["case"]["train"]:
        return {"losses": each}
    p = torch.exp(z - lse)
    p.scatter_add_(1, at, torch.full_like(lse, -1.0))
    p *= (valid / count)[:, None]
    return {"loss": (each.double().sum() / count).float(), "dx": (p @ w).to(s["x"].dtype), "dw": (p.T @ x).to(s["w"].dtype)}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"norm": _norm, "drop": _drop, "embed": _embed, "loss": _loss}[op](s)
    m = s["layer"]
    if not case.get("train", True):
        with torch.no_grad():
            return {"losses": m(s["x"], s["t"])} if op == "loss" else {"y": m(s["ids"] if op == "embed" else s["x"])}
    if op == "loss":
        loss = m(s["x"], s["t"])
        dx, dw = torch.autograd.grad(loss, (s["x"], m.weight))
        return {"loss": loss.detach(), "dx": dx, "dw": dw}
    if op == "embed":
        y = m(s["ids"])
        return {"y": y.detach(), "dw": torch.autograd.grad(y, m.weight, s["dy"])[0]}
    if op == "norm":
        y = m(s["x"])
        dx, dw, db = torch.autograd.grad(y, (s["x"], m.weight, m.bias), s["dy"])
        return {"y": y.detach(), "dx": dx, "dw": dw, "db": db}
    if s["res"] is None:
        y = m(s["x"])
        return {"y": y.detach(), "dx": torch.autograd.grad(y, s["x"], s["dy"])[0]}
    y = m(s["x"], s["res"])
    dx, dres = torch.autograd.grad(y, (s["x"], s["res"]), s["dy"])
    return {"y": y.detach(), "dx": dx, "dres": dres}


# -------------------------------------------------------------------- work --

def work(case):
    op, size = case["op"], 2 if case["dtype"] == "bf16" else 4
    train = case.get("train", True)
    if op in ("norm", "drop"):
        n = case["rows"] * case["cols"]
        if op == "norm":
            return {"bytes": n * size * (4 if train else 2) + case["cols"] * 4 * (4 if train else 2), "flops": n * (20 if train else 7)}
        return {"bytes": n * size * (5 if case["residual"] else 4), "flops": n * (3 if case["residual"] else 2)}
    n, v, cols = case["tokens"], case["vocab"], case["cols"]
    if op == "embed":
        each = 8 * n + 2 * n * cols * size
        return {"bytes": each + ((n + v) * cols * size if train else 0), "flops": n * cols * (2 if train else 1)}
    bytes_ = (n + v) * cols * size + 8 * n + 4
    return {"bytes": bytes_ + ((n + v) * cols * size if train else 0), "flops": n * v * (cols * (6 if train else 2) + 4)}


# ------------------------------------------------------- exact values (64 bits) --

def _draws_np(n, tag, step, seed):
    """16-bit draws of n consecutive elements, by the published rounds in 64-bit words."""
    u64 = np.uint64
    ctr = np.zeros((4, (n + 7) // 8), u64)
    ctr[0], ctr[2], ctr[3] = np.arange(ctr.shape[1], dtype=u64), u64(tag), u64(step)
    mask, sh = u64(MASK32), u64(32)
    for r in range(10):
        k0, k1 = u64((seed + r * 0x9E3779B9) & MASK32), u64((r * 0xBB67AE85) & MASK32)
        a, b = ctr[0] * u64(0xD2511F53), ctr[2] * u64(0xCD9E8D57)
        ctr = np.stack(((b >> sh) ^ ctr[1] ^ k0, b & mask, (a >> sh) ^ ctr[3] ^ k1, a & mask))
    return ctr.astype("<u4").T.copy().view("<u2").reshape(-1)[:n]


def _exact_norm(s, train):
    x, w, b = s["x"].detach().double(), s["w"].double(), s["b"].double()
    var, mu = torch.var_mean(x, dim=1, correction=0, keepdim=True)
    sd = (var + EPS) ** 0.5
    hat = (x - mu) / sd
    out = {"y": torch.addcmul(b, hat, w)}
    if train:
        dy = s["dy"].double()
        # the derivative of a vector over its length: what is left across the
        # mean and across hat
        h = dy * w / sd
        across = torch.einsum("ij,ij->i", h, hat) / x.shape[1]
        out["dx"] = h - torch.addcmul((h.sum(dim=1) / x.shape[1]).unsqueeze(1), hat, across.unsqueeze(1))
        out["dw"] = torch.einsum("ij,ij->j", dy, hat)
        out["db"] = dy.sum(dim=0)
    return out


def _exact_drop(s, p):
    x, dy, t = s["x"].detach().double(), s["dy"].double(), int(np.rint(65536 * p))
    draws = torch.from_numpy(_draws_np(x.numel(), TAG, STEP, s["seed"]).astype(np.int32)).cuda().view(x.shape)
    factor = (draws >= t).double() / (1.0 - t / 65536.0)
    out = {"y": x * factor, "dx": dy * factor}
    if s["res"] is not None:
        out["y"] += s["res"].detach().double()
        out["dres"] = dy
    return out


def _exact_embed(s, train):
    w, ids = s["w"].detach().double(), s["ids"]
    out = {"y": torch.index_select(w, 0, ids) * s["scale"]}
    if train:
        order = torch.argsort(ids, stable=True)
        words, counts = torch.unique_consecutive(ids[order], return_counts=True)
        # sums of runs as differences of 64-bit running sums, in blocks of columns
        dw, ends = torch.zeros_like(w), counts.cumsum(0)
        for c in range(0, w.shape[1], 512):
            run_ = s["dy"][order, c:c + 512].double().cumsum(0)
            upto = run_[ends - 1]
            dw[words, c:c + 512] = torch.diff(upto, dim=0, prepend=torch.zeros_like(upto[:1])) * s["scale"]
        out["dw"] = dw
    return out


def _exact_loss(s, train):
    w, x, t = s["w"].detach().double(), s["x"].detach().double(), s["t"]
    rows = torch.nonzero(t != IGNORE)[:, 0]
    losses, dx = torch.zeros(len(t), dtype=torch.float64, device="cuda"), torch.zeros_like(x)
    dw = torch.zeros_like(w) if train else None
    for part in rows.split(1024):
        z, here = x[part] @ w.t(), t[part]
        log_p = torch.log_softmax(z, dim=1)
        place = torch.arange(len(part), device="cuda")
        losses[part] = -log_p[place, here]
        if train:
            slope = log_p.exp_()
            slope[place, here] -= 1.0
            slope /= len(rows)
            dx[part] = slope @ w
            dw.addmm_(slope.t(), x[part])
    return {"loss": losses.sum() / len(rows), "dx": dx, "dw": dw} if train else {"losses": losses}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case["train"])
    if case["op"] == "drop":
        return _exact_drop(s, case["p"])
    return (_exact_embed if case["op"] == "embed" else _exact_loss)(s, case["train"])
