"""The 8-bit linear layer and its weight update: cases, plain forms and exact values.

Operators: per-token and per-channel int8 quantisation, the int8 matrix
product, the serving linear (token scales formed in the call), the training
layer (forward and both gradients), and the AdamW step over many tensors with
32-bit or 8-bit states, with or without clipping by the global gradient norm.

``own`` selects the side: False runs the plain torch forms below, True the
library's calls.
"""

import math
import random

import numpy as np
import torch

own = False

MASK32 = 0xFFFFFFFF
BLOCK = 256              # elements that share one scale in an 8-bit optimizer state
TINY = 2.0 ** -126
LR, BETAS, EPS, DECAY, FIRST_STEP, MAX_NORM = 1e-3, (0.9, 0.999), 1e-8, 0.1, 1000, 1.0
OPERAND_W, OPERAND_D = 1, 3


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a decode batch's activations: one scale per token
        {"name": "quant_tokens", "op": "quant", "rows": 48, "cols": 4096, "dtype": "bf16", "axes": 2, "rounding": "rne"},
        # an output gradient of a training step: both orientations, stochastic rounding
        {"name": "quant_gradient", "op": "quant", "rows": 16384, "cols": 4096, "dtype": "bf16", "axes": 3, "rounding": "sr"},
        # a short ragged batch against an odd-sized projection
        {"name": "gemm_ragged", "op": "gemm", "m": 1001, "n": 2570, "k": 1337, "out": "f32"},
        # the gate projection of an 8-billion-parameter model's MLP, 16384 tokens
        {"name": "gemm_gate", "op": "gemm", "m": 16384, "n": 14336, "k": 4096, "out": "bf16"},
        # serving: one token through the gate projection
        {"name": "linear_token", "op": "linear", "tokens": 1, "cin": 4096, "cout": 14336, "dtype": "bf16"},
        # serving: a ragged decode batch through the down projection
        {"name": "linear_batch", "op": "linear", "tokens": 37, "cin": 14336, "cout": 4096, "dtype": "bf16"},
        # training step of a small model's fused query-key-value projection
        {"name": "layer_small", "op": "layer", "tokens": 1000, "cin": 768, "cout": 2304, "dtype": "f32"},
        # training step of the gate projection
        {"name": "layer_gate", "op": "layer", "tokens": 8192, "cin": 4096, "cout": 14336, "dtype": "bf16"},
        # the update of a small model: many tensors from one element up, clipped
        {"name": "adamw32_many", "op": "adamw", "bits": 32, "tensors": 148, "largest": 1 << 20, "shapes": 1, "clip": True, "rounding": "rne"},
        # the update of one MLP's three projections
        {"name": "adamw32_mlp", "op": "adamw", "bits": 32, "tensors": 3, "largest": 4096 * 14336, "shapes": 0, "clip": False, "rounding": "rne"},
        # the same two with 8-bit states
        {"name": "adamw8_many", "op": "adamw", "bits": 8, "tensors": 148, "largest": 1 << 20, "shapes": 1, "clip": True, "rounding": "rne"},
        {"name": "adamw8_mlp", "op": "adamw", "bits": 8, "tensors": 3, "largest": 4096 * 14336, "shapes": 0, "clip": False, "rounding": "sr"},
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm; one in three is made a multiple of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.34 and v > 64:
        v -= v % 64
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["quant", "gemm", "linear", "layer", "adamw", "adamw"])
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 16384), "cols": _log(rng, 1, 4096), "dtype": rng.choice(["bf16", "f32"]),
                "axes": rng.choice([1, 2, 3]), "rounding": rng.choice(["rne", "sr"])}
    if op == "gemm":
        return {"op": op, "m": _log(rng, 1, 16384), "n": _log(rng, 64, 14336), "k": _log(rng, 64, 4096),
                "out": rng.choice(["f32", "bf16"])}
    if op == "linear":
        return {"op": op, "tokens": _log(rng, 1, 512), "cin": _log(rng, 256, 14336), "cout": _log(rng, 256, 14336),
                "dtype": rng.choice(["bf16", "f32"])}
    if op == "layer":
        return {"op": op, "tokens": _log(rng, 16, 8192), "cin": _log(rng, 64, 4096), "cout": _log(rng, 64, 14336),
                "dtype": rng.choice(["bf16", "f32"])}
    return {"op": op, "bits": rng.choice([8, 32]), "tensors": _log(rng, 1, 300), "largest": _log(rng, 256, 1 << 20),
            "shapes": rng.randrange(1, 1000), "clip": rng.choice([True, False]), "rounding": rng.choice(["rne", "sr"])}


def _sizes(case):
    """Element counts of the tensors of an optimizer case: all alike, or spread from one element up."""
    if not case["shapes"]:
        return [case["largest"]] * case["tensors"]
    rng = random.Random(case["shapes"])
    return [case["largest"]] + [_log(rng, 1, case["largest"]) for _ in range(case["tensors"] - 1)]


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _activations(g, rows, cols, dtype):
    """Gaussian values with a few strong channels, as hidden states have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= 1 + 20 * (torch.rand(cols, generator=g, device="cuda") < 0.005)
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case, "seed": seed % 1000}
    if own:
        from spectral_split_quantized_amd import layer, metis, optim
        metis.init_device()
        s.update(layer=layer, metis=metis, optim=optim)
    if op == "quant":
        s["x"] = _activations(g, case["rows"], case["cols"], _dtype(case["dtype"]))
    elif op == "gemm":
        for name, rows in (("a", case["m"]), ("b", case["n"])):
            s[name], s["s" + name] = _codes(_activations(g, rows, case["k"], torch.float32), 1)
            if own:
                s["q" + name] = metis.I8.from_codes(s[name], s["s" + name])
    elif op == "linear":
        s["x"] = _activations(g, case["tokens"], case["cin"], _dtype(case["dtype"]))
        w = torch.randn(case["cout"], case["cin"], generator=g, device="cuda") * case["cin"] ** -0.5
        s["w"], s["sw"] = _codes(w, 1)
        if own:
            s["qw"] = metis.I8.from_codes(s["w"], s["sw"])
    elif op == "layer":
        dt = _dtype(case["dtype"])
        s["x"] = _activations(g, case["tokens"], case["cin"], dt).requires_grad_(own)
        s["w"] = torch.randn(case["cin"], case["cout"], generator=g, device="cuda") * case["cin"] ** -0.5
        s["dy"] = (torch.randn(case["tokens"], case["cout"], generator=g, device="cuda") * 1e-3).to(dt)
        if own:
            s["lin"] = layer.Int8Linear(case["cin"], case["cout"], rounding="sr", seed=s["seed"], weight=s["w"])
            s["lin"].step = 5
    else:
        # every buffer is one allocation in which each tensor starts on a block, as a sharded trainer keeps them
        sizes = _sizes(case)
        counts = [-(-n // BLOCK) for n in sizes]
        fill = _filled(sizes, counts)
        rnd = lambda: torch.randn(sum(counts), BLOCK, generator=g, device="cuda") * fill  # noqa: E731
        s["t"], s["counts"] = FIRST_STEP, counts
        s["p"], s["g"] = rnd() * 0.02, rnd() * 1e-3
        spread = torch.exp(2 * rnd()) * fill
        m, r = rnd() * 3e-4 * spread, 1e-3 * spread
        if case["bits"] == 32:
            s["m"], s["v"] = m, r.square()
        else:
            (s["m"], s["ms"]), (s["v"], s["vs"]) = _encode(m, False), _encode(r, True)
        if own:
            views = {k: _views(s[k], sizes, counts) for k in ("p", "g")}
            views.update({k: _views(v, sizes, counts) for k, v in _adamw_outputs(s, {}).items() if k in ("m", "v")})
            for p, gr in zip(views["p"], views["g"]):
                p.requires_grad_(True)
                p.grad = gr
            opt = optim.AdamW(views["p"], lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, state_bits=case["bits"],
                              min_8bit_size=0, rounding=case["rounding"], seed=s["seed"],
                              max_norm=MAX_NORM if case["clip"] else None)
            for i, p in enumerate(views["p"]):
                opt.state[p] = {"step": FIRST_STEP, "exp_avg": views["m"][i], "exp_avg_sq": views["v"][i]}
            if case["bits"] == 8:
                for p, ms, vs in zip(views["p"], s["ms"].split(counts), s["vs"].split(counts)):
                    opt.state[p].update(exp_avg_scale=ms, exp_avg_sq_scale=vs)
            s["opt"] = opt
    return s


# ------------------------------------------------------------- plain forms --

def _mulhilo(a, const):
    """High and low words of the 64-bit product of 32-bit words held in int64."""
    lo, hi = (a & 0xFFFF) * const, (a >> 16) * const
    return ((hi + (lo >> 16)) >> 16) & MASK32, ((hi << 16) + lo) & MASK32


def _philox(q, tag, step, seed):
    """The four words of the Philox4x32-10 blocks of counters (q lo, q hi, tag, step)."""
    c0, c1 = q & MASK32, q >> 32
    c2, c3 = torch.zeros_like(q) + tag, torch.full_like(q, step)
    k0, k1 = seed & MASK32, seed >> 32
    for _ in range(10):  # the generator's ten rounds
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    return c0, c1, c2, c3


def _uniform16(rows, cols, tag, step, seed):
    """The 16-bit draws of a matrix's elements in row-major order, times 2^-16."""
    n = rows * cols
    words = torch.stack(_philox(torch.arange((n + 7) // 8, device="cuda"), tag, step, seed), 1)
    halves = torch.stack((words & 0xFFFF, words >> 16), 2).reshape(-1)[:n]
    return halves.reshape(rows, cols).float() * 2.0 ** -16


def _codes(x, axis, u=None):
    """int8 codes with K along `axis` (0: transposed) and one scale per line."""
    x = x.float()
    x, u = (x, u) if axis else (x.T, None if u is None else u.T)
    scale = (x.abs().amax(1).double() / 127).float().clamp_min(TINY)
    y = x * (1 / scale.double()).float()[:, None]
    c = torch.round(y) if u is None else torch.floor(y) + (u < y - torch.floor(y))
    return c.clamp(-127, 127).to(torch.int8), scale


def _product(a, sa, b, sb, dtype=torch.float32):
    return ((a.float() @ b.float().T) * sa[:, None] * sb).to(dtype)


def _encode(x, positive, half=None):
    """E4M3 codes of blocks (rows of x) with power-of-two scales; a positive x never becomes zero where `positive`."""
    amax = x.abs().amax(1)
    e = ((amax.view(torch.int32) >> 23) - 127 - 7).clamp_min(-126)
    scale = ((e + 127) << 23).view(torch.float32)
    y = x.abs() / scale[:, None]                                     # exact: a power of two
    low = y < 2.0 ** -6
    bits = torch.where(low, y + 2.0 ** -6, y).view(torch.int32)
    bits = bits + (0x7FFFF + ((bits >> 20) & 1) if half is None else half << 4)
    c = (bits >> 20) - torch.where(low, 968, 960)
    c = torch.where((x != 0) & (c == 0), 1, c) if positive else c | torch.where(x < 0, 128, 0)
    return c.to(torch.uint8), scale


def _filled(sizes, counts):
    """1 where a block's place holds an element of its tensor, 0 behind the tensor's end."""
    n = torch.tensor(sizes, device="cuda").repeat_interleave(torch.tensor(counts, device="cuda"))
    return (_places(counts) < n[:, None]).float()


def _places(counts):
    """Each place's index within its tensor."""
    c = torch.tensor(counts, device="cuda")
    first = (c.cumsum(0) - c).repeat_interleave(c)
    return ((torch.arange(first.numel(), device="cuda") - first) * BLOCK)[:, None] + torch.arange(BLOCK, device="cuda")


def _views(buffer, sizes, counts):
    """The tensors in a buffer of blocks."""
    return [part.view(-1)[:n] for part, n in zip(buffer.split(counts), sizes)]


def _halves(counts, step, seed):
    """The 32-bit draw of each place, as its low and its high half."""
    tag = torch.tensor([(i & 0xFFFF) << 16 | OPERAND_W << 12 | 6 << 8 for i in range(len(counts))], device="cuda")
    tag = tag.repeat_interleave(torch.tensor(counts, device="cuda"))
    q = _places(counts)[:, ::4] >> 2
    w = torch.stack(_philox(q, tag[:, None], step, seed), 2).view(-1, BLOCK)
    return (w & 0xFFFF).int(), (w >> 16).int()


def _adamw(s):
    case, gr, out = s["case"], s["g"], {}
    s["t"] += 1
    (b1, b2), eight = BETAS, case["bits"] == 8
    if case["clip"]:
        norm = gr.double().square().sum().sqrt()
        out["norm"] = norm.float()
        gr = gr * (MAX_NORM / (norm + 1e-6)).clamp_max(1.0).float()
    m = s["m"].view(torch.float8_e4m3fn).float() * s["ms"][:, None] if eight else s["m"]
    v = (s["v"].view(torch.float8_e4m3fn).float() * s["vs"][:, None]).square() if eight else s["v"]
    m = b1 * m + (1 - b1) * gr
    v = b2 * v + (1 - b2) * gr * gr
    r = v.double().sqrt().float()
    step = m / (r / math.sqrt(1 - b2 ** s["t"]) + EPS)
    s["p"].copy_(s["p"] * (1 - LR * DECAY) - LR / (1 - b1 ** s["t"]) * step)
    if eight:
        low, high = _halves(s["counts"], s["t"], s["seed"]) if case["rounding"] == "sr" else (None, None)
        for name, x, half in (("m", m, low), ("v", r, high)):
            codes, scale = _encode(x, name == "v", half)
            s[name].copy_(codes)
            s[name + "s"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_outputs(s, out)


def _adamw_outputs(s, out):
    """The updated buffers themselves; 8-bit states as the E4M3 values that they hold, next to their blocks' scales."""
    out["p"] = s["p"].detach()
    if s["case"]["bits"] == 8:
        out.update(m=s["m"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn), ms=s["ms"], vs=s["vs"])
    else:
        out.update(m=s["m"], v=s["v"])
    return out


def _layer(s):
    x, w, dy = s["x"].detach(), s["w"], s["dy"]
    u = _uniform16(*dy.shape, OPERAND_D << 12, 5, s["seed"])
    y = _product(*_codes(x, 1), *_codes(w, 0), x.dtype)
    dx = _product(*_codes(dy, 1, u), *_codes(w, 1), x.dtype)
    dw = _product(*_codes(x, 0), *_codes(dy, 0, u))
    return {"y": y, "dx": dx, "dw": dw}


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "quant":
        if own:
            metis = s["metis"]
            q = metis.int8_quantize(s["x"], case["axes"], rounding=metis.SR if case["rounding"] == "sr" else metis.RNE,
                                    seed=s["seed"], tag=OPERAND_D << 12, step=5)
            got = {"0": q.ax0, "1": q.ax1}
            return {k + a: t for a, o in got.items() if o is not None for k, t in (("c", o.codes[:, :o.k_len]), ("s", o.scales))}
        u = _uniform16(*s["x"].shape, OPERAND_D << 12, 5, s["seed"]) if case["rounding"] == "sr" else None
        got = {a: _codes(s["x"], int(a), u) for a in ("0", "1") if case["axes"] & (1 + int(a))}
        return {k + a: t for a, o in got.items() for k, t in (("c", o[0]), ("s", o[1]))}
    if op == "gemm":
        dt = _dtype(case["out"])
        if own:
            return s["metis"].int8_gemm(s["qa"], s["qb"], out_dtype=dt)
        return _product(s["a"], s["sa"], s["b"], s["sb"], dt)
    if op == "linear":
        if own:
            return s["metis"].int8_linear(s["x"], s["qw"])
        return _product(*_codes(s["x"], 1), s["w"], s["sw"], s["x"].dtype)
    if op == "layer":
        if not own:
            return _layer(s)
        s["x"].grad = s["lin"].weight.grad = None
        y = s["lin"](s["x"])
        y.backward(s["dy"])
        return {"y": y.detach(), "dx": s["x"].grad, "dw": s["lin"].weight.grad}
    if not own:
        return _adamw(s)
    s["opt"].step()
    return _adamw_outputs(s, {"norm": s["opt"].grad_norm} if case["clip"] else {})


# -------------------------------------------------------------------- work --

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "quant":
        n, lines = case["rows"] * case["cols"], {1: case["cols"], 2: case["rows"], 3: case["rows"] + case["cols"]}[case["axes"]]
        sides = 2 if case["axes"] == 3 else 1
        return {"bytes": n * (size[case["dtype"]] + sides) + 4 * lines, "flops": n * (1 + 2 * sides)}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * (k + 4) + m * n * size[case["out"]], "flops": 2 * m * n * k}
    if op == "linear":
        t, i, o = case["tokens"], case["cin"], case["cout"]
        return {"bytes": o * (i + 4) + t * (i + o) * size[case["dtype"]], "flops": 2 * t * i * o}
    if op == "layer":
        t, i, o = case["tokens"], case["cin"], case["cout"]
        return {"bytes": 2 * t * (i + o) * size[case["dtype"]] + 2 * i * o * 4, "flops": 6 * t * i * o}
    sizes = _sizes(case)
    n, blocks = sum(sizes), sum(-(-k // BLOCK) for k in sizes)
    return {"bytes": 28 * n if case["bits"] == 32 else 16 * n + 16 * blocks, "flops": 15 * n}


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
    return ctr.astype("<u4").T.copy().view("<u2").reshape(-1)[:n].astype(np.float64) / 65536


def _values(x, draws=None):
    """The 64-bit values that int8 rows stand for: the format's definition, its
    binary32 steps (scale, reciprocal, scaled value) rounded where it says."""
    x = x.double()
    scale = (x.abs().max(dim=1).values / 127.0).float().double()
    scale = torch.maximum(scale, torch.full_like(scale, TINY))
    scaled = (x * (1.0 / scale).float().double().unsqueeze(1)).float().double()
    if draws is None:
        whole = scaled.round()
    else:
        whole = scaled.floor()
        whole = whole + (draws < (scaled - whole)).double()
    return whole.clip(-127.0, 127.0) * scale.unsqueeze(1)


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "quant":
        x = s["x"].detach().double().abs()
        out = {}
        if case["axes"] & 1:
            out.update(c0=None, s0=(x.max(dim=0).values / 127.0).clip(min=TINY))
        if case["axes"] & 2:
            out.update(c1=None, s1=(x.max(dim=1).values / 127.0).clip(min=TINY))
        return out
    if op == "gemm":
        return (s["a"].double() * s["sa"].double().unsqueeze(1)) @ (s["b"].double() * s["sb"].double().unsqueeze(1)).t()
    if op == "linear":
        return _values(s["x"].detach()) @ (s["w"].double() * s["sw"].double().unsqueeze(1)).t()
    if op == "layer":
        x, w, dy = s["x"].detach(), s["w"], s["dy"]
        draws = torch.from_numpy(_draws_np(dy.numel(), OPERAND_D << 12, 5, s["seed"])).cuda().view(dy.shape)
        out = {"y": _values(x) @ _values(w.t()).t(), "dx": _values(dy, draws) @ _values(w).t()}
        out["dw"] = _values(x.t()) @ _values(dy.t(), draws.t()).t()
        return out
    t = FIRST_STEP + 1
    grad, p = s["g"].detach().double(), s["p"].detach().double()
    m, v = s["m"].detach(), s["v"].detach()
    out = {}
    if case["clip"]:
        out["norm"] = torch.linalg.vector_norm(grad)
        grad = grad * min(1.0, MAX_NORM / (float(out["norm"]) + 1e-6))
    if case["bits"] == 8:
        m = m.view(torch.float8_e4m3fn).double() * s["ms"].double().unsqueeze(1)
        v = (v.view(torch.float8_e4m3fn).double() * s["vs"].double().unsqueeze(1)) ** 2
    else:
        m, v = m.double(), v.double()
    m = m * BETAS[0] + grad * (1.0 - BETAS[0])
    v = v * BETAS[1] + grad ** 2 * (1.0 - BETAS[1])
    away = (m / (1.0 - BETAS[0] ** t)) / ((v / (1.0 - BETAS[1] ** t)).sqrt() + EPS)
    out["p"] = p - LR * DECAY * p - LR * away
    if case["bits"] == 8:
        out.update(m=None, v=None, ms=None, vs=None)
    else:
        out.update(m=m, v=v)
    return out
