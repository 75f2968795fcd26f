"""A PyTorch linear layer whose three GEMMs run through the Metis path.

"Metis: Training LLMs with FP4 Quantization" (整体框架): the weight W, the
activation X and the output gradient D of a linear layer are each split into
a low-rank part and a residual (关键设计 1), quantised to NVFP4 (W4A4G4), and
every GEMM of the forward and backward pass -- Y = X W, dX = D W^T,
dW = X^T D -- is evaluated through the split.  The right factor of each
operand is cached and re-sketched every ``refresh`` steps (关键设计 3).

This module is marshalling only: ``metis.prepare_operand`` and
``metis.gemm_fwd`` / ``metis.gemm_bwd`` run every step in the HIP library.
The weight is stored as in the pages' notation, ``in_features x
out_features`` (Y = X W), as an fp32 master.
"""

import weakref

import torch

from . import metis

__all__ = ["MetisLinear", "Int8Linear", "Int8Frozen", "set_step"]


class _MetisLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, mod):
        lead = x.shape[:-1]
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        # X is the K-along-columns operand of Y = X W and the K-along-rows
        # operand of dW = X^T D; W the reverse (Y = X W, then dX = D W^T)
        both = metis.AXIS0 | metis.AXIS1
        qx = metis.prepare_operand(x2, mod.cfg, True, mod.tags["X"], mod.step, mod._factors("X", x2), both)
        qw = metis.prepare_operand(w.detach(), mod.cfg, False, mod.tags["W"], mod.step, mod._factors("W", w), both)
        y = metis.gemm_fwd(qx, qw)
        ctx.mod, ctx.qx, ctx.qw, ctx.lead = mod, qx, qw, lead
        ctx.x_dtype = x.dtype
        mod.last = {"X": qx, "W": qw}
        return y.reshape(*lead, w.shape[1])

    @staticmethod
    def backward(ctx, dy):
        mod = ctx.mod
        d2 = dy.reshape(-1, dy.shape[-1]).contiguous().float()
        both = metis.AXIS0 | metis.AXIS1
        qd = metis.prepare_operand(d2, mod.cfg, True, mod.tags["D"], mod.step, mod._factors("D", d2), both)
        want_dx, want_dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        dx, dw = metis.gemm_bwd(qd, ctx.qw, ctx.qx, want_dx=want_dx, want_dw=want_dw)
        mod.last["D"] = qd
        gx = dx.reshape(*ctx.lead, dx.shape[1]).to(ctx.x_dtype) if want_dx else None
        return gx, dw if want_dw else None, None


class MetisLinear(torch.nn.Module):
    """y = x W (no bias) with W, X and the output gradient quantised through
    the spectral split.

    ``k``: rank of the split; ``s``: oversampling of the sketch; ``l_k``:
    rows sampled from X and D for the sketch (W is not sampled); ``refresh``:
    steps between re-sketches; ``rounding``: "sr" (the pages' default) or
    "rne"; ``seed`` and ``layer`` select the Philox streams.  The caller sets
    the training step with :func:`set_step` (a factor sketched at step t is
    reused while step - t < refresh).  Dimensions must be multiples of 16."""

    def __init__(self, in_features, out_features, k, s=8, l_k=0, refresh=8, rounding="sr", seed=0, layer=0,
                 device="cuda", weight=None):
        super().__init__()
        if weight is None:
            weight = torch.empty(in_features, out_features, dtype=torch.float32, device=device)
            torch.nn.init.normal_(weight, std=in_features ** -0.5)
        if tuple(weight.shape) != (in_features, out_features):
            raise ValueError("weight must be in_features x out_features")
        self.weight = torch.nn.Parameter(weight.to(device=device, dtype=torch.float32).contiguous())
        self.k = k
        self.cfg = metis.make_config(k=k, s=s, l_k=l_k, refresh=refresh,
                                     rounding=metis.SR if rounding == "sr" else metis.RNE, seed=seed)
        self.tags = {"X": metis.make_tag(layer, metis.OPERAND_X),
                     "W": metis.make_tag(layer, metis.OPERAND_W),
                     "D": metis.make_tag(layer, metis.OPERAND_D)}
        self.step = 0
        self.factors = {}
        self.last = {}

    def _factors(self, name, m):
        f = self.factors.get(name)
        if f is None or (f.rows, f.cols) != tuple(m.shape):
            f = metis.Factors(m.shape[0], m.shape[1], self.k, m.device)
            self.factors[name] = f
        return f

    def forward(self, x):
        return _MetisLinearFn.apply(x, self.weight, self)


def _rows(x):
    """x as a matrix of its last dimension's rows, row-major (a copy where it is not)."""
    x = x.reshape(-1, x.shape[-1])
    rows, cols = x.shape
    return x if (cols <= 1 or x.stride(1) == 1) and (rows <= 1 or x.stride(0) >= cols) else x.contiguous()


_EAGER = weakref.WeakSet()  # nodes of Int8Linear recorded outside a capture, while their graphs live


def _capturing(t):
    return t.is_cuda and torch.cuda.is_current_stream_capturing()


def _product(a, b, dtype):
    """A-hat B-hat^T of two int8 operands.  Lines longer than a product's int32
    sums allow are taken in runs, whose binary32 products are added."""
    if a.k_len <= metis.INT8_MAX_K:
        return metis.int8_gemm(a, b, out_dtype=dtype)
    run = metis.INT8_MAX_K // 128 * 128
    total = None
    for k in range(0, a.k_len, run):
        n = min(run, a.k_len - k)
        cut = [metis.I8.wrap(q.codes[:, k:k + metis.int8_pitch(n)].contiguous(), q.scales, n) for q in (a, b)]
        part = metis.int8_gemm(*cut, out_dtype=torch.float32)
        total = part if total is None else total.add_(part)
    return total.to(dtype)


class _Int8LinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, mod, record):
        # needs_input_grad says nothing of torch.no_grad(): record is the
        # caller's grad mode (inside a forward it is always off)
        need_x, need_w = (record and need for need in ctx.needs_input_grad[:2])
        capturing = False
        if need_x or need_w:
            capturing = _capturing(x)
            mod._watch(ctx, [id(t) for t, need in ((x, need_x), (w, need_w)) if need and t.is_leaf], capturing)
        # the same orientations as above: X along both axes (Y and dW), W
        # along both (Y and dX); an orientation whose product is not wanted is
        # left out
        qx = metis.int8_quantize(_rows(x), metis.AXIS1 | (metis.AXIS0 if need_w else 0))
        qw = metis.int8_quantize(w, metis.AXIS0 | (metis.AXIS1 if need_x else 0))
        y = _product(qx.ax1, qw.ax0, x.dtype)
        q0, q1 = qx.ax0, qw.ax1
        ctx.save_for_backward(q0 and q0.codes, q0 and q0.scales, q1 and q1.codes, q1 and q1.scales)
        ctx.lead, ctx.x_dtype, ctx.w_shape = x.shape[:-1], x.dtype, w.shape
        ctx.rounding, ctx.seed, ctx.tag = mod.rounding, mod.seed, mod.tags["D"]
        ctx.step, ctx.count = mod.step, mod._captured_count() if capturing else None
        return y.reshape(*ctx.lead, w.shape[1])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        need_x, need_w = ctx.needs_input_grad[:2]
        d2 = _rows(dy)
        dx = dw = None
        if d2.shape[0] == 0:  # no tokens: sums over nothing
            dx = dy.new_zeros((*ctx.lead, ctx.w_shape[0]), dtype=ctx.x_dtype) if need_x else None
            dw = dy.new_zeros(ctx.w_shape, dtype=torch.float32) if need_w else None
            return dx, dw, None, None
        xc, xs, wc, ws = ctx.saved_tensors
        qd = metis.int8_quantize(d2, (metis.AXIS1 if need_x else 0) | (metis.AXIS0 if need_w else 0),
                                 rounding=ctx.rounding, seed=ctx.seed, tag=ctx.tag, step=ctx.step, step_count=ctx.count)
        if need_x:
            dx = _product(qd.ax1, metis.I8.wrap(wc, ws, ctx.w_shape[1]), ctx.x_dtype).reshape(*ctx.lead, ctx.w_shape[0])
        if need_w:
            dw = _product(metis.I8.wrap(xc, xs, d2.shape[0]), qd.ax0, torch.float32)
        return dx, dw, None, None


class Int8Linear(torch.nn.Module):
    """y = x W (no bias) with all three products in int8: X, W and the output
    gradient D carry one scale per token or channel, along the axis that each
    product reduces over.

    X and W are rounded to nearest, D stochastically (``rounding`` "sr", the
    default, with the draws of ``seed``, ``layer`` and the step that
    :func:`set_step` sets) or to nearest ("rne").  Passes captured into a graph
    read the step on the GPU: set it between replays, on their stream, and a
    replay takes its draws (until then, those of the capture's step).  Recording in a capture is refused while a graph
    from outside it lives (so with torch.cuda.make_graphed_callables, which
    keeps its last warm-up pass).  x is bfloat16 or float32; y and its gradient have
    x's type, the weight (``in_features x out_features``) and its gradient are
    float32.  A product over more than 131071 (tokens, for the weight's
    gradient) is taken in runs of codes, whose binary32 products are added; the
    scales are those of whole lines.  ``frozen()`` gives the serving form, with the weight quantised
    once."""

    def __init__(self, in_features, out_features, rounding="sr", seed=0, layer=0, device="cuda", weight=None):
        super().__init__()
        if rounding not in ("sr", "rne"):
            raise ValueError("rounding must be 'sr' or 'rne', got %r" % (rounding,))
        if weight is None:
            weight = torch.empty(in_features, out_features, dtype=torch.float32, device=device)
            torch.nn.init.normal_(weight, std=in_features ** -0.5)
        if tuple(weight.shape) != (in_features, out_features):
            raise ValueError("weight must be in_features x out_features")
        self.weight = torch.nn.Parameter(weight.to(device=device, dtype=torch.float32).contiguous())
        self.rounding = metis.SR if rounding == "sr" else metis.RNE
        self.seed, self._step, self._count = seed, 0, None
        self.tags = {"D": metis.make_tag(layer, metis.OPERAND_D)}
        self._make_count()

    @property
    def step(self):
        """The training step, which selects the draws."""
        return self._step

    @step.setter
    def step(self, step):
        if self._replayed:
            if _capturing(self._count):
                raise RuntimeError("set the step outside the capture: replays read the one that is set then")
            self._count.fill_(step)
        self._step = step

    def _make_count(self):
        # the step on the weight's GPU, for captured passes: -1 until it is set
        # after the first of them.  The same memory for as long as the weight
        # stays there.
        if self._count is not None and self._count.device == self.weight.device:
            return
        self._count, self._replayed = None, False
        if self.rounding == metis.SR and self.weight.is_cuda:
            with torch.inference_mode(False):
                self._count = torch.full((), -1, dtype=torch.int64, device=self.weight.device)

    def _captured_count(self):
        self._replayed = self._count is not None
        return self._count

    def _apply(self, fn, recurse=True):
        super()._apply(fn, recurse)
        self._make_count()
        return self

    @property
    def _eager(self):
        """This layer's nodes of graphs from outside a capture that live."""
        return [c for c in _EAGER if c.layer() is self]

    def _watch(self, ctx, leaves, capturing):
        """Refuses to record a graph in a capture while one from outside it
        lives, of this layer or of another with the same weight or input: both
        would accumulate a leaf's gradient through one node, which belongs to
        the other's stream, and joining that stream from a capture ends the
        process.  (A living graph holds its leaves, so their ids are theirs.)"""
        if not capturing:
            ctx.layer, ctx.leaves = weakref.ref(self), leaves
            _EAGER.add(ctx)
        elif any(c.layer() is self or any(i in c.leaves for i in leaves) for c in _EAGER):
            raise RuntimeError("a graph of this layer from outside the capture is alive, or one with the same weight or "
                               "input: drop its outputs first")

    def __getstate__(self):
        state = super().__getstate__() if hasattr(super(), "__getstate__") else self.__dict__
        return {k: v for k, v in state.items() if k != "_count"}

    def __setstate__(self, state):
        state = dict(state)
        state.setdefault("_step", state.pop("step", 0))  # "step": saved before it was on the GPU too
        super().__setstate__(state)
        self._count = None
        self._make_count()

    def forward(self, x):
        if x.shape[-1] != self.weight.shape[0]:
            raise ValueError("x has %d features, the layer %d" % (x.shape[-1], self.weight.shape[0]))
        return _Int8LinearFn.apply(x, self.weight, self, torch.is_grad_enabled())

    def frozen(self):
        """The serving form of this layer with its present weight."""
        with torch.no_grad():
            return Int8Frozen(metis.int8_quantize(self.weight, metis.AXIS0).ax0)


class Int8Frozen(torch.nn.Module):
    """y = x W for serving, W held as int8 with one scale per output channel;
    the tokens of x are quantised in the call.  At most 131071 inputs.  No
    gradients."""

    def __init__(self, w):
        super().__init__()
        self.k_len = w.k_len
        self.register_buffer("codes", w.codes)
        self.register_buffer("scales", w.scales)

    def _apply(self, fn, recurse=True):
        scales = self.scales
        super()._apply(fn, recurse)
        if self.scales.dtype != torch.float32:  # the format's, whatever type the model takes
            self.scales = scales.to(self.scales.device)
        return self

    def get_extra_state(self):
        """The number of inputs, which the padded codes do not tell."""
        return torch.tensor(self.k_len)

    def set_extra_state(self, state):
        pass  # compared before anything is loaded

    def _load_from_state_dict(self, state_dict, prefix, local_metadata, strict, missing_keys, unexpected_keys, error_msgs):
        key, codes = prefix + "_extra_state", state_dict.get(prefix + "codes")
        if key in state_dict:
            k_len = int(state_dict[key])
        else:  # saved without it: codes behind this layer's inputs must be the padding's zeros
            k_len = self.k_len if codes is None or not codes[:, self.k_len:].any() else "more"
        if k_len != self.k_len:
            error_msgs.append("size mismatch for %scodes: a layer of %s inputs, here %d" % (prefix, k_len, self.k_len))
            return
        super()._load_from_state_dict(state_dict, prefix, local_metadata, strict, missing_keys, unexpected_keys, error_msgs)
        if key in missing_keys:
            missing_keys.remove(key)

    @torch.no_grad()
    def forward(self, x):
        w = metis.I8.wrap(self.codes, self.scales, self.k_len)
        y = metis.int8_linear(_rows(x), w)
        return y.reshape(*x.shape[:-1], w.outer)


def set_step(model, step):
    """Set the training step of every MetisLinear and Int8Linear in ``model``."""
    for m in model.modules():
        if isinstance(m, (MetisLinear, Int8Linear)):
            m.step = step
