"""PyTorch layers on the library: linear layers whose three GEMMs run through
the Metis path or in int8, and what stands around them in a language model
(layer norm, dropout, embedding, the loss over the vocabulary).

"Metis: Training LLMs with FP4 Quantization" (整体框架): the weight W, the
activation X and the output gradient D of a linear layer are each split into
a low-rank part and a residual (关键设计 1), quantised to NVFP4 (W4A4G4), and
every GEMM of the forward and backward pass -- Y = X W, dX = D W^T,
dW = X^T D -- is evaluated through the split.  The right factor of each
operand is cached and re-sketched every ``refresh`` steps (关键设计 3).

The layers around the linear ones have first derivatives in reverse mode;
second ones, forward mode, torch.func's transforms and tracing raise
(torch.compile leaves their calls out of its graphs).

This module is marshalling only: ``metis.prepare_operand`` and
``metis.gemm_fwd`` / ``metis.gemm_bwd`` run every step in the HIP library, as
do the calls of the other layers.
The weight is stored as in the pages' notation, ``in_features x
out_features`` (Y = X W), as an fp32 master.
"""

import ctypes
import weakref

import torch

from . import metis

__all__ = ["MetisLinear", "Int8Linear", "Int8Frozen", "LayerNorm", "Dropout", "Embedding", "LinearCrossEntropy", "set_step"]


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


def _refuse_alive(leaves, layer=None):
    """Refuses to record a graph in a capture while one from outside it
    lives, of this layer or with one of the same leaves: both would accumulate
    a leaf's gradient through one node, which belongs to the other's stream,
    and joining that stream from a capture ends the process.  (A living graph
    holds its leaves, so their ids are theirs.)"""
    ids = [id(t) for t in leaves]
    if any((layer is not None and c.layer() is layer) or any(i in c.leaves for i in ids) for c in _EAGER) \
            or (_ext is not None and any(_ext.alive(t) for t in leaves)):  # (not loaded: it has no graphs)
        raise RuntimeError("a graph of this layer from outside the capture is alive, or one with the same weight or "
                           "input: drop its outputs first")


def _watch(ctx, layer, leaves, capturing):
    if capturing:
        _refuse_alive(leaves, layer)
    else:
        ctx.layer, ctx.leaves = weakref.ref(layer), [id(t) for t in leaves]
        _EAGER.add(ctx)


_ext = None


def _layers():
    """The extension that holds the nodes of the layers around the linear ones
    (raises if it has not been built)."""
    global _ext
    if _ext is None:
        try:
            from . import _layers as ext
        except ImportError as e:
            raise ImportError("_layers.so cannot be loaded (%s); run python -m spectral_split_quantized_amd.build" % e) from e
        lib = metis.load()
        names = ("last_error", "layernorm_fwd", "layernorm_bwd_workspace", "layernorm_bwd", "dropout", "embedding_fwd",
                 "embedding_bwd_workspace", "embedding_bwd", "cross_entropy_workspace", "cross_entropy_fwd", "cross_entropy_bwd")
        ext.init([ctypes.cast(getattr(lib, "metis_" + n), ctypes.c_void_p).value for n in names], metis.MetisError, _refuse_alive)
        _ext = ext
    return _ext


class _Stepped(torch.nn.Module):
    """The training step, which selects a layer's draws: ``step``, and the same
    on the GPU for passes captured into a graph, which read it there."""

    def _count_device(self):
        """The GPU that the count lives on, or None."""
        raise NotImplementedError

    def _init_step(self):
        self._step, self._count = 0, None
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
        # -1 until the step is set after the first captured pass.  The same
        # memory for as long as the layer stays on its GPU.
        device = self._count_device()
        if self._count is not None and self._count.device == device:
            return
        self._count, self._replayed = None, False
        if device is not None:
            with torch.inference_mode(False):
                self._count = torch.full((), -1, dtype=torch.int64, device=device)

    def _captured_count(self):
        self._replayed = self._count is not None
        return self._count

    def _apply(self, fn, recurse=True):
        super()._apply(fn, recurse)
        self._make_count()
        return self

    def __getstate__(self):
        state = super().__getstate__() if hasattr(super(), "__getstate__") else self.__dict__
        return {k: v for k, v in state.items() if k != "_count"}

    def __setstate__(self, state):
        state = dict(state)
        state.setdefault("_step", state.pop("step", 0))  # "step": saved before it was on the GPU too
        super().__setstate__(state)
        self._count = None
        self._make_count()


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
            _watch(ctx, mod, [t for t, need in ((x, need_x), (w, need_w)) if need and t.is_leaf], capturing)
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


class Int8Linear(_Stepped):
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
        self.seed = seed
        self.tags = {"D": metis.make_tag(layer, metis.OPERAND_D)}
        self._init_step()

    def _count_device(self):
        return self.weight.device if self.rounding == metis.SR and self.weight.is_cuda else None

    @property
    def _eager(self):
        """This layer's nodes of graphs from outside a capture that live."""
        return [c for c in _EAGER if c.layer() is self]

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


# ------------------------------------------------ around the linear layers --

def _parameter(weight, device):
    """A layer's parameter: a Parameter as it is (shared between layers), a
    tensor as a new one."""
    return weight if isinstance(weight, torch.nn.Parameter) else torch.nn.Parameter(weight.to(device).contiguous())


class LayerNorm(torch.nn.Module):
    """Layer norm over the last dimension, with a weight and a bias (``affine``
    False: without).  x is bfloat16 or float32, y and the gradient of x have
    its type, the parameters and their gradients theirs (float32 unless
    ``dtype`` or given tensors say otherwise).  Sums are in binary32."""

    def __init__(self, features, eps=1e-5, affine=True, weight=None, bias=None, device="cuda", dtype=torch.float32):
        super().__init__()
        self.features, self.eps = features, eps
        if not affine:
            if weight is not None or bias is not None:
                raise ValueError("a layer norm without parameters takes no weight and no bias")
            self.weight = self.bias = None
            return
        if weight is None:
            weight = torch.ones(features, dtype=dtype if bias is None else bias.dtype, device=device)
        if bias is None:
            bias = torch.zeros(features, dtype=weight.dtype, device=device)
        if tuple(weight.shape) != (features,) or tuple(bias.shape) != (features,) or weight.dtype != bias.dtype:
            raise ValueError("weight and bias must be %d values of one type" % features)
        self.weight, self.bias = _parameter(weight, device), _parameter(bias, device)

    def forward(self, x):
        if x.shape[-1] != self.features:
            raise ValueError("x has %d features, the layer %d" % (x.shape[-1], self.features))
        return _layers().layer_norm(x, self.weight, self.bias, self.eps)


class Dropout(_Stepped):
    """x with each value dropped with probability ``p`` (to the nearest
    multiple of 2^-16) and the others scaled to keep the mean, plus
    ``residual`` if one is given.  The mask is never stored: the backward pass
    draws it again.

    The draws are those of ``seed``, ``layer`` and the step that
    :func:`set_step` sets, at the value's row-major position; a layer that runs
    twice in a step draws the same mask twice, so each place of a model has a
    Dropout with a ``layer`` number of its own.  Passes captured into a graph
    read the step on the GPU, as Int8Linear's do: set it between replays, on
    their stream.  In eval mode, or with p = 0, nothing is dropped.  x and the
    residual are bfloat16 or float32, of one type and shape."""

    def __init__(self, p=0.1, seed=0, layer=0, device="cuda"):
        super().__init__()
        if not 0 <= p <= 1:
            raise ValueError("p must lie in [0, 1], got %r" % (p,))
        self.p, self.seed, self.tag = p, seed, metis.make_tag(layer, metis.OPERAND_X)
        self.register_buffer("_place", torch.empty(0, device=device), persistent=False)
        self._init_step()

    def _count_device(self):
        return self._place.device if self._place.is_cuda else None

    def forward(self, x, residual=None):
        if not self.training or self.p == 0:
            if residual is None:
                return x
            if residual.shape != x.shape or residual.dtype != x.dtype:
                raise ValueError("the residual must have x's shape and type")
            return x + residual
        count = None
        if _capturing(x):
            count = self._captured_count()
            if count is None:  # replays would draw the capture's mask for ever
                raise RuntimeError("a captured pass reads the step on the GPU: move the layer there first")
        return _layers().dropout(x, residual, self.p, self.seed, self.tag, self._step, count)


class Embedding(torch.nn.Module):
    """``scale`` times the weight's rows (vocab x features) of the given token
    numbers (int32 or int64), in the weight's type or ``out_dtype``.  The
    gradient of a row is summed over its tokens in order, in binary32; row
    ``padding_idx`` takes none.  A token number outside the vocabulary gives a
    row of zeros, and the next ``metis.status_sync`` reports it."""

    def __init__(self, vocab, features, scale=1.0, padding_idx=None, weight=None, out_dtype=None, device="cuda",
                 dtype=torch.float32):
        super().__init__()
        if padding_idx is not None and not 0 <= padding_idx < vocab:
            raise ValueError("padding_idx must lie in [0, %d), got %r" % (vocab, padding_idx))
        if weight is None:
            weight = torch.empty(vocab, features, dtype=dtype, device=device)
            torch.nn.init.normal_(weight, std=0.02)
        if tuple(weight.shape) != (vocab, features):
            raise ValueError("weight must be vocab x features")
        self.weight = _parameter(weight, device)
        self.scale, self.padding_idx, self.out_dtype = scale, padding_idx, out_dtype
        self._padding = -1 if padding_idx is None else padding_idx
        self._out = -1 if out_dtype is None else metis.dtype_code(out_dtype)

    def forward(self, ids):
        return _layers().embedding(self.weight, ids, self.scale, self._padding, self._out)


class LinearCrossEntropy(torch.nn.Module):
    """The softmax cross entropy of the logits x W^T against target words, the
    logits never stored: the last product of a language model and its loss in
    one.  The weight is vocab x features and may be an Embedding's.

    ``reduction``: "mean" over the tokens that have a target (0 where none
    has), "sum", or "none" (the loss of each token).  A token whose target is
    ``ignore_index`` is left out: no loss, zero gradients, whatever its row of x
    holds; so is one whose target is not a word, which the next
    ``metis.status_sync`` reports.  x and the weight are bfloat16 or float32 and
    their gradients theirs; losses are float32."""

    def __init__(self, features, vocab, weight=None, ignore_index=-100, reduction="mean", device="cuda", dtype=torch.float32):
        super().__init__()
        if reduction not in ("mean", "sum", "none"):
            raise ValueError("reduction must be 'mean', 'sum' or 'none', got %r" % (reduction,))
        if weight is None:
            weight = torch.empty(vocab, features, dtype=dtype, device=device)
            torch.nn.init.normal_(weight, std=features ** -0.5)
        if tuple(weight.shape) != (vocab, features):
            raise ValueError("weight must be vocab x features")
        self.weight = _parameter(weight, device)
        self.ignore_index, self.reduction = ignore_index, reduction
        self._reduction = ("none", "sum", "mean").index(reduction)

    def forward(self, x, targets):
        return _layers().linear_cross_entropy(x, self.weight, targets, self.ignore_index, self._reduction)


def set_step(model, step):
    """Set the training step of every MetisLinear, Int8Linear and Dropout in ``model``."""
    for m in model.modules():
        if isinstance(m, (MetisLinear, Int8Linear, Dropout)):
            m.step = step
