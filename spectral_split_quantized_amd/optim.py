"""AdamW over a model's parameters through the library: one launch for many
tensors, states in 32 or in 8 bits, clipping by the global gradient norm
without a host round trip.

Marshalling only: ``metis.grad_norm`` and ``metis.adamw_step`` state the
formulas and the formats.
"""

import torch

from . import metis

__all__ = ["AdamW"]

_SETTINGS = ("state_bits", "min_8bit_size", "rounding", "seed", "max_norm", "capturable")


class AdamW(torch.optim.Optimizer):
    """AdamW with decoupled weight decay.

    ``state_bits``: 8 holds both moments in E4M3 with a scale per 256 elements
    (parameters of fewer than ``min_8bit_size`` elements keep 32 bits), 32 in
    float32.  ``rounding``: "sr" (stochastic, draws from ``seed``, the
    parameter's place and the step) or "rne" for 8-bit states and bfloat16
    parameters; to nearest, 8-bit states cannot follow slow changes.
    ``max_norm``: clip the gradients' norm over all groups; ``grad_norm`` then
    holds the last step's norm, a one-element tensor on the GPU.
    ``capturable``: the step count lives on the GPU, so that a step captured
    into a graph advances it on every replay (lr and the other values are
    those of the capture); every parameter then needs a gradient in every step.

    Elements whose update is not finite are left as they are, and the next
    ``metis.status_sync`` reports it.  Parameters are float32 or bfloat16, on
    one GPU and contiguous."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, state_bits=8,
                 min_8bit_size=4096, rounding="sr", seed=0, max_norm=None, capturable=False):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32, got %r" % (state_bits,))
        if rounding not in ("sr", "rne"):
            raise ValueError("rounding must be 'sr' or 'rne', got %r" % (rounding,))
        if not (lr >= 0 and eps >= 0 and weight_decay >= 0 and all(0 <= b < 1 for b in betas)):
            raise ValueError("lr, eps and weight_decay must not be negative and betas lie in [0, 1)")
        if max_norm is not None and not max_norm > 0:
            raise ValueError("max_norm must be positive, got %r" % (max_norm,))
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay))
        seen = [p for g in self.param_groups for p in g["params"]]
        if len(set(seen)) != len(seen):
            raise ValueError("a parameter appears twice")
        self.state_bits, self.min_8bit_size = state_bits, min_8bit_size
        self.rounding = metis.SR if rounding == "sr" else metis.RNE
        self.seed, self.max_norm, self.capturable = seed, max_norm, capturable
        self.grad_norm = None
        self._clip = None
        self._tables = {}

    def _init_state(self, p):
        eight = self.state_bits == 8 and p.numel() >= self.min_8bit_size
        m, v, ms, vs = metis.adamw_state(p.numel(), 8 if eight else 32, p.device)
        state = {"step": torch.zeros((), dtype=torch.int64, device=p.device) if self.capturable else 0,
                 "exp_avg": m.view(p.shape), "exp_avg_sq": v.view(p.shape)}
        if eight:
            state.update(exp_avg_scale=ms, exp_avg_sq_scale=vs)
        self.state[p] = state
        return state

    @torch.no_grad()
    def step(self, closure=None):
        """One update; returns the closure's loss, if there is one."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        capturing = torch.cuda.is_available() and torch.cuda.is_current_stream_capturing()
        if capturing and not self.capturable:
            raise RuntimeError("an AdamW step needs capturable=True to be captured into a graph")
        calls, first = [], 0
        for group in self.param_groups:
            params = group["params"]
            grads = [p.grad for p in params]
            tags = range(first, first + len(params))
            first += len(params)
            if True in [g is None for g in grads]:
                if self.capturable:
                    raise RuntimeError("with capturable=True every parameter needs a gradient")
                have = [i for i, g in enumerate(grads) if g is not None]
                params, grads, tags = ([x[i] for i in have] for x in (params, grads, tags))
            if not params:
                continue
            states = [self.state[p] for p in params]
            if not all(states):
                if capturing:
                    raise RuntimeError("take one AdamW step before the capture: the states' first zeros would be captured")
                states = [s or self._init_state(p) for p, s in zip(params, states)]
            # parameters that missed steps have counts of their own
            counts = {0} if self.capturable else {s["step"] for s in states}
            if len(counts) == 1:
                calls.append((group, params, grads, states, tags))
                continue
            for count in sorted(counts):
                some = [i for i, s in enumerate(states) if s["step"] == count]
                calls.append((group, *([x[i] for i in some] for x in (params, grads, states, tags))))
        if not calls:
            return loss
        tables = []
        for k, (_, params, grads, states, tags) in enumerate(calls):
            if not all(map(torch.Tensor.is_contiguous, grads)):
                grads = [g.contiguous() for g in grads]
            columns = ([s["exp_avg"] for s in states], [s["exp_avg_sq"] for s in states],
                       [s.get("exp_avg_scale") for s in states], [s.get("exp_avg_sq_scale") for s in states])
            kept = self._tables.setdefault(k, metis._AdamWTable())
            tables.append((*kept.update(params, grads, columns, tags), grads))
        if len({d for _, d, _ in tables}) != 1:
            raise ValueError("the parameters must be on one GPU")
        device, clip = tables[0][1], None
        if self.max_norm is not None:
            if self._clip is None or self._clip.get_device() != device:
                self._clip = torch.empty(2, dtype=torch.float32, device=torch.device("cuda", device))
            whole = tables[0][0] if len(tables) == 1 else metis.np.concatenate([t for t, _, _ in tables])
            metis._grad_norm_run(whole, device, self.max_norm, self._clip)
            self.grad_norm, clip = self._clip[0], self._clip[1]
        for (group, _, _, states, _), (table, device, _) in zip(calls, tables):
            if self.capturable:
                torch._foreach_add_([s["step"] for s in states], 1)
                count = states[0]["step"]
            else:
                count = states[0]["step"] + 1
            metis._adamw_run(table, device, group["lr"], group["betas"], group["eps"], group["weight_decay"], count, clip,
                             self.rounding, self.seed)
            if not self.capturable:
                for s in states:
                    s["step"] = count
        return loss

    def __getstate__(self):
        return {**super().__getstate__(), **{k: getattr(self, k) for k in _SETTINGS}}

    def __setstate__(self, state):
        super().__setstate__(state)
        self.grad_norm = self._clip = None
        self._tables = {}

    def load_state_dict(self, state_dict):
        """As torch's, but the states keep their own types (torch would cast
        8-bit codes to the parameters' type)."""
        super().load_state_dict(state_dict)
        saved = {i: p for group, here in zip(state_dict["param_groups"], self.param_groups)
                 for i, p in zip(group["params"], here["params"])}
        for i, state in state_dict["state"].items():
            if i in saved:
                p = saved[i]
                self.state[p] = {k: v.detach().clone().to(p.device) if isinstance(v, torch.Tensor) else v
                                 for k, v in state.items()}
