"""AdamW over a model's parameters through the library: one launch for many
tensors, states in 32 or in 8 bits, clipping by the global gradient norm
without a host round trip.

Marshalling only: ``metis.grad_norm`` and ``metis.adamw_step`` state the
formulas and the formats.
"""

import torch

from . import metis

__all__ = ["AdamW"]

_STATES = ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
_SETTINGS = ("state_bits", "min_8bit_size", "rounding", "seed", "max_norm", "capturable")


class AdamW(torch.optim.Optimizer):
    """AdamW with decoupled weight decay.  By default its states are in 8 bits,
    rounded stochastically; ``state_bits=32`` is the plain optimizer.

    ``state_bits``: 8 holds both moments in E4M3 with a scale per 256 elements
    (parameters of fewer than ``min_8bit_size`` elements keep 32 bits), 32 in
    float32.  ``rounding``: "sr" (stochastic, draws from ``seed``, the
    parameter's place and the step) or "rne" for 8-bit states and bfloat16
    parameters; to nearest, 8-bit states cannot follow slow changes.
    ``max_norm``: clip the gradients' norm over all groups; ``grad_norm`` then
    holds the last step's norm, a one-element tensor on the GPU, new in each
    step (with ``capturable`` one tensor that every step and replay writes:
    clone what is to be kept).
    ``capturable``: the step count lives on the GPU, so that a step captured
    into a graph advances it on every replay (lr and the other values are
    those of the capture); every parameter then needs a gradient in every step.
    Parameters whose counts are equal share one count tensor, and each of a
    group's count tensors takes a call of its own; to set one parameter's count
    by hand, give its state a new tensor.

    Elements whose update is not finite are left as they are (8-bit moments are
    encoded again with their block's scale, which the other elements may have
    raised), and the next ``metis.status_sync`` reports it.  Parameters are float32 or bfloat16, on
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
        self.grad_norm = self._clip = None
        self._apart = {}

    def _init_state(self, p, count=None):
        """A new state; ``count``: the step count tensor it shares, if any."""
        if count is None:
            count = torch.zeros((), dtype=torch.int64, device=p.device) if self.capturable else 0
        eight = self.state_bits == 8 and p.numel() >= self.min_8bit_size
        m, v, ms, vs = metis.adamw_state(p.numel(), 8 if eight else 32, p.device)
        state = {"step": count, "exp_avg": m.view(p.shape), "exp_avg_sq": v.view(p.shape)}
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
        ext, calls, first = metis._tensors(), [], 0  # calls: (group, table, device, step count, states, gradients)
        for group in self.param_groups:
            params = group["params"]
            table = metis._table(len(params))
            found = ext.fill_state(params, self.state, first, self.capturable, table)
            if found is not None:
                calls.append((group, table, *found, None))
            else:
                calls.extend(self._sorted_calls(group, first, capturing))
            first += len(params)
        if not calls:
            return loss
        device, clip = calls[0][2], None
        if any(c[2] != device for c in calls):
            raise ValueError("the parameters must be on one GPU")
        if self.max_norm is not None:
            if not self.capturable or self._clip is None or self._clip.get_device() != device:
                self._clip = torch.empty(2, dtype=torch.float32, device=torch.device("cuda", device))
            whole = calls[0][1] if len(calls) == 1 else metis.np.concatenate([c[1] for c in calls])
            metis._grad_norm_run(whole, device, self.max_norm, self._clip)
            self.grad_norm, clip = self._clip[0], self._clip[1]
        if self.capturable:
            counts = {id(c[3]): c[3] for c in calls}
            if capturing:
                self._apart.update(counts)
            torch._foreach_add_(list(counts.values()), 1)
        for group, table, device, count, states, _ in calls:
            if not self.capturable:
                count += 1
            metis._adamw_run(table, device, group["lr"], group["betas"], group["eps"], group["weight_decay"], count, clip,
                             self.rounding, self.seed)
            if not self.capturable:
                for s in states:
                    s["step"] = count
        return loss

    def _sorted_calls(self, group, first, capturing):
        """A group's calls where its parameters are not all alike: without a
        gradient (left out), without a state (made), with a gradient to be
        copied into rows, or with step counts of their own (a call each)."""
        have = [(first + i, p) for i, p in enumerate(group["params"]) if p.grad is not None]
        if self.capturable and len(have) != len(group["params"]):
            raise RuntimeError("with capturable=True every parameter needs a gradient")
        new = [p for _, p in have if not self.state[p]]
        if new and capturing:
            raise RuntimeError("take one AdamW step before the capture: the states' first zeros would be captured")
        count = torch.zeros((), dtype=torch.int64, device=new[0].device) if new and self.capturable else None
        for p in new:
            self._init_state(p, count)
        if self.capturable and not capturing:
            self._share_counts([self.state[p] for _, p in have])
        sets = {}
        for i, p in have:
            count = self.state[p]["step"]
            sets.setdefault(id(count) if self.capturable else count, []).append((i, p))
        calls = []
        for _, some in sets.items() if self.capturable else sorted(sets.items()):
            params, states = [p for _, p in some], [self.state[p] for _, p in some]
            grads = [p.grad.contiguous() for p in params]
            table = metis._table(len(params))
            device = metis._tensors().fill(params, grads, *([s.get(k) for s in states] for k in _STATES),
                                           [metis.make_tag(i, metis.OPERAND_W) for i, _ in some], table)
            calls.append((group, table, device, states[0]["step"], states, grads))
        return calls

    def _share_counts(self, states):
        """One tensor for equal counts on the GPU, of tensors that come here for
        the first time: those read before differ and go up together, and those
        of a capture are its replays'."""
        new = {id(s["step"]): s["step"] for s in states if id(s["step"]) not in self._apart}
        first, shared = {}, {}
        if len(new) > 1:
            for (i, c), value in zip(new.items(), torch.cat([c.reshape(1) for c in new.values()]).tolist()):
                shared[i] = first.setdefault(value, c)
            for s in states:
                s["step"] = shared.get(id(s["step"]), s["step"])
        self._apart.update((id(s["step"]), s["step"]) for s in states)

    def __getstate__(self):
        return {**super().__getstate__(), **{k: getattr(self, k) for k in _SETTINGS}}

    def __setstate__(self, state):
        super().__setstate__(state)
        self.grad_norm = self._clip = None
        self._apart = {}

    def load_state_dict(self, state_dict):
        """As torch's, but the states keep their own types (torch would cast
        8-bit codes to the parameters' type), and the step count takes the
        form that ``capturable`` asks for.  States are new memory: capture a
        step anew after loading."""
        super().load_state_dict(state_dict)
        saved = {i: p for group, here in zip(state_dict["param_groups"], self.param_groups)
                 for i, p in zip(group["params"], here["params"])}
        counts = {}
        for i, state in state_dict["state"].items():
            if i in saved:
                p = saved[i]
                self.state[p] = {k: v.detach().clone().to(p.device) if isinstance(v, torch.Tensor) else v
                                 for k, v in state.items()}
                step = self.state[p].get("step")
                if self.capturable and step is not None:
                    key = (p.device, int(step))  # equal counts: one tensor
                    if key not in counts:
                        counts[key] = torch.tensor(key[1], dtype=torch.int64, device=p.device)
                    self.state[p]["step"] = counts[key]
                elif isinstance(step, torch.Tensor):
                    self.state[p]["step"] = int(step)
