"""The optimizer's host side (no GPU work): the library's calls are recorded
in place of being run."""

import ctypes
import types

import numpy as np
import pytest
import torch

from oracle import adamw
from spectral_split_quantized_amd import metis, optim


@pytest.fixture
def runs(monkeypatch):
    """Per call of the step: (its parameters, its number, the number's tensor or None)."""
    calls, filled = [], []

    def fill(params, *rest):
        filled.append((rest[-1], params))
        return 0

    def run(table, device, lr, betas, eps, weight_decay, step, *_):
        (params,) = [p for t, p in filled if t is table]
        calls.append((params, int(step), step if isinstance(step, torch.Tensor) else None))

    ext = types.SimpleNamespace(fill=fill, fill_state=lambda *a: None)
    monkeypatch.setattr(metis, "_tensors", lambda: ext)
    monkeypatch.setattr(metis, "_adamw_run", run)
    return calls


def _params(n, grads=True):
    ps = [torch.nn.Parameter(torch.zeros(4)) for _ in range(n)]
    for p in ps:
        p.grad = torch.ones(4) if grads else None
    return ps


def _taken(runs):
    """{parameter: step's number} of the recorded calls."""
    return {p: t for params, t, _ in runs for p in params}


@pytest.mark.parametrize("saved", [False, True])
def test_loaded_counts_that_differ_are_stepped_each_by_its_own(runs, saved):
    """A parameter without a gradient in some steps has a count of its own,
    also after loading into an optimizer whose counts are on the GPU."""
    src = optim.AdamW(_params(3), capturable=saved)
    for p, t in zip(src.param_groups[0]["params"], (1000, 3, 1000)):
        src._init_state(p)["step"] = torch.tensor(t) if saved else t
    ps = _params(3)
    opt = optim.AdamW(ps, capturable=True)
    opt.load_state_dict(src.state_dict())
    for t in (1, 2):
        runs.clear()
        opt.step()
        taken = _taken(runs)
        assert [taken[p] for p in ps] == [1000 + t, 3 + t, 1000 + t] and len(runs) == 2
        assert [int(opt.state[p]["step"]) for p in ps] == [1000 + t, 3 + t, 1000 + t]
        for params, _, count in runs:  # the tensor that a replay reads is the one that the state shows
            assert all(opt.state[p]["step"] is count for p in params)


def test_a_parameter_that_joins_late_starts_at_its_own_first_step(runs):
    ps = _params(3)
    opt = optim.AdamW(ps[:2], capturable=True)
    opt.step()
    opt.step()
    opt.add_param_group({"params": ps[2:]})
    runs.clear()
    opt.step()
    assert [_taken(runs)[p] for p in ps] == [3, 3, 1]
    # in one group: a state dict that lacks a parameter
    state = opt.state_dict()
    del state["state"][1]
    ps = _params(3)
    other = optim.AdamW([{"params": ps[:2]}, {"params": ps[2:]}], capturable=True)
    other.load_state_dict(state)
    runs.clear()
    other.step()
    assert [_taken(runs)[p] for p in ps] == [4, 1, 2]


def test_equal_counts_are_one_tensor_advanced_once(runs):
    """One call for all, over groups too, and a count shared by two groups goes up by one."""
    ps = _params(4)
    opt = optim.AdamW([{"params": ps[:2]}, {"params": ps[2:]}], capturable=True)
    opt.step()
    assert len(runs) == 2
    again = optim.AdamW([{"params": ps[:2]}, {"params": ps[2:]}], capturable=True)
    again.load_state_dict(opt.state_dict())
    assert len({id(s["step"]) for s in again.state.values()}) == 1
    runs.clear()
    again.step()
    assert len(runs) == 2 and all(int(s["step"]) == 2 for s in again.state.values())
    assert all(int(s["step"]) == 1 for s in opt.state.values())  # loading takes copies


def test_equal_counts_on_tensors_of_their_own_are_joined(runs, monkeypatch):
    """States set by hand or by another loader, a count tensor each: one call a
    value, and the values are read once, not in every step."""
    ps = _params(5)
    opt = optim.AdamW(ps, capturable=True)
    for p, t in zip(ps, (7, 7, 2, 7, 2)):
        opt._init_state(p)["step"] = torch.tensor(t)
    read, cat = [], torch.cat
    monkeypatch.setattr(torch, "cat", lambda ts: read.append(len(ts)) or cat(ts))
    for k in (1, 2, 3):
        runs.clear()
        opt.step()
        assert [_taken(runs)[p] for p in ps] == [7 + k, 7 + k, 2 + k, 7 + k, 2 + k] and len(runs) == 2
    assert read == [5]
    opt.state[ps[4]]["step"] = torch.tensor(10)  # set by hand
    runs.clear()
    opt.step()
    assert [_taken(runs)[p] for p in ps] == [11, 11, 6, 11, 11] and read == [5]


def test_count_tensors_of_a_capture_are_not_replaced(runs, monkeypatch):
    """Replays advance and read the memory of the capture, whatever an eager
    step finds there later."""
    ps = _params(3)
    opt = optim.AdamW(ps, capturable=True)
    counts = [opt._init_state(p)["step"] for p in ps]
    with monkeypatch.context() as inside:
        inside.setattr(torch.cuda, "is_available", lambda: True)
        inside.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        opt.step()
    opt.step()
    assert all(opt.state[p]["step"] is c for p, c in zip(ps, counts)) and [int(c) for c in counts] == [2, 2, 2]


def test_oracle_keeps_values_that_are_not_finite_out_of_the_scale():
    x = np.linspace(0.1, 1.0, 300).astype(np.float32)
    want, s = adamw.encode(x)
    for bad in (np.nan, np.inf, -np.inf):
        y = x.copy()
        y[[3, 280]] = bad
        codes, scales = adamw.encode(y)
        good = np.setdiff1d(np.arange(300), [3, 280])
        assert np.array_equal(scales, s) and np.array_equal(codes[good], want[good])
        d = adamw.decode(codes, scales)
        assert np.isnan(d[[3, 280]]).all() and np.isfinite(d[good]).all()


def test_tensors_beyond_a_launch_are_refused():
    """A launch of 256 threads a workgroup takes fewer than 2^24 of them, each 4096 elements."""
    lib = metis.load()
    t = np.zeros(1, metis._ADAMW_TENSOR)
    for name in ("param", "grad", "m", "v", "m_scale", "v_scale"):
        t[name] = 4096
    t["state_bits"], t["param_dtype"], t["grad_dtype"] = 8, 1, 1
    ptr, most = ctypes.c_void_p(t.ctypes.data), (2 ** 24 - 1) * 4096
    cfg = metis._AdamWConfig(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)
    t["n"] = most + 1
    assert lib.metis_adamw_step(ptr, 1, ctypes.byref(cfg), None) == metis.E_UNSUPPORTED
    assert lib.metis_grad_norm(ptr, 1, 1.0, ptr, ptr, 1 << 62, None) == metis.E_UNSUPPORTED
    t["n"] = most
    assert lib.metis_grad_norm(ptr, 1, 1.0, ptr, ptr, 8, None) == metis.E_WORKSPACE  # admitted, as far as the workspace
