"""Host-side checks of the int8 and AdamW entry points (no GPU work): argument
errors are synchronous, sizes are right, bindings refuse bad operands."""

import ctypes

import numpy as np
import pytest
import torch

from spectral_split_quantized_amd import metis, optim
from spectral_split_quantized_amd.layer import Int8Linear, MetisLinear, set_step

D = ctypes.c_void_p(4096)  # aligned stand-in, never dereferenced


def _i8(outer, k, codes=4096, scales=4096):
    return metis._I8(codes, scales, outer, k)


def _quant(M=D, dtype=0, rows=64, cols=48, ld=48, axes=2, rounding=0, step=0, ax0=None, ax1=None, ws=D, n=1 << 30):
    lib = metis.load()
    ref = lambda q: None if q is None else ctypes.byref(q)  # noqa: E731
    return lib.metis_int8_quantize(M, dtype, rows, cols, ld, axes, rounding, 0, 0, step, ref(ax0), ref(ax1), ws, n, None)


def test_quantize_argument_errors():
    ok = _i8(64, 48)
    assert _quant(M=None, ax1=ok) == metis.E_INVALID
    assert _quant(dtype=5, ax1=ok) == metis.E_INVALID
    assert _quant(ld=47, ax1=ok) == metis.E_INVALID
    assert _quant(rows=-1, ax1=_i8(-1, 48)) == metis.E_INVALID
    for axes in (0, 4, -1):
        assert _quant(axes=axes, ax0=ok, ax1=ok) == metis.E_INVALID
    assert _quant(rounding=2, ax1=ok) == metis.E_INVALID
    assert _quant(step=-1, ax1=ok) == metis.E_INVALID
    assert _quant(ax1=None) == metis.E_INVALID
    assert _quant(ax1=_i8(64, 47)) == metis.E_INVALID and _quant(ax1=_i8(63, 48)) == metis.E_INVALID
    assert _quant(axes=1, ax0=_i8(64, 48)) == metis.E_INVALID  # not the transpose's shape
    assert _quant(ax1=_i8(64, 48, codes=4100)) == metis.E_INVALID
    assert _quant(ax1=_i8(64, 48, codes=None)) == metis.E_INVALID
    assert _quant(axes=1, ax0=_i8(48, 64), ws=D, n=16) == metis.E_WORKSPACE
    assert _quant(axes=1, ax0=_i8(48, 64), ws=None) == metis.E_WORKSPACE
    assert _quant(axes=1, ax0=_i8(48, 64), ws=ctypes.c_void_p(4100)) == metis.E_INVALID
    assert _quant(rows=0, ax1=_i8(0, 48, None, None)) == metis.OK  # nothing to do


def test_gemm_and_linear_argument_errors():
    lib = metis.load()

    def gemm(a, b, C=D, dt=1, ldc=64, ws=D, n=1 << 30):
        return lib.metis_int8_gemm(ctypes.byref(a), ctypes.byref(b), C, dt, ldc, ws, n, None)

    assert gemm(_i8(8, 128), _i8(64, 129)) == metis.E_INVALID
    assert gemm(_i8(8, 0), _i8(64, 0)) == metis.E_INVALID
    assert gemm(_i8(8, 131072), _i8(64, 131072)) == metis.E_UNSUPPORTED
    assert gemm(_i8(8, 128), _i8(64, 128), ldc=63) == metis.E_INVALID
    assert gemm(_i8(8, 128), _i8(64, 128), C=None) == metis.E_INVALID
    assert gemm(_i8(8, 128), _i8(64, 128), dt=2) == metis.E_INVALID
    assert gemm(_i8(8, 128), _i8(64, 128), C=ctypes.c_void_p(4098)) == metis.E_INVALID
    assert gemm(_i8(0, 128, None, None), _i8(64, 128)) == metis.OK
    assert lib.metis_int8_gemm_workspace(40, 64, 8192) > 0
    assert gemm(_i8(40, 8192), _i8(64, 8192), n=16) == metis.E_WORKSPACE
    assert gemm(_i8(40, 8192), _i8(64, 8192), ws=None) == metis.E_WORKSPACE
    assert gemm(_i8(40, 8192), _i8(64, 8192), ws=ctypes.c_void_p(4104)) == metis.E_INVALID

    def linear(w, X=D, dt=0, tokens=2, ldx=128, ldy=64, ws=D, n=1 << 20):
        return lib.metis_int8_linear(X, dt, tokens, ldx, ctypes.byref(w), D, 0, ldy, ws, n, None)

    assert linear(_i8(64, 128), X=None) == metis.E_INVALID
    assert linear(_i8(64, 128), dt=3) == metis.E_INVALID
    assert linear(_i8(64, 128), tokens=-1) == metis.E_INVALID
    assert linear(_i8(64, 128), ldx=127) == metis.E_INVALID
    assert linear(_i8(64, 128), ldy=63) == metis.E_INVALID
    assert linear(_i8(64, 128), tokens=5, n=64) == metis.E_WORKSPACE
    assert linear(_i8(64, 128), tokens=5, ws=None) == metis.E_WORKSPACE
    assert lib.metis_int8_linear_workspace(1, 64, 128) == 0  # a single token needs none
    assert linear(_i8(64, 0), ldx=0) == metis.E_INVALID
    assert linear(_i8(64, 128), tokens=0) == metis.OK
    assert lib.metis_int8_linear_workspace(7, 64, 129) >= 7 * 256 + 28


def test_pitch_and_layout():
    lib = metis.load()
    for k in (0, 1, 255, 256, 257, 4096):
        assert lib.metis_int8_pitch(k) == metis.int8_pitch(k) >= k
    q = metis.I8.from_codes(torch.full((3, 5), -7, dtype=torch.int8), torch.tensor([1.0, 2.0, 4.0]))
    assert tuple(q.codes.shape) == (3, 128) and not q.codes[:, 5:].any()
    assert q.dequantize()[2].tolist() == [-28.0] * 5


def test_bindings_refuse_bad_operands():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        metis.int8_quantize(x)
    with pytest.raises(ValueError):
        metis.int8_quantize(x[:, ::2])
    with pytest.raises(TypeError):
        metis.int8_quantize(x.double())
    with pytest.raises(ValueError):
        metis.int8_quantize(x, 0)
    with pytest.raises(ValueError):
        metis.int8_quantize(x, metis.AXIS1, out=metis.I8Operand(4, 8, metis.AXIS0, "cpu"))
    a, b = metis.I8(4, 100, "cpu"), metis.I8(5, 100, "cpu")
    with pytest.raises(ValueError):
        metis.int8_gemm(a, metis.I8(5, 99, "cpu"))
    with pytest.raises(ValueError):
        metis.int8_gemm(a, b, C=torch.empty(4, 6))
    with pytest.raises(ValueError):
        metis.int8_gemm(a, b, C=torch.empty(4, 5, dtype=torch.float16))
    with pytest.raises(ValueError):
        metis.int8_gemm(a, b, C=torch.empty(5, 4).T)
    with pytest.raises(ValueError, match="GPU"):
        metis.int8_gemm(a, b)
    b.codes = b.codes[:, :100]
    with pytest.raises(ValueError, match="contiguous"):
        metis.int8_gemm(a, b)
    with pytest.raises(ValueError):
        metis.int8_linear(x, a)
    with pytest.raises(ValueError):
        metis.I8.from_codes(x.to(torch.int8), torch.ones(3))
    with pytest.raises(ValueError):
        Int8Linear(4, 4, rounding="up", device="cpu")
    with pytest.raises(ValueError):
        Int8Linear(4, 4, weight=torch.zeros(4, 5), device="cpu")
    with pytest.raises(ValueError, match="features"):
        Int8Linear(4, 4, device="cpu")(torch.zeros(2, 5))


def test_set_step_reaches_both_kinds():
    net = torch.nn.Sequential(MetisLinear(16, 32, 2, device="cpu"), Int8Linear(32, 16, device="cpu", layer=3))
    set_step(net, 7)
    assert [m.step for m in net] == [7, 7]
    assert net[1].tags["D"] == metis.make_tag(3, metis.OPERAND_D)


@pytest.mark.parametrize("mode,x_grad,w_grad,axes", [
    (torch.no_grad, True, True, (2, 1)), (torch.inference_mode, False, True, (2, 1)), (torch.enable_grad, False, False, (2, 1)),
    (torch.enable_grad, False, True, (3, 1)), (torch.enable_grad, True, False, (2, 3)), (torch.enable_grad, True, True, (3, 3))])
def test_forward_quantises_what_its_gradients_need(monkeypatch, mode, x_grad, w_grad, axes):
    """The orientations of X and W that a forward pass asks for, and whether it
    counts as a graph that lives: without a gradient to come, neither."""
    asked = []

    def quantize(m, ax, **kw):
        asked.append(ax)
        return metis.I8Operand(m.shape[0], m.shape[1], ax, "cpu")

    monkeypatch.setattr(metis, "int8_quantize", quantize)
    monkeypatch.setattr(metis, "int8_gemm", lambda a, b, out_dtype: torch.zeros(a.outer, b.outer, dtype=out_dtype))
    lin = Int8Linear(6, 4, device="cpu")
    lin.weight.requires_grad_(w_grad)
    x = torch.zeros(3, 6, requires_grad=x_grad)
    with mode():
        y = lin(x)
    assert tuple(asked) == axes and (metis.AXIS0, metis.AXIS1) == (1, 2)
    assert len(lin._eager) == (axes != (2, 1)) and y.requires_grad == (axes != (2, 1))


def _adamw(tensor=None, count=1, **cfg):
    t = np.zeros(max(count, 1), metis._ADAMW_TENSOR)
    for name in ("param", "grad", "m", "v", "m_scale", "v_scale"):
        t[name] = 4096
    t["n"], t["state_bits"], t["param_dtype"], t["grad_dtype"] = 10, 8, 1, 1
    for k, v in (tensor or {}).items():
        t[k] = v
    c = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)
    c.update(cfg)
    return t, metis._AdamWConfig(**c)


@pytest.mark.parametrize("tensor,cfg", [
    ({"n": -1}, {}), ({"param": 0}, {}), ({"grad": 0}, {}), ({"m": 0}, {}), ({"v_scale": 0}, {}), ({"state_bits": 16}, {}),
    ({"param_dtype": 2}, {}), ({"grad_dtype": -1}, {}), ({"param": 4098}, {}), ({"grad": 4097}, {}),
    ({"state_bits": 32, "m": 4098}, {}), ({"m_scale": 4098}, {}),
    ({}, {"step": 0}), ({}, {"lr": -1.0}), ({}, {"lr": float("nan")}), ({}, {"eps": float("inf")}), ({}, {"beta1": 1.0}),
    ({}, {"beta2": -0.1}), ({}, {"weight_decay": -1.0}), ({}, {"rounding": 3})])
def test_adamw_argument_errors(tensor, cfg):
    t, c = _adamw(tensor, **cfg)
    assert metis.load().metis_adamw_step(ctypes.c_void_p(t.ctypes.data), 1, ctypes.byref(c), None) == metis.E_INVALID
    assert b"adamw_step" in metis.load().metis_last_error()


def test_adamw_null_lists_and_norm_errors():
    lib = metis.load()
    t, c = _adamw()
    ptr = ctypes.c_void_p(t.ctypes.data)
    assert lib.metis_adamw_step(None, 1, ctypes.byref(c), None) == metis.E_INVALID
    assert lib.metis_adamw_step(ptr, -1, ctypes.byref(c), None) == metis.E_INVALID
    assert lib.metis_adamw_step(ptr, 1, None, None) == metis.E_INVALID
    assert lib.metis_grad_norm(ptr, 1, 0.0, D, D, 1 << 20, None) == metis.E_INVALID
    assert lib.metis_grad_norm(ptr, 1, float("nan"), D, D, 1 << 20, None) == metis.E_INVALID
    assert lib.metis_grad_norm(ptr, 1, 1.0, None, D, 1 << 20, None) == metis.E_INVALID
    assert lib.metis_grad_norm(ptr, 1, 1.0, D, D, 8, None) == metis.E_WORKSPACE
    t["n"] = (1 << 31) * 4096
    assert lib.metis_grad_norm(ptr, 1, 1.0, D, D, 1 << 62, None) == metis.E_UNSUPPORTED
    t["n"] = 1 << 20
    assert lib.metis_grad_norm_workspace(ptr, 1) == 64 * 8 or lib.metis_grad_norm_workspace(ptr, 1) > 64 * 8


def test_adamw_binding_refusals():
    p = torch.zeros(10)
    m, v, ms, vs = metis.adamw_state(10, 8, "cpu")
    assert m.dtype == torch.float8_e4m3fn and tuple(ms.shape) == (1,)
    with pytest.raises(ValueError, match="GPU"):
        metis.adamw_step([p], [p], [m], [v], [ms], [vs], lr=1.0, step=1)
    with pytest.raises(ValueError):
        metis.adamw_step([p], [p], [m, m], [v], lr=1.0, step=1)
    with pytest.raises(ValueError):
        metis.adamw_state(10, 16)
    with pytest.raises(ValueError):
        metis.grad_norm([])
    with pytest.raises(ValueError, match="GPU"):
        metis.grad_norm([p])
    metis.adamw_step([], [], [], [], lr=1.0, step=1)  # nothing to do


def test_optimizer_refusals():
    p = torch.nn.Parameter(torch.zeros(4))
    for kw in (dict(state_bits=4), dict(rounding="up"), dict(lr=-1.0), dict(betas=(0.9, 1.0)), dict(max_norm=0.0),
               dict(eps=-1e-8), dict(weight_decay=-0.1)):
        with pytest.raises(ValueError):
            optim.AdamW([p], **kw)
    opt = optim.AdamW([p])
    opt.step()  # no gradient anywhere: nothing to do
    p.grad = torch.ones(4)
    with pytest.raises(ValueError, match="GPU"):
        opt.step()
    q = torch.nn.Parameter(torch.zeros(4))
    cap = optim.AdamW([p, q], capturable=True)
    with pytest.raises(RuntimeError, match="gradient"):
        cap.step()


@pytest.mark.parametrize("saved,here", [(False, False), (False, True), (True, False), (True, True)])
def test_step_counts_follow_the_loading_optimizer(saved, here):
    """A checkpoint's step counts, host integers or tensors, in the form that the loading optimizer advances."""
    p = torch.nn.Parameter(torch.zeros(300))
    opt = optim.AdamW([p], capturable=saved, min_8bit_size=1)
    opt._init_state(p)["step"] += 7
    other = optim.AdamW([torch.nn.Parameter(torch.zeros(300))], capturable=here, min_8bit_size=1)
    other.load_state_dict(opt.state_dict())
    (state,) = other.state.values()
    assert state["step"] == 7 and isinstance(state["step"], torch.Tensor if here else int)
    if here:
        assert state["step"].dtype == torch.int64 and state["step"] is not opt.state[p]["step"]
    assert state["exp_avg"].dtype == torch.float8_e4m3fn and opt.state[p]["step"] == 7
