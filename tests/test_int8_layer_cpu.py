"""The int8 layer's and binding's host side (no GPU work)."""

import copy
import ctypes
import pickle
import weakref

import pytest
import torch

from spectral_split_quantized_amd import layer, metis
from spectral_split_quantized_amd.layer import Int8Frozen, Int8Linear

D = ctypes.c_void_p(4096)  # aligned stand-in, never dereferenced


def test_step_count_pointer_and_tensor_are_checked():
    lib = metis.load()

    def counted(count, ax1=True, rounding=1):
        q = metis._I8(4096, 4096, 64, 48)
        return lib.metis_int8_quantize_counted(D, 0, 64, 48, 48, 2, rounding, 0, 0, 0, count, None,
                                               ctypes.byref(q) if ax1 else None, None, 0, None)

    assert counted(None) == metis.E_INVALID and counted(ctypes.c_void_p(4100)) == metis.E_INVALID
    assert counted(D, ax1=False) == metis.E_INVALID and counted(D, rounding=2) == metis.E_INVALID
    x = torch.zeros(4, 8)
    for bad in (torch.zeros(1), torch.zeros(2, dtype=torch.int64), torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="int64"):
            metis.int8_quantize(x, step_count=bad)


def test_step_survives_copies():
    lin = Int8Linear(4, 6, device="cpu")
    lin.step = 5
    state = lin.__getstate__()
    state["step"] = state.pop("_step")  # as saved when the step was a plain attribute
    old = Int8Linear.__new__(Int8Linear)
    old.__setstate__(state)
    for m in (copy.deepcopy(lin), pickle.loads(pickle.dumps(lin)), lin.float(), old):
        assert m.step == 5 and torch.equal(m.weight, lin.weight)
    assert list(lin.state_dict()) == ["weight"]


@pytest.fixture
def stubbed(monkeypatch):
    """The layer's calls answered with operands and products of zeros."""
    monkeypatch.setattr(metis, "int8_quantize", lambda m, axes, **kw: metis.I8Operand(*m.shape, axes, "cpu"))
    monkeypatch.setattr(metis, "int8_gemm", lambda a, b, out_dtype=torch.float32: torch.zeros(a.outer, b.outer, dtype=out_dtype))
    return monkeypatch


@pytest.mark.parametrize("shared", ["weight", "input", "layer"])
def test_capture_is_refused_while_an_eager_graph_of_a_shared_leaf_lives(stubbed, shared):
    """Two layers with one weight or one input, or one layer whose weight is
    computed: recording in a capture would meet the eager graph's leaf."""
    a, b = Int8Linear(4, 6, device="cpu"), Int8Linear(4, 6, device="cpu")
    leaf = torch.randn(3, 4, requires_grad=True)
    x, z = leaf, torch.randn(3, 4, requires_grad=True)
    if shared == "weight":
        b.weight = a.weight
    elif shared == "input":
        z = leaf
    else:
        b = a
        a.weight.requires_grad_(False)
    alive = a(x)
    with stubbed.context() as inside:
        inside.setattr(layer, "_capturing", lambda t: True)
        with pytest.raises(RuntimeError, match="alive"):
            b(z)
        free = Int8Linear(4, 6, device="cpu")  # shares nothing
        assert free(torch.randn(3, 4, requires_grad=True)).requires_grad
        with torch.no_grad():
            b(z)  # records nothing
        del alive
        assert b(z).requires_grad
    assert not a._eager and not b._eager  # what a capture records does not count


def test_longest_line_of_a_product():
    lib = metis.load()

    def gemm(k):
        a, b = metis._I8(4096, 4096, 0, k), metis._I8(4096, 4096, 64, k)  # no rows: nothing is enqueued
        return lib.metis_int8_gemm(ctypes.byref(a), ctypes.byref(b), D, 1, 64, None, 0, None)

    assert gemm(metis.INT8_MAX_K) == metis.OK and gemm(metis.INT8_MAX_K + 1) == metis.E_UNSUPPORTED


def test_long_reductions_are_cut_into_products_that_fit(stubbed):
    """No product of the layer is asked for more than its limit, and the runs cover every code once."""
    asked = []

    def gemm(a, b, out_dtype=torch.float32):
        assert a.k_len == b.k_len and a.codes.shape == (a.outer, metis.int8_pitch(a.k_len)) and a.codes.is_contiguous()
        asked.append(a.k_len)
        return torch.ones(a.outer, b.outer, dtype=out_dtype)

    stubbed.setattr(metis, "int8_gemm", gemm)
    for tokens, cin, cout, runs in ((131071, 2, 3, [2, 3, 131071]), (131072, 2, 3, [2, 3, 130944, 128]),
                                    (2, 3, 262000, [3, 130944, 130944, 112, 2]), (2, 140000, 3, [130944, 9056, 3, 2])):
        asked.clear()
        lin = Int8Linear(cin, cout, device="cpu")
        x = torch.zeros(tokens, cin, requires_grad=True)
        y = lin(x)
        y.sum().backward()
        assert asked == runs
        assert y[0, 0].item() == (2 if cin > 131071 else 1) and lin.weight.grad[0, 0].item() == (2 if tokens > 131071 else 1)


def _frozen(k, n=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(1, 128, (n, k), generator=g, dtype=torch.int8)
    return Int8Frozen(metis.I8.from_codes(codes, torch.rand(n, generator=g) + 0.5))


@pytest.mark.parametrize("there", [96, 97, 128])
@pytest.mark.parametrize("nested", [False, True])
def test_frozen_states_of_another_input_size_are_refused(there, nested):
    """All of these have code rows of 128 bytes."""
    wrap = (lambda m: torch.nn.Sequential(torch.nn.Identity(), m)) if nested else (lambda m: m)
    for here in (96, 97, 128):
        src, dst = _frozen(there), _frozen(here, seed=1)
        before = dst.codes.clone()
        if here == there:
            assert not any(wrap(dst).load_state_dict(wrap(src).state_dict()))
            assert torch.equal(dst.codes, src.codes) and torch.equal(dst.scales, src.scales)
        else:
            with pytest.raises(RuntimeError, match="size mismatch"):
                wrap(dst).load_state_dict(wrap(src).state_dict())
            assert torch.equal(dst.codes, before) and dst.k_len == here


def test_frozen_states_saved_without_the_input_size():
    state = _frozen(97).state_dict()
    assert int(state.pop("_extra_state")) == 97
    same = _frozen(97, seed=1)
    same.load_state_dict(state)
    assert torch.equal(same.codes, state["codes"])
    with pytest.raises(RuntimeError, match="size mismatch"):
        _frozen(96).load_state_dict(state)


@pytest.mark.parametrize("cast", [lambda m: m.to(torch.bfloat16), lambda m: m.half(), lambda m: m.double(),
                                  lambda m: m.bfloat16().float(), lambda m: m.to("cpu")])
def test_frozen_scales_keep_their_type_and_values(cast):
    m = _frozen(20)
    codes, scales = m.codes.clone(), m.scales.clone()
    out = cast(torch.nn.Sequential(m, torch.nn.Linear(2, 2)))
    assert out[0] is m and m.scales.dtype == torch.float32 and torch.equal(m.scales, scales)
    assert m.codes.dtype == torch.int8 and torch.equal(m.codes, codes) and list(m.state_dict()) == ["codes", "scales", "_extra_state"]
    metis.I8.wrap(m.codes, m.scales, m.k_len)._c()  # an operand that the library takes


@pytest.mark.parametrize("x_grad,w_grad,kept", [(True, True, 4), (True, False, 2), (False, True, 2)])
def test_saved_codes_pass_hooks_and_are_freed(stubbed, x_grad, w_grad, kept):
    """What the backward pass needs is saved as autograd saves tensors: hooks
    see it, a backward pass frees it, a second one is refused."""
    lin = Int8Linear(4, 6, device="cpu")
    lin.weight.requires_grad_(w_grad)
    packed, unpacked = [], []

    def pack(t):
        packed.append(t)
        return t.clone()

    def unpack(t):
        unpacked.append(t)
        return t

    x = torch.zeros(3, 4, requires_grad=x_grad)
    with torch.autograd.graph.saved_tensors_hooks(pack, unpack):
        y = lin(x)
    assert len(packed) == kept and {t.dtype for t in packed} == {torch.int8, torch.float32}
    y.sum().backward()
    assert len(unpacked) == kept
    with pytest.raises(RuntimeError, match="second time"):
        y.sum().backward()
    z = lin(x)
    codes = [weakref.ref(t) for t in z.grad_fn.saved_tensors if t is not None]
    assert len(codes) == kept
    z.sum().backward(retain_graph=True)
    z.sum().backward()
    assert not any(r() is not None for r in codes) and z.grad_fn is not None


def test_sizes_beyond_a_launch_are_refused():
    """A launch of 256 threads a workgroup takes fewer than 2^24 of them."""
    lib = metis.load()

    def quant(rows, cols, axes):
        a, b = metis._I8(4096, 4096, cols, rows), metis._I8(4096, 4096, rows, cols)
        return lib.metis_int8_quantize(D, 0, rows, cols, cols, axes, 0, 0, 0, 0, ctypes.byref(a), ctypes.byref(b), D, 16, None)

    most = (2 ** 24 - 1) * 128
    for axes in (1, 3):
        assert quant(most, 128, axes) == metis.E_WORKSPACE  # admitted, as far as the workspace
        for rows, cols in ((most + 1, 128), (most, 129), (2 ** 31 - 1, 1), (128, most + 1), (2 ** 20, 2 ** 20)):
            assert quant(rows, cols, axes) == metis.E_UNSUPPORTED
    assert quant(2 ** 31, 1, 2) == metis.E_UNSUPPORTED
