"""GPU tests of the int8 path (metis_int8_quantize, metis_int8_gemm,
metis_int8_linear and the layer on them) against oracle/int8.py.

The quantiser's codes and scales and the products are defined to the last bit
(int32 sums are exact, the epilogue rounds binary32 step by step), so every
comparison is for equality, except that of the layer's gradients with the
exact products, whose bound is derived where it stands."""

import numpy as np
import pytest
import torch

from oracle import int8
from spectral_split_quantized_amd import metis
from spectral_split_quantized_amd.layer import Int8Linear, set_step

from gpu_helpers import say

pytestmark = pytest.mark.gpu

BOTH = metis.AXIS0 | metis.AXIS1


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X; none is visible")
    metis.load()
    torch.cuda.set_device(0)


def _inputs(rows, cols, seed, dtype):
    """Gaussian rows of very different sizes, with an all-zero row and column,
    negative zeros, a strong channel and magnitudes near binary32's ends."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, dtype=torch.float64)
    x *= torch.exp(torch.empty(rows, 1, dtype=torch.float64).uniform_(-9, 9, generator=g))
    if rows > 4 and cols > 4:
        x[1] = 0.0
        x[2] = -0.0
        x[3] *= 1e-37
        x[4] = x[4] / x[4].abs().max() * 3e38
        x[:, 3] = 0.0
        x[0, 4] *= 100
    return x.to(dtype)


def _np(t):
    return t.detach().float().cpu().numpy()


def _gemm32(a, b):
    """The product's definition in binary32 steps."""
    s = a[0].astype(np.float64) @ b[0].astype(np.float64).T  # exact integers below 2^53
    return s.astype(np.float32) * np.asarray(a[1], np.float32)[:, None] * np.asarray(b[1], np.float32)[None, :]


def _upload(q):
    return metis.I8.from_codes(torch.from_numpy(q[0]).cuda(), torch.from_numpy(q[1]).cuda())


def _random(rng, outer, k):
    codes = rng.integers(-127, 128, (outer, k), dtype=np.int8)
    return codes, np.exp(rng.uniform(-4, 4, outer)).astype(np.float32)


@pytest.mark.parametrize("rounding", ["rne", "sr"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("axes", [metis.AXIS0, metis.AXIS1, BOTH])
@pytest.mark.parametrize("shape", [(1, 1), (1, 200), (200, 1), (7, 9), (64, 128), (129, 257), (130, 1000), (5, 9000), (300, 40)])
def test_quantize_bit_exact(shape, axes, dtype, rounding):
    say("int8 quantize %s axes %d %s %s" % (shape, axes, dtype, rounding))
    x = _inputs(*shape, 3 + shape[0], dtype)
    kw = dict(seed=0x1234567890AB, tag=0x5A3C, step=7)
    q = metis.int8_quantize(x.cuda(), axes, rounding=metis.SR if rounding == "sr" else metis.RNE, **kw)
    metis.status_sync()
    for axis, got in ((0, q.ax0), (1, q.ax1)):
        if got is None:
            assert not axes & (1 + axis)
            continue
        codes, scales = int8.quantize(_np(x), axis, rounding, **kw)
        assert np.array_equal(got.scales.cpu().numpy(), scales)
        assert np.array_equal(got.codes[:, :got.k_len].cpu().numpy(), codes)
        assert not got.codes[:, got.k_len:].any()  # the padding is zero


@pytest.mark.parametrize("cols", [16384, 16385, 40000])
def test_quantize_long_rows(cols):
    """Rows longer than a workgroup keeps in registers are read again."""
    say("int8 quantize long rows %d" % cols)
    x = _inputs(6, cols, 5, torch.float32)
    q = metis.int8_quantize(x.cuda(), metis.AXIS1, rounding=metis.SR, seed=1, tag=2, step=3)
    metis.status_sync()
    codes, scales = int8.quantize(_np(x), 1, "sr", 1, 2, 3)
    assert np.array_equal(q.ax1.scales.cpu().numpy(), scales)
    assert np.array_equal(q.ax1.codes[:, :cols].cpu().numpy(), codes)


@pytest.mark.parametrize("axes", [metis.AXIS1, BOTH])
@pytest.mark.parametrize("first,ld", [(0, 333), (1, 333), (8, 336), (3, 336)])
def test_quantize_strided_and_misaligned_views(first, ld, axes):
    say("int8 quantize view from column %d of %d, axes %d" % (first, ld, axes))
    wide = _inputs(150, ld, 11, torch.bfloat16)
    x = wide[:, first:first + 250]
    q = metis.int8_quantize(wide.cuda()[:, first:first + 250], axes)
    metis.status_sync()
    for axis, got in ((0, q.ax0), (1, q.ax1)):
        if got is not None:
            codes, scales = int8.quantize(_np(x), axis)
            assert np.array_equal(got.scales.cpu().numpy(), scales)
            assert np.array_equal(got.codes[:, :got.k_len].cpu().numpy(), codes)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("axes", [metis.AXIS0, metis.AXIS1])
def test_quantize_non_finite_sets_numeric_status(axes, bad):
    say("int8 non-finite input axes %d %s" % (axes, bad))
    M = torch.randn(64, 128, device="cuda")
    M[17, 45] = bad
    metis.int8_quantize(M, axes)
    with pytest.raises(metis.MetisError) as ei:
        metis.status_sync()
    assert ei.value.status == metis.E_NUMERIC
    metis.int8_quantize(torch.randn(64, 128, device="cuda"), axes)
    metis.status_sync()


@pytest.mark.parametrize("rows,cols", [(3, 1 << 25), (1 << 22, 3)])
def test_quantize_very_long_lines(rows, cols):
    """One long axis, both orientations: sampled lines against the definition."""
    say("int8 quantize %d x %d" % (rows, cols))
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    q = metis.int8_quantize(x, BOTH)
    metis.status_sync()
    for got, y in ((q.ax1, x), (q.ax0, x.T)):
        some = torch.tensor(sorted({0, y.shape[0] // 2, y.shape[0] - 1}), device="cuda")
        codes, scales = int8.quantize(_np(y[some].contiguous()), 1)
        assert np.array_equal(got.scales[some].cpu().numpy(), scales)
        assert np.array_equal(got.codes[some][:, :got.k_len].cpu().numpy(), codes)


def test_quantize_empty_is_a_no_op():
    for shape in ((0, 5), (5, 0), (0, 0)):
        q = metis.int8_quantize(torch.zeros(shape, device="cuda"), BOTH)
        assert (q.ax0.outer, q.ax1.outer) == (shape[1], shape[0])
    metis.status_sync()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 17, 129), (3, 1000, 64), (16, 33, 500), (17, 64, 2000), (32, 16, 40),
                                   (33, 200, 777), (64, 130, 128), (65, 129, 300), (200, 7, 1000), (128, 128, 128),
                                   (300, 500, 250), (1000, 2100, 400), (4100, 4099, 130), (5000, 3, 129)])
def test_gemm_equals_definition(m, n, k, out):
    say("int8 gemm %d x %d x %d %s" % (m, n, k, out))
    rng = np.random.default_rng(m + n + k)
    a, b = _random(rng, m, k), _random(rng, n, k)
    C = metis.int8_gemm(_upload(a), _upload(b), out_dtype=out)
    metis.status_sync()
    want = torch.from_numpy(_gemm32(a, b)).to(out)
    assert C.dtype == out and torch.equal(C.cpu(), want)


@pytest.mark.parametrize("m", [5, 300])
def test_gemm_longest_sums_stay_in_int32(m):
    """k_len at its limit with every product at 127^2 and at 128^2, and one beyond it refused."""
    k = 131071
    say("int8 gemm longest k, %d rows" % m)
    ones = lambda r: metis.I8.from_codes(torch.full((r, k), 127, dtype=torch.int8, device="cuda"),  # noqa: E731
                                         torch.ones(r, device="cuda"))
    C = metis.int8_gemm(ones(m), ones(9))
    low = metis.I8.from_codes(torch.full((9, k), -128, dtype=torch.int8, device="cuda"), torch.ones(9, device="cuda"))
    C2 = metis.int8_gemm(low, low)
    metis.status_sync()
    assert bool((C == float(np.float32(127 * 127 * k))).all()) and bool((C2 == float(np.float32(128 * 128 * k))).all())
    with pytest.raises(metis.MetisError) as ei:
        metis.int8_gemm(metis.I8(m, k + 1), metis.I8(9, k + 1))
    assert ei.value.status == metis.E_UNSUPPORTED


@pytest.mark.parametrize("m", [9, 150])
def test_gemm_writes_only_its_view(m):
    say("int8 gemm into a view, %d rows" % m)
    rng = np.random.default_rng(m)
    a, b = _random(rng, m, 200), _random(rng, 77, 200)
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.full((m + 2, 100), 7.0, dtype=dt, device="cuda")
        metis.int8_gemm(_upload(a), _upload(b), C=buf[1:m + 1, 5:82])
        metis.status_sync()
        want = torch.full((m + 2, 100), 7.0, dtype=dt)
        want[1:m + 1, 5:82] = torch.from_numpy(_gemm32(a, b)).to(dt)
        assert torch.equal(buf.cpu(), want)


def test_operands_beyond_32_bit_offsets():
    """Code rows that start past 4 GiB, on the tiled product and the quantiser."""
    rows, k = 70000, 65536
    say("int8 operand of %d x %d codes" % (rows, k))
    g = torch.Generator(device="cuda").manual_seed(2)
    base = torch.randint(-127, 128, (1000, k), generator=g, dtype=torch.int8, device="cuda")
    big = metis.I8(rows, k)
    for r in range(0, rows, 1000):
        big.codes[r:r + 1000] = base
    big.scales.copy_(torch.arange(rows, device="cuda") % 7 + 1)
    small = metis.I8.from_codes(base[:100].clone(), torch.ones(100, device="cuda"))
    want = (base[:, :].double() @ base[:100].double().T).float()
    C = metis.int8_gemm(big, small)
    metis.status_sync()
    for r in (0, 65000, 69000):
        assert torch.equal(C[r:r + 1000], want * big.scales[r:r + 1000, None])
    C2 = metis.int8_gemm(metis.I8.from_codes(base[:3].clone(), torch.ones(3, device="cuda")), big, out_dtype=torch.float32)
    metis.status_sync()
    assert torch.equal(C2[:, 69000:], want[:, :3].T * big.scales[None, 69000:])
    del big, C, C2
    x = torch.zeros(rows, 32768, dtype=torch.bfloat16, device="cuda")  # 4.6 GB
    x[-1] = torch.randn(32768, generator=g, device="cuda").to(torch.bfloat16)
    q = metis.int8_quantize(x, metis.AXIS1, rounding=metis.SR, seed=5)
    e0 = (rows - 1) * 32768
    metis.status_sync()
    from oracle import philox
    u = philox.halves(np.arange(e0, e0 + 32768, dtype=np.uint64), 5, 0, 0) / 65536
    xr = _np(x[-1])
    s = np.float32(np.abs(xr).max() / np.float32(127))
    y = xr * (np.float32(1) / s)
    code = np.floor(y) + (u < y - np.floor(y))
    assert np.array_equal(q.ax1.codes[-1].cpu().numpy(), np.clip(code, -127, 127).astype(np.int8))
    assert not q.ax1.codes[:-1].any()


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, None), (torch.float32, None), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("tokens,k,n", [(1, 64, 16), (1, 4096, 1000), (1, 4097, 33), (1, 16384, 50), (1, 16385, 20), (2, 1337, 257),
                                        (5, 200, 64), (16, 513, 100),
                                        (37, 5000, 300), (64, 128, 128), (65, 300, 400), (500, 260, 390)])
def test_linear_equals_its_parts(tokens, k, n, dtype, out):
    say("int8 linear %d tokens, %d -> %d, %s" % (tokens, k, n, dtype))
    x = _inputs(tokens, k, tokens, torch.float32).clamp(-1e4, 1e4).to(dtype)
    w = _random(np.random.default_rng(k), n, k)
    y = metis.int8_linear(x.cuda(), _upload(w), out_dtype=out)
    metis.status_sync()
    want = torch.from_numpy(_gemm32(int8.quantize(_np(x)), w)).to(out or dtype)
    assert y.dtype == want.dtype and torch.equal(y.cpu(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_linear_of_misaligned_and_strided_views(tokens, dtype):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    wide = torch.randn(tokens, 777, generator=g, device="cuda").to(dtype)
    w = _upload(_random(np.random.default_rng(tokens), 60, 701))
    buf = torch.full((tokens, 70), 7.0, dtype=dtype, device="cuda")
    y = metis.int8_linear(wide[:, 3:704], w, Y=buf[:, 5:65])
    metis.status_sync()
    assert torch.equal(y, metis.int8_linear(wide[:, 3:704].contiguous(), w))
    assert bool((buf[:, :5] == 7).all()) and bool((buf[:, 65:] == 7).all())


def test_workspaces():
    """A caller's workspace is used where it is large enough and refused on another device."""
    x = torch.randn(200, 300, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    a, b = metis.int8_quantize(x, BOTH, workspace=ws), metis.int8_quantize(x, BOTH)
    assert torch.equal(a.ax0.codes, b.ax0.codes)
    q = metis.int8_quantize(torch.randn(20, 4096, device="cuda")).ax1
    assert torch.equal(metis.int8_gemm(q, q, workspace=ws), metis.int8_gemm(q, q))
    for call in (lambda w: metis.int8_quantize(x, BOTH, workspace=w), lambda w: metis.grad_norm([x], workspace=w)):
        with pytest.raises(ValueError, match="workspace"):
            call(torch.empty(1 << 20, dtype=torch.uint8))


@pytest.mark.parametrize("tokens", [1, 3])
def test_linear_non_finite_token_is_reported(tokens):
    x = torch.randn(tokens, 256, device="cuda")
    x[-1, 100] = float("nan")
    metis.int8_linear(x, _upload(_random(np.random.default_rng(1), 40, 256)))
    with pytest.raises(metis.MetisError):
        metis.status_sync()


def _quantised_products(x, w, d, seed, tag, step, rounding="sr"):
    q = int8.quantize
    y = _gemm32(q(x, 1), q(w, 0))
    dx = _gemm32(q(d, 1, rounding, seed, tag, step), q(w, 1))
    dw = _gemm32(q(x, 0), q(d, 0, rounding, seed, tag, step))
    return y, dx, dw


@pytest.mark.parametrize("rounding", ["sr", "rne"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,cin,cout", [(1, 16, 16), (33, 100, 70), (300, 130, 257)])
def test_layer_forward_and_gradients(tokens, cin, cout, dtype, rounding):
    say("int8 layer %d tokens %d -> %d %s" % (tokens, cin, cout, dtype))
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, cin, generator=g).to(dtype)
    w = torch.randn(cin, cout, generator=g)
    d = torch.randn(tokens, cout, generator=g).to(dtype)
    lin = Int8Linear(cin, cout, rounding=rounding, seed=21, layer=4, weight=w.cuda())
    set_step(lin, 6)
    xg = x.cuda().requires_grad_(True)
    y = lin(xg)
    y.backward(d.cuda())
    metis.status_sync()
    want = _quantised_products(_np(x), w.numpy(), _np(d), 21, metis.make_tag(4, metis.OPERAND_D), 6, rounding)
    for got, ref, dt in ((y, want[0], dtype), (xg.grad, want[1], dtype), (lin.weight.grad, want[2], torch.float32)):
        assert got.dtype == dt and torch.equal(got.detach().cpu(), torch.from_numpy(ref).to(dt))


def test_layer_gradients_against_exact_products():
    """The int8 gradients stay near the unquantised ones: with independent
    rounding errors of variance s^2 / 12 (nearest) and at most s^2 / 4
    (stochastic) a product of K terms is off by about sqrt(K) times the
    operands' errors; five times that bounds the root mean square."""
    g = torch.Generator().manual_seed(0)
    T, I, O = 512, 256, 384
    x, w, d = (torch.randn(s, generator=g) for s in ((T, I), (I, O), (T, O)))
    lin = Int8Linear(I, O, seed=1, weight=w.cuda())
    xg = x.cuda().requires_grad_(True)
    lin(xg).backward(d.cuda())
    metis.status_sync()
    for got, ref, k in ((xg.grad, d @ w.T, O), (lin.weight.grad, x.T @ d, T)):
        step = 5.0 / 127  # lines of a few hundred Gaussians reach 5 at most here
        assert max(t.abs().max() for t in (x, w, d)) < 5
        rms = (got.cpu() - ref).pow(2).mean().sqrt()
        assert rms <= 5 * np.sqrt(k * step ** 2 * (1 / 12 + 1 / 4))


def test_layer_partial_gradients_batched_input_and_frozen_form():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(4, 10, 96, generator=g).to(torch.bfloat16).cuda()
    lin = Int8Linear(96, 80, weight=torch.randn(96, 80, generator=g).cuda(), rounding="rne")
    d = torch.randn(4, 10, 80, generator=g).to(torch.bfloat16).cuda()
    xg = x.clone().requires_grad_(True)
    y = lin(xg)
    assert tuple(y.shape) == (4, 10, 80)
    y.backward(d)
    full = (y.detach(), xg.grad.clone(), lin.weight.grad.clone())
    # the weight alone, the input alone, an expanded (stride 0) gradient
    lin.weight.grad = None
    lin(x).backward(d)
    assert torch.equal(lin.weight.grad, full[2])
    lin.weight.requires_grad_(False)
    xh = x.clone().requires_grad_(True)
    lin(xh).backward(d)
    assert torch.equal(xh.grad, full[1])
    xs = x.clone().requires_grad_(True)
    lin(xs).sum().backward()
    xe = x.clone().requires_grad_(True)
    lin(xe).backward(torch.ones(4, 10, 80, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(xs.grad, xe.grad)
    frozen = lin.frozen()
    assert torch.equal(frozen(x), full[0]) and not any(p.requires_grad for p in frozen.parameters())
    copy = Int8Linear(96, 80).frozen()
    copy.load_state_dict(frozen.state_dict())
    assert torch.equal(copy(x), full[0])
    metis.status_sync()


def test_layer_odd_inputs():
    """Transposed, expanded and one-dimensional inputs, and no tokens at all."""
    g = torch.Generator().manual_seed(4)
    lin = Int8Linear(48, 20, weight=torch.randn(48, 20, generator=g).cuda(), rounding="rne")
    x = torch.randn(48, 30, generator=g).cuda()
    assert torch.equal(lin(x.T), lin(x.T.contiguous()))
    one = torch.randn(48, generator=g).cuda()
    want = lin(one[None].contiguous())
    assert torch.equal(lin(one), want[0]) and torch.equal(lin(one.expand(5, 48)), want.expand(5, 20))
    frozen = lin.frozen()
    assert torch.equal(frozen(one), want[0]) and torch.equal(frozen(x.T), lin(x.T))
    none = torch.zeros(2, 0, 48, device="cuda", requires_grad=True)
    y = lin(none)
    assert tuple(y.shape) == (2, 0, 20) and tuple(frozen(none).shape) == (2, 0, 20)
    y.sum().backward()
    assert tuple(none.grad.shape) == (2, 0, 48) and not lin.weight.grad.any()
    metis.status_sync()


def test_layer_in_a_graph():
    """A forward and backward pass captured and replayed on new inputs, and
    refused while a graph from outside the capture lives."""
    g = torch.Generator(device="cuda").manual_seed(5)
    lin = Int8Linear(64, 40, weight=torch.randn(64, 40, generator=g, device="cuda"))
    x = torch.randn(50, 64, generator=g, device="cuda", requires_grad=True)
    d = torch.randn(50, 40, generator=g, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lin(x).backward(d)
    torch.cuda.current_stream().wait_stream(side)
    x.grad = lin.weight.grad = None
    alive = lin(x.detach())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d += 0
        with pytest.raises(RuntimeError, match="alive"):
            lin(x)
    del alive
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lin(x)
        y.backward(d)
    for i in range(3):
        xi = torch.randn(50, 64, generator=g, device="cuda") * (i + 1)
        di = torch.randn(50, 40, generator=g, device="cuda")
        with torch.no_grad():
            x.copy_(xi)
            d.copy_(di)
        x.grad.zero_()
        lin.weight.grad.zero_()
        graph.replay()
        torch.cuda.synchronize()
        twin = Int8Linear(64, 40, weight=lin.weight.detach())
        xt = xi.clone().requires_grad_(True)
        yt = twin(xt)
        yt.backward(di)
        assert torch.equal(y, yt) and torch.equal(x.grad, xt.grad) and torch.equal(lin.weight.grad, twin.weight.grad)
    metis.status_sync()


def test_other_stream_and_graph_replays():
    """Calls on a side stream, and a captured linear replayed on new inputs
    between eager work."""
    rng = np.random.default_rng(8)
    w = _upload(_random(rng, 300, 700))
    x = torch.randn(20, 700, device="cuda")
    want = metis.int8_linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = metis.int8_linear(x, w)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    static = x.clone()
    metis.init_device()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = metis.int8_quantize(static, BOTH, rounding=metis.SR, seed=4)
        y = metis.int8_linear(static, w)
        z = metis.int8_gemm(q.ax0, q.ax0)
    for i in range(4):
        fresh = torch.randn(20, 700, device="cuda") * (i + 1)
        static.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        e = metis.int8_quantize(fresh, BOTH, rounding=metis.SR, seed=4)
        assert torch.equal(y, metis.int8_linear(fresh, w))
        assert torch.equal(q.ax0.codes, e.ax0.codes) and torch.equal(q.ax1.codes, e.ax1.codes)
        assert torch.equal(z, metis.int8_gemm(e.ax0, e.ax0))
    metis.status_sync()


def test_same_operand_on_both_sides_and_repeatability():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(400, 300, generator=g, device="cuda")
    q = metis.int8_quantize(x).ax1
    C = metis.int8_gemm(q, q)
    assert torch.equal(C, metis.int8_gemm(q, q))
    metis.status_sync()
    a = (q.codes.cpu().numpy()[:, :300], q.scales.cpu().numpy())
    assert np.array_equal(C.cpu().numpy(), _gemm32(a, a))
