"""GPU tests of the int8 layer beside its formulas: captured passes and their
steps.  The passes are defined to the last bit, so comparisons are for
equality."""

import copy

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
    metis.init_device()


@pytest.mark.parametrize("axes", [metis.AXIS0, metis.AXIS1, BOTH])
def test_quantize_with_a_step_on_the_gpu(axes):
    say("int8 quantize, step on the GPU, axes %d" % axes)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(130, 333, generator=g, device="cuda")
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    for step in (0, 1, 7, 2 ** 31 + 5, 4):
        count.fill_(-1 if step == 4 else step)  # negative: the call's own step
        a = metis.int8_quantize(x, axes, rounding=metis.SR, seed=3, tag=9, step=4, step_count=count)
        b = metis.int8_quantize(x, axes, rounding=metis.SR, seed=3, tag=9, step=step)
        for p, q in ((a.ax0, b.ax0), (a.ax1, b.ax1)):
            assert (p is None) == (q is None)
            assert p is None or torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
    metis.status_sync()


def test_captured_layer_takes_the_draws_of_the_step_that_is_set():
    say("int8 layer, replays at different steps")
    g = torch.Generator(device="cuda").manual_seed(5)
    lin = Int8Linear(64, 40, weight=torch.randn(64, 40, generator=g, device="cuda"), seed=2, layer=3)
    x = torch.randn(50, 64, generator=g, device="cuda", requires_grad=True)
    d = torch.randn(50, 40, generator=g, device="cuda")
    set_step(lin, 11)
    lin(x).backward(d)
    torch.cuda.synchronize()
    x.grad = lin.weight.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lin(x)
        y.backward(d)
        with pytest.raises(RuntimeError, match="outside the capture"):
            set_step(lin, 12)
    seen = []
    for step in (None, 12, 13, 13, 5):  # None: the step of the capture
        if step is not None:
            set_step(lin, step)
        assert lin.step == (11 if step is None else step)
        x.grad.zero_()
        lin.weight.grad.zero_()
        graph.replay()
        torch.cuda.synchronize()
        twin = Int8Linear(64, 40, weight=lin.weight.detach(), seed=2, layer=3)
        twin.step = lin.step
        xt = x.detach().clone().requires_grad_(True)
        yt = twin(xt)
        yt.backward(d)
        assert torch.equal(y, yt) and torch.equal(x.grad, xt.grad) and torch.equal(lin.weight.grad, twin.weight.grad)
        seen.append(x.grad.clone())
    assert torch.equal(seen[2], seen[3]) and not any(torch.equal(seen[i], seen[j]) for i, j in ((0, 1), (1, 2), (2, 4)))
    metis.status_sync()


def test_step_follows_copies_and_moves():
    x = torch.randn(5, 16, device="cuda", requires_grad=True)
    lin = Int8Linear(16, 8)
    lin.step = 4
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lin(x)
        assert lin.to("cuda").float() is lin  # the graph's address stays
    at = lin._count.data_ptr()
    assert lin._count.item() == -1
    lin.step = 5
    assert lin.to("cuda").float()._count.data_ptr() == at and lin._count.item() == lin.step == 5
    twin = copy.deepcopy(lin)
    twin.step = 6
    assert lin.step == 5 and twin.step == 6 and lin._count.item() == 5 and twin._count.data_ptr() != at
    moved = Int8Linear(16, 8, device="cpu")
    moved.step = 9
    moved = moved.to("cuda")
    assert moved.step == 9 and moved._count.is_cuda
    assert Int8Linear(16, 8, rounding="rne")._count is None and moved.cpu()._count is None
    del y


def _runs(a, b):
    """(the product in binary64, a bound of the binary32 errors): codes and
    scales of both sides, cut in runs of 130944 codes.  A run's product has
    three roundings of an exact sum, a sum of runs one for each addition."""
    total, size = 0.0, 0.0
    for k in range(0, a[0].shape[1], 130944):
        x, y = (q[0][:, k:k + 130944].astype(np.float64) for q in (a, b))
        part = x @ y.T * a[1].astype(np.float64)[:, None] * b[1].astype(np.float64)
        total, size = total + part, size + np.abs(part)
    return total, 2.0 ** -24 * 1.001 * (3 + a[0].shape[1] // 130944) * size


@pytest.mark.parametrize("tokens,cin,cout", [(131071, 6, 5), (131072, 20, 24), (262200, 5, 3), (5, 3, 131200), (4, 131200, 7)])
def test_reductions_longer_than_one_product(tokens, cin, cout):
    """Every product of the layer over more codes than int32 sums hold: tokens
    for dW, output features for dX, input features for Y."""
    say("int8 layer, %d tokens, %d -> %d" % (tokens, cin, cout))
    g = torch.Generator().manual_seed(tokens)
    x, w, d = (torch.randn(s, generator=g) for s in ((tokens, cin), (cin, cout), (tokens, cout)))
    lin = Int8Linear(cin, cout, seed=2, weight=w.cuda())
    lin.step = 3
    xg = x.cuda().requires_grad_(True)
    y = lin(xg)
    y.backward(d.cuda())
    metis.status_sync()
    x, w, d = x.numpy(), w.numpy(), d.numpy()
    q, sr = int8.quantize, ("sr", 2, metis.make_tag(0, metis.OPERAND_D), 3)
    for got, a, b in ((y, q(x, 1), q(w, 0)), (xg.grad, q(d, 1, *sr), q(w, 1)), (lin.weight.grad, q(x, 0), q(d, 0, *sr))):
        want, bound = _runs(a, b)
        assert np.all(np.abs(got.detach().cpu().numpy() - want) <= bound)
    # bfloat16: the sum of the runs is rounded once
    xb = torch.from_numpy(x).to(torch.bfloat16).cuda()
    got = lin(xb)
    want, bound = _runs(q(xb.float().cpu().numpy(), 1), q(w, 0))
    assert got.dtype == torch.bfloat16
    assert np.all(np.abs(got.detach().float().cpu().numpy() - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound))


def test_frozen_form_in_a_model_cast_to_bfloat16():
    g = torch.Generator().manual_seed(2)
    lin = Int8Linear(96, 40, weight=torch.randn(96, 40, generator=g).cuda(), rounding="rne")
    x = torch.randn(7, 96, generator=g).to(torch.bfloat16).cuda()
    frozen = lin.frozen()
    want = frozen(x)
    assert torch.equal(frozen.to(torch.bfloat16)(x), want) and torch.equal(frozen.cpu().bfloat16().cuda()(x), want)
    metis.status_sync()


def test_more_rows_than_one_launch_takes():
    """2^24 rows of 256 threads each are 2^32 work items: rows on both sides of
    the cut, against the same rows alone and the definition's draws."""
    rows, cols = (1 << 24) + 300, 520
    say("int8 quantize %d rows" % rows)
    g = torch.Generator(device="cuda").manual_seed(3)
    part = torch.randn(1000, cols, generator=g, device="cuda").to(torch.bfloat16)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[:1000] = part
    x[-1000:] = part
    q = metis.int8_quantize(x).ax1
    want = metis.int8_quantize(part).ax1
    for s in (slice(0, 1000), slice(rows - 1000, rows)):
        assert torch.equal(q.codes[s], want.codes) and torch.equal(q.scales[s], want.scales)
    assert not q.codes[1000:-1000].any()
    q = metis.int8_quantize(x, rounding=metis.SR, seed=5, tag=1, step=2).ax1
    metis.status_sync()
    from oracle import philox
    for row in (0, rows - 1000, rows - 301, rows - 300, rows - 1):
        e0 = row * cols
        u = philox.halves(np.arange(e0, e0 + cols, dtype=np.uint64), 5, 1, 2) / 65536
        xr = x[row].float().cpu().numpy()
        y = xr * (np.float32(1) / np.float32(np.abs(xr).max() / np.float32(127)))
        code = np.floor(y) + (u < y - np.floor(y))
        assert np.array_equal(q.codes[row, :cols].cpu().numpy(), np.clip(code, -127, 127).astype(np.int8))


def test_more_output_channels_than_one_launch_takes():
    """The kernels for a few tokens take 16 channels a workgroup of up to 512 threads."""
    n, k = (1 << 27) + 100, 100
    say("int8 linear to %d channels" % n)
    g = torch.Generator(device="cuda").manual_seed(4)
    base = metis.I8.from_codes(torch.randint(-127, 128, (1000, k), generator=g, dtype=torch.int8, device="cuda"),
                               torch.rand(1000, generator=g, device="cuda"))
    w = metis.I8(n, k)
    w.codes.zero_()
    w.scales.fill_(1.0)
    for s in (slice(0, 1000), slice(n - 1000, n)):
        w.codes[s] = base.codes
        w.scales[s] = base.scales
    for tokens in (1, 2):
        x = torch.randn(tokens, k, generator=g, device="cuda")
        for out in (torch.float32, torch.bfloat16):
            y = metis.int8_linear(x, w, out_dtype=out)
            want = metis.int8_linear(x, base, out_dtype=out)
            assert torch.equal(y[:, :1000], want) and torch.equal(y[:, -1000:], want) and not y[:, 1000:-1000].any()
    metis.status_sync()
