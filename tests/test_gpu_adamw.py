"""GPU tests of the AdamW step (metis_adamw_step), the gradient norm
(metis_grad_norm) and the optimizer on them, against oracle/adamw.py.

Moments, codes and scales are defined to the last bit and compared for
equality.  A parameter p' = p d - c m / (r k + eps) is held to
4 * 2^-24 |p| (the roundings of d, of the product and of the difference) plus
16 * 2^-24 of the step's largest terms: c, m (three roundings), r (v: five
roundings, halved by the root, and the root's), k, eps, the product, the sum,
the hardware reciprocal (two half units) and the two products after it.  A
bf16 parameter adds half a unit, 2^-8 relative to nearest, a whole one
stochastically."""

import copy

import numpy as np
import pytest
import torch

from oracle import adamw
from spectral_split_quantized_amd import metis, optim
from spectral_split_quantized_amd.layer import Int8Linear

from gpu_helpers import say

pytestmark = pytest.mark.gpu

LR, BETAS, EPS, DECAY = 1e-2, (0.9, 0.999), 1e-8, 0.1
SIZES = [1, 3, 4, 5, 63, 255, 256, 257, 1023, 1024, 1025, 4095, 4096, 4097, 9000, 0, 20000]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X; none is visible")
    metis.load()
    torch.cuda.set_device(0)


def _np(t):
    return t.detach().float().cpu().numpy().reshape(-1)


def _codes(t):
    return t.view(torch.uint8).cpu().numpy().reshape(-1)


class Case:
    """Parameters, gradients and states on both sides."""

    def __init__(self, sizes, bits, p_dtype=torch.float32, g_dtype=torch.float32, seed=0, misaligned=False):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda n, s: torch.randn(n, generator=g) * s * torch.exp(3 * torch.randn(n, generator=g))  # noqa: E731
        def up(x, dtype):
            buf = torch.empty(x.numel() + 1, dtype=dtype, device="cuda")[1 if misaligned else 0:][:x.numel()]
            return buf.copy_(x)
        self.p = [up(rnd(n, 0.02), p_dtype) for n in sizes]
        self.g = [up(rnd(n, 1e-3), g_dtype) for n in sizes]
        m, r = [rnd(n, 1e-3).numpy() for n in sizes], [np.abs(rnd(n, 1e-3).numpy()) for n in sizes]
        for x in r:
            x[::7] = 0.0  # moments of elements without a gradient so far
        for x in m:
            x[::7] = 0.0
        self.bits = bits
        if bits == 32:
            self.m = [up(torch.from_numpy(x), torch.float32) for x in m]
            self.v = [up(torch.from_numpy(x * x), torch.float32) for x in r]
            self.ms = self.vs = [None] * len(sizes)
        else:
            def enc(xs, positive):
                pairs = [adamw.encode(x, positive=positive) for x in xs]
                return ([up(torch.from_numpy(c), torch.uint8).view(torch.float8_e4m3fn) for c, _ in pairs],
                        [torch.from_numpy(s).cuda() for _, s in pairs])
            self.m, self.ms = enc(m, False)
            self.v, self.vs = enc(r, True)

    def expect(self, t, clip=None, rounding="rne", seed=0, tags=None, b=BETAS):
        out = []
        for i in range(len(self.p)):
            p, g = _np(self.p[i]), _np(self.g[i])
            if clip is not None:
                g = g * np.float32(clip)
            if self.bits == 8:
                m = adamw.decode(_codes(self.m[i]), self.ms[i].cpu().numpy())
                v = adamw.decode(_codes(self.v[i]), self.vs[i].cpu().numpy()) ** 2
            else:
                m, v = _np(self.m[i]), _np(self.v[i])
            m1, v1, r1 = adamw.moments(g, m, v, *b)
            p1, _, _ = adamw.step(p, g, m, v, LR, *b, EPS, DECAY, t)
            den = r1.astype(np.float64) / np.sqrt(1 - b[1] ** t) + EPS
            tol = 2.0 ** -24 * (4 * np.abs(p) + 16 * LR / (1 - b[0] ** t) * (b[0] * np.abs(m) + (1 - b[0]) * np.abs(g)) / den)
            if self.p[i].dtype == torch.bfloat16:
                tol += np.abs(p1) * (2.0 ** -7 if rounding == "sr" else 2.0 ** -8) + 1e-40
            e = {"p": p1, "tol": tol}
            if self.bits == 8:
                tag = metis.make_tag(i, metis.OPERAND_W) if tags is None else tags[i]
                lo, hi = adamw.draws(len(p), seed, tag, t) if rounding == "sr" else (None, None)
                (e["m"], e["ms"]), (e["v"], e["vs"]) = adamw.encode(m1, lo), adamw.encode(r1, hi, True)
            else:
                e["m"], e["v"] = m1, v1
            out.append(e)
        return out

    def check(self, expect):
        for i, e in enumerate(expect):
            if not len(e["p"]):
                continue
            if self.bits == 8:
                assert np.array_equal(self.ms[i].cpu().numpy(), e["ms"]) and np.array_equal(self.vs[i].cpu().numpy(), e["vs"])
                assert np.array_equal(_codes(self.v[i]), e["v"]), "r codes of tensor %d" % i
                assert np.array_equal(_codes(self.m[i]), e["m"]), "m codes of tensor %d" % i
            else:
                assert np.array_equal(_np(self.m[i]), e["m"]) and np.array_equal(_np(self.v[i]), e["v"])
            err = np.abs(_np(self.p[i]).astype(np.float64) - e["p"])
            assert np.all(err <= e["tol"]), "tensor %d: %g of %g" % (i, (err - e["tol"]).max(), err.max())

    def step(self, t, **kw):
        metis.adamw_step(self.p, self.g, self.m, self.v, self.ms, self.vs, lr=LR, betas=BETAS, eps=EPS,
                         weight_decay=DECAY, step=t, **kw)


@pytest.mark.parametrize("misaligned", [False, True])
@pytest.mark.parametrize("rounding", ["rne", "sr"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype,g_dtype", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16),
                                             (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_step_against_oracle(p_dtype, g_dtype, bits, rounding, misaligned):
    say("adamw %d bits, %s / %s, %s, misaligned %s" % (bits, p_dtype, g_dtype, rounding, misaligned))
    c = Case(SIZES, bits, p_dtype, g_dtype, 1, misaligned)
    for t in (1, 2, 1000):
        want = c.expect(t, rounding=rounding, seed=0x123456789A)
        c.step(t, rounding=metis.SR if rounding == "sr" else metis.RNE, seed=0x123456789A)
        metis.status_sync()
        c.check(want)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_holds(bits):
    sizes = [(37 * i) % 700 for i in range(200)]
    say("adamw %d tensors, %d bits" % (len(sizes), bits))
    c = Case(sizes, bits, seed=2)
    want = c.expect(3)
    c.step(3)
    metis.status_sync()
    c.check(want)


def test_mixed_widths_and_types_in_one_call():
    a, b = Case([300, 5000], 8, torch.bfloat16, torch.bfloat16, 3), Case([4097, 10], 32, seed=4)
    want = a.expect(5, tags=[11, 22], rounding="sr", seed=1), b.expect(5)
    order = [0, 2, 1, 3]
    join = lambda k: [(getattr(a, k) + getattr(b, k))[i] for i in order]  # noqa: E731
    metis.adamw_step(*(join(k) for k in ("p", "g", "m", "v", "ms", "vs")), lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY,
                     step=5, rounding=metis.SR, seed=1, tags=[11, 0, 22, 0])
    metis.status_sync()
    a.check(want[0])
    b.check(want[1])


def test_stochastic_bf16_parameters_are_unbiased():
    """A step a twentieth of the parameter's spacing moves it by the right amount on average."""
    n = 1 << 16
    p = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    g = torch.full((n,), -1.0, device="cuda")
    m, v, _, _ = metis.adamw_state(n, 32)
    lr = 2.0 ** -7 / 20
    metis.adamw_step([p], [g], [m], [v], lr=lr, weight_decay=0.0, step=1, rounding=metis.SR, seed=5)
    metis.status_sync()
    up = (p.float() - 1).mean().item()
    assert set(p.float().unique().tolist()) == {1.0, 1 + 2.0 ** -7}
    # the share of n draws at 1/20, five standard deviations
    assert abs(up - lr) < 5 * 2.0 ** -7 * np.sqrt(0.05 * 0.95 / n)


def test_slow_moments_move_on_average():
    """Constant gradients: r approaches |g| through steps far below its
    spacing D <= r / 8 (to nearest it would stand still).  The codes keep the
    mean of r in each step; the mean of v = r^2 gains their variance, at most
    D times the step d = (1 - b2) (g^2 - v) / 2 r, so v moves at a rate
    between 1 and 1 + 1/16 times the exact one: v / g^2 lies between
    1 - b2^T and 1 - b2^(17/16 T).  Half a percent for the mean over n draws."""
    n, T = 1 << 14, 400
    p = torch.zeros(n, device="cuda")
    g = torch.full((n,), 0.3, device="cuda")
    g[::256] = 1.0
    m, v, ms, vs = metis.adamw_state(n, 8)
    for t in range(1, T + 1):
        metis.adamw_step([p], [g], [m], [v], [ms], [vs], lr=0.0, step=t, rounding=metis.SR, seed=2)
    metis.status_sync()
    r = v.float().view(-1, 256) * vs[:, None]
    mean = r[:, 1:].mean().item()
    low, high = (0.3 * np.sqrt(1 - BETAS[1] ** (T * k)) for k in (1, 17 / 16))
    assert low * 0.995 < mean < high * 1.005


def test_non_finite_updates_leave_the_element_and_are_reported():
    for bits in (32, 8):
        say("adamw non-finite gradients, %d bits" % bits)
        c = Case([600], bits, seed=6)
        want = c.expect(2)  # the other elements do not depend on these three
        c.g[0][5], c.g[0][300], c.g[0][599] = float("nan"), float("inf"), 1e30
        before = [t.clone() for t in (c.p[0], c.m[0], c.v[0])]
        c.step(2)
        with pytest.raises(metis.MetisError) as ei:
            metis.status_sync()
        assert ei.value.status == metis.E_NUMERIC
        bad = [5, 300, 599]
        good = [i for i in range(600) if i not in bad]
        assert torch.equal(c.p[0][bad], before[0][bad])
        err = np.abs(_np(c.p[0]) - want[0]["p"])
        assert np.all(err[good] <= want[0]["tol"][good])
        if bits == 32:
            assert torch.equal(c.m[0][bad], before[1][bad]) and torch.equal(c.v[0][bad], before[2][bad])
        else:
            assert torch.isfinite(c.m[0].float()).all() and torch.isfinite(c.ms[0]).all() and torch.isfinite(c.vs[0]).all()


def test_zero_eps_and_zero_gradient_is_not_finite_but_contained():
    p = torch.ones(10, device="cuda")
    m, v, _, _ = metis.adamw_state(10, 32)
    metis.adamw_step([p], [torch.zeros(10, device="cuda")], [m], [v], lr=0.1, eps=0.0, step=1)
    with pytest.raises(metis.MetisError):
        metis.status_sync()
    assert bool((p == 1).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grad_norm(dtype):
    g = torch.Generator().manual_seed(4)
    sizes = [1, 0, 5, 16383, 16384, 16385, 40001] + [3] * 300
    grads = [(torch.randn(n, generator=g) * 10).to(dtype) for n in sizes]
    views = [torch.empty(n + 1, dtype=dtype, device="cuda")[1:].copy_(x) for n, x in zip(sizes, grads)]
    want = adamw.norm([x.float().numpy() for x in grads])
    for tensors in ([x.cuda() for x in grads], views):
        out = metis.grad_norm(tensors, 0.5)
        assert torch.equal(out, metis.grad_norm(tensors, 0.5))
        # binary64 sums: one rounding to binary32 each
        assert abs(out[0].item() - want) <= 2.0 ** -24 * want * 1.001
        assert abs(out[1].item() - 0.5 / (want + 1e-6)) <= 2.0 ** -24 * out[1].item() * 1.001
    assert metis.grad_norm(tensors, 1e9)[1].item() == 1.0 and metis.grad_norm(tensors)[1].item() == 1.0
    tensors[3][7] = float("nan")
    assert torch.isnan(metis.grad_norm(tensors, 0.5)).all()
    zero = metis.grad_norm([torch.zeros(5, device="cuda")], 1.0)
    assert zero.tolist() == [0.0, 1.0]


def test_more_than_two_to_the_31_elements():
    n = (1 << 31) + 300
    say("adamw over %d elements" % n)
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-3:] = 1.0
    m, v, ms, vs = metis.adamw_state(n, 8)
    metis.adamw_step([p], [g], [m], [v], [ms], [vs], lr=0.5, weight_decay=0.0, step=1)
    out = metis.grad_norm([g], 1.0)
    metis.status_sync()
    assert p[-5:].tolist() == [0, 0, -0.5, -0.5, -0.5] and not p[:-3].any()
    assert (m[-3:].float() * ms[-1]).tolist() == pytest.approx([0.1] * 3, rel=2.0 ** -4)
    assert out[0].item() == pytest.approx(3 ** 0.5, rel=2.0 ** -23)


def test_lists_are_checked():
    """What the library would write twice, or past an end, is refused before anything is enqueued."""
    buf = torch.zeros(200, device="cuda")
    g = torch.ones(100, device="cuda")
    new = lambda n=1: [torch.zeros(100, device="cuda") for _ in range(n)]  # noqa: E731

    def step(p, grads, m, v, ms=None, vs=None):
        metis.adamw_step(p, grads, m, v, ms, vs, lr=1.0, step=1)

    a, b = buf[:100], buf[99:199]
    for p, m, v in (([a, a], new(2), new(2)), ([a, b], new(2), new(2)), ([a], [a], new()), ([a], new(), [buf[50:150]])):
        with pytest.raises(ValueError, match="twice"):
            step(p, [g] * len(p), m, v)
    m = new()
    with pytest.raises(ValueError, match="twice"):
        step([a], [g], m, m)
    for p, gr, m, v in (([a], [g[:99]], new(), new()), ([a], [g], [m[0][:99]], new()), ([buf[::2]], [g], new(), new()),
                        ([a], [torch.ones(200, device="cuda")[::2]], new(), new()), ([a], [g.cpu()], new(), new())):
        with pytest.raises(ValueError):
            step(p, gr, m, v)
    for p, gr, m, v in (([a], [g.half()], new(), new()), ([a.half()], [g], new(), new()), ([a], [g], [m[0].half()], new()),
                        ([a], [g], [m[0].to(torch.float8_e4m3fn)], new()), ([a], [None], new(), new())):
        with pytest.raises(TypeError):
            step(p, gr, m, v)
    c, d, cs, ds = metis.adamw_state(100, 8)
    with pytest.raises(ValueError):
        step([a], [g], [c], [d], [cs], [None])
    with pytest.raises(ValueError):
        step([a], [g], [c], [d], [cs], [ds[:0]])
    with pytest.raises(TypeError):
        step([a], [g], new(), new(), [cs], [ds])
    step([a], [g], [c], [d], [cs], [ds])
    metis.status_sync()
    assert bool((a == -1).all()) and not buf[100:].any()


def test_gradients_may_share_memory_but_not_with_what_is_written():
    buf = torch.zeros(300, device="cuda")
    new = lambda n=1: [torch.zeros(100, device="cuda") for _ in range(n)]  # noqa: E731
    before = buf.clone()
    for g, p, m, v in ((buf[50:150], buf[:100], new(), new()), (buf[:100], buf[:100], new(), new()),
                       (buf[50:150], torch.zeros(100, device="cuda"), [buf[100:200]], new()),
                       (buf[199:299], torch.zeros(100, device="cuda"), new(), [buf[100:200]]),
                       (buf[:100].view(torch.bfloat16)[100:], buf[50:150], new(), new())):
        with pytest.raises(ValueError, match="overlap"):
            metis.adamw_step([p], [g[:100]], m, v, lr=1.0, step=1)
    torch.cuda.synchronize()
    assert torch.equal(buf, before)
    p, buf[:] = new(2), 1.0
    metis.adamw_step([*p, buf[200:]], [buf[:100], buf[50:150], buf[100:200]], new(3), new(3), lr=1.0, step=1)
    metis.status_sync()
    assert all(bool((x == -1).all()) for x in p) and not buf[200:].any() and bool((buf[:200] == 1).all())


# ----------------------------------------------------------- the optimizer --

def _params(seed=0, sizes=((50, 90), (90,), (64, 64), (1,))):
    g = torch.Generator().manual_seed(seed)
    ps = [torch.nn.Parameter(torch.randn(s, generator=g).cuda()) for s in sizes]
    return ps, g


def _set_grads(ps, g):
    for p in ps:
        p.grad = torch.randn(p.shape, generator=g).cuda() * 0.1


def test_optimizer_matches_the_formula_over_steps():
    """32-bit states against the float64 formula for ten steps, two groups,
    clipping, and a parameter without a gradient in some steps."""
    ps, g = _params()
    opt = optim.AdamW([{"params": ps[:2]}, {"params": ps[2:], "lr": 3e-3, "weight_decay": 0.0}], lr=1e-2, weight_decay=0.1,
                      state_bits=32, max_norm=1.0)
    ref = [(_np(p).astype(np.float64), 0.0, 0.0, 0) for p in ps]
    for t in range(10):
        _set_grads(ps, g)
        if t % 3 == 1:
            ps[1].grad = None
        opt.step()
        have = [p.grad for p in ps if p.grad is not None]
        norm = adamw.norm([_np(x) for x in have])
        assert opt.grad_norm.item() == pytest.approx(norm, rel=2.0 ** -23)
        coef = float(np.float32(min(1.0, 1.0 / (norm + 1e-6))))
        for i, p in enumerate(ps):
            if p.grad is None:
                continue
            q, m, v, k = ref[i]
            gr = _np(p.grad).astype(np.float64) * coef
            q, m, v = adamw.step(q, gr, m, v, 1e-2 if i < 2 else 3e-3, 0.9, 0.999, 1e-8, 0.1 if i < 2 else 0.0, k + 1)
            ref[i] = (q, m, v, k + 1)
    metis.status_sync()
    for p, (q, _, _, k) in zip(ps, ref):
        assert opt.state[p]["step"] == k
        # ten steps of at most lr each, relative roundings of a few units
        assert np.all(np.abs(_np(p) - q) <= 10 * (4 * 2.0 ** -24 * (np.abs(q) + 1) + 40 * 2.0 ** -24 * 1e-2))


def test_optimizer_state_widths_and_state_dict():
    ps, g = _params(1)
    opt = optim.AdamW(ps, lr=1e-2, seed=3)
    _set_grads(ps, g)
    opt.step()
    assert ["exp_avg_scale" in opt.state[p] for p in ps] == [True, False, True, False]  # 4500, 90, 4096 and 1 elements
    assert opt.state[ps[0]]["exp_avg"].dtype == torch.float8_e4m3fn
    # a copy goes on exactly as the original
    twins = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    other = optim.AdamW(twins, lr=5.0, seed=3)
    other.load_state_dict(opt.state_dict())
    assert other.param_groups[0]["lr"] == 1e-2
    for _ in range(3):
        _set_grads(ps, g)
        for a, b in zip(ps, twins):
            b.grad = a.grad.clone()
        opt.step()
        other.step()
    metis.status_sync()
    for a, b in zip(ps, twins):
        assert torch.equal(a, b)
        for k, s in opt.state[a].items():
            o = other.state[b][k]
            assert torch.equal(s.view(torch.uint8), o.view(torch.uint8)) if isinstance(s, torch.Tensor) else s == o


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_advances_on_every_replay(bits):
    say("captured adamw step, %d bits" % bits)
    ps, g = _params(2)
    twins = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    opt = optim.AdamW(ps, lr=1e-2, state_bits=bits, max_norm=0.5, capturable=True, seed=8)
    eager = optim.AdamW(twins, lr=1e-2, state_bits=bits, max_norm=0.5, seed=8)
    for p in ps:
        p.grad = torch.zeros_like(p)

    def feed():
        for a, b in zip(ps, twins):
            b.grad = torch.randn(a.shape, generator=g).cuda()
            a.grad.copy_(b.grad)

    feed()
    opt.step()  # states are made outside the capture
    eager.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for _ in range(4):
        feed()
        graph.replay()
        torch.cuda.synchronize()
        eager.step()
        assert torch.equal(opt.grad_norm, eager.grad_norm)
        for a, b in zip(ps, twins):
            for k in ("exp_avg", "exp_avg_sq"):
                assert torch.equal(opt.state[a][k].view(torch.uint8), eager.state[b][k].view(torch.uint8))
            # the bias corrections by squaring and by pow agree to binary64 rounding
            assert torch.allclose(a, b, rtol=2.0 ** -22, atol=2.0 ** -24 * 1e-2)
    assert all(opt.state[p]["step"].item() == 5 for p in ps)
    metis.status_sync()


def test_uncapturable_step_is_refused_in_a_capture():
    ps, g = _params(3)
    opt = optim.AdamW(ps, lr=1e-2)
    _set_grads(ps, g)
    opt.step()
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros(1, device="cuda")
    with torch.cuda.graph(graph):
        x += 1
        with pytest.raises(RuntimeError, match="capturable"):
            opt.step()
    graph.replay()
    torch.cuda.synchronize()


def test_closure_and_no_gradients():
    p = torch.nn.Parameter(torch.ones(5, device="cuda"))
    opt = optim.AdamW([p], lr=0.1, weight_decay=0.0, state_bits=32)

    def closure():
        opt.zero_grad()
        loss = (p * p).sum()
        loss.backward()
        return loss

    assert opt.step(closure).item() == 5.0 and bool((p < 1).all())
    before = p.detach().clone()
    opt.zero_grad()
    opt.step()
    assert torch.equal(p, before)


def test_first_step_in_a_capture_is_refused():
    ps, g = _params(5)
    opt = optim.AdamW(ps, capturable=True)
    _set_grads(ps, g)
    x = torch.zeros(1, device="cuda")
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        x += 1
        with pytest.raises(RuntimeError, match="before the capture"):
            opt.step()


def test_replaced_parameters_gradients_and_states_are_seen():
    """Between steps: a parameter's data on new memory, gradients of another
    type and layout, states moved by hand, and the optimizer copied."""
    ps, g = _params(6, ((70, 80), (4100,)))
    twins = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    opt, ref = (optim.AdamW(x, lr=1e-2, seed=1) for x in (ps, twins))
    for t in range(5):
        _set_grads(ps, g)
        for a, b in zip(ps, twins):
            b.grad = a.grad.clone()
        if t == 1:
            ps[0].data = ps[0].detach().clone()
        if t == 2:
            ps[0].grad = ps[0].grad.T.contiguous().T
        if t == 3:
            for s in opt.state.values():
                s["exp_avg"] = s["exp_avg"].clone()
                s["exp_avg_scale"] = s["exp_avg_scale"].clone()
        if t == 4:
            opt = copy.deepcopy(opt)
            for a, p in zip(ps, opt.param_groups[0]["params"]):
                p.grad = a.grad
            ps = opt.param_groups[0]["params"]
        opt.step()
        ref.step()
        assert all(torch.equal(a, b) for a, b in zip(ps, twins))
    metis.status_sync()


def test_quantised_network_trains():
    """Two int8 layers and the 8-bit optimizer together: every parameter gets
    a finite gradient and moves, and the frozen network equals the trained one."""
    g = torch.Generator().manual_seed(9)
    net = torch.nn.Sequential(Int8Linear(96, 200, layer=0), torch.nn.GELU(), Int8Linear(200, 64, layer=1))
    opt = optim.AdamW(net.parameters(), lr=1e-3, max_norm=1.0)
    x, y = (torch.randn(300, n, generator=g).cuda() for n in (96, 64))
    start = [p.detach().clone() for p in net.parameters()]
    for t in range(3):
        for m in (net[0], net[2]):
            m.step = t
        opt.zero_grad()
        (net(x) - y).pow(2).mean().backward()
        assert all(torch.isfinite(p.grad).all() for p in net.parameters())
        opt.step()
    metis.status_sync()
    assert all(not torch.equal(a, p) for a, p in zip(start, net.parameters()))
    frozen = torch.nn.Sequential(net[0].frozen(), torch.nn.GELU(), net[2].frozen())
    with torch.no_grad():
        assert torch.equal(frozen(x), net(x))
