"""GPU tests of the optimizer's states: step counts of their own, stored
values that are not finite, values kept beside a new maximum.

Moments, codes and scales are defined to the last bit and compared for
equality, with oracle/adamw.py or with an optimizer whose counts are host
integers."""

import numpy as np
import pytest
import torch

from oracle import adamw
from spectral_split_quantized_amd import metis, optim

from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X; none is visible")
    metis.load()
    torch.cuda.set_device(0)


def _params(seed, sizes):
    g = torch.Generator().manual_seed(seed)
    return [torch.nn.Parameter(torch.randn(s, generator=g).cuda()) for s in sizes], g


@pytest.mark.parametrize("bits", [32, 8])
def test_counts_that_differ_in_a_captured_step(bits):
    """A parameter that had no gradient in some steps, loaded into an optimizer
    whose counts are on the GPU: eager and replayed steps equal those of host
    counts, stochastic draws included."""
    say("adamw, counts that differ, %d bits" % bits)
    ps, g = _params(1, ((50, 90), (4100,), (700,)))
    twins = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    eager = optim.AdamW(twins, lr=1e-2, state_bits=bits, min_8bit_size=1, seed=8)
    for t in range(5):
        for i, p in enumerate(twins):
            p.grad = None if i == 1 and t % 2 else torch.randn(p.shape, generator=g).cuda()
        eager.step()
    opt = optim.AdamW(ps, lr=1e-2, state_bits=bits, min_8bit_size=1, capturable=True, seed=8)
    opt.load_state_dict(eager.state_dict())
    assert [int(opt.state[p]["step"]) for p in ps] == [5, 3, 5]
    for a, b in zip(ps, twins):
        a.data.copy_(b.data)
        a.grad = torch.zeros_like(a)

    def feed():
        for a, b in zip(ps, twins):
            b.grad = torch.randn(a.shape, generator=g).cuda()
            a.grad.copy_(b.grad)

    def check():
        torch.cuda.synchronize()
        eager.step()
        for a, b in zip(ps, twins):
            for k in opt.state[a]:
                if k != "step":
                    assert torch.equal(opt.state[a][k].view(torch.uint8), eager.state[b][k].view(torch.uint8)), k
            # the bias corrections by squaring and by pow agree to binary64 rounding
            assert torch.allclose(a, b, rtol=2.0 ** -22, atol=2.0 ** -24 * 1e-2)

    feed()
    opt.step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for _ in range(3):
        feed()
        graph.replay()
        check()
    assert [int(opt.state[p]["step"]) for p in ps] == [9, 7, 9]
    metis.status_sync()


BETAS, EPS = (0.9, 0.999), 1e-8


class Eight:
    """One tensor with 8-bit states that hold given moments."""

    def __init__(self, n, seed):
        rng = np.random.default_rng(seed)
        rnd = lambda s: (rng.standard_normal(n) * s * np.exp(rng.standard_normal(n))).astype(np.float32)  # noqa: E731
        self.p, self.g = torch.from_numpy(rnd(0.02)).cuda(), torch.from_numpy(rnd(1e-3)).cuda()
        (m, ms), (v, vs) = adamw.encode(rnd(1e-3)), adamw.encode(np.abs(rnd(1e-3)), positive=True)
        self.m, self.v = (torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in (m, v))
        self.ms, self.vs = torch.from_numpy(ms).cuda(), torch.from_numpy(vs).cuda()

    def codes(self):
        return [t.view(torch.uint8).cpu().numpy() for t in (self.m, self.v)]

    def scales(self):
        return [t.cpu().numpy() for t in (self.ms, self.vs)]

    def expect(self, bad, t, rounding, seed):
        """(m codes, scales), (r codes, scales) after a step in which the
        elements ``bad`` keep their moments."""
        (mc, vc), (ms, vs) = self.codes(), self.scales()
        m, r = adamw.decode(mc, ms), adamw.decode(vc, vs)
        with np.errstate(all="ignore"):
            m1, _, r1 = adamw.moments(self.g.cpu().numpy(), m, r * r, *BETAS)
        m1[bad], r1[bad] = m[bad], np.abs(r[bad])
        lo, hi = adamw.draws(len(m), seed, metis.make_tag(0, metis.OPERAND_W), t) if rounding == "sr" else (None, None)
        return adamw.encode(m1, lo), adamw.encode(r1, hi, True)

    def step(self, t, rounding, seed):
        metis.adamw_step([self.p], [self.g], [self.m], [self.v], [self.ms], [self.vs], lr=1e-2, betas=BETAS, eps=EPS, step=t,
                         rounding=metis.SR if rounding == "sr" else metis.RNE, seed=seed)

    def check(self, want):
        (mc, vc), (ms, vs) = self.codes(), self.scales()
        assert np.array_equal(ms, want[0][1]) and np.array_equal(vs, want[1][1])
        assert np.array_equal(mc, want[0][0]) and np.array_equal(vc, want[1][0])


def _reported():
    with pytest.raises(metis.MetisError) as ei:
        metis.status_sync()
    assert ei.value.status == metis.E_NUMERIC


@pytest.mark.parametrize("rounding", ["rne", "sr"])
def test_stored_nan_stays_in_its_element(rounding):
    """NaN codes in a state, a NaN, an infinite and a negative r in damaged
    blocks: the elements keep what they had, their neighbours go on."""
    say("adamw, NaN in stored states, %s" % rounding)
    s = Eight(1500, 3)
    s.m.view(torch.uint8)[5], s.m.view(torch.uint8)[6] = 0x7F, 0xFF      # NaN in m
    s.v.view(torch.uint8)[300] = 0x7F                                    # NaN in r
    s.ms[2], s.vs[3] = float("nan"), float("inf")                        # a block of each
    s.v.view(torch.uint8)[1030] |= 0x80                                  # a negative r whose update is not finite
    s.g[1030] = float("nan")
    bad = np.array([5, 6, 300, *range(512, 1024), 1030])
    before = s.p.clone()
    for t in (1, 2):
        want = s.expect(bad, t, rounding, 9)
        s.step(t, rounding, 9)
        _reported()
        s.check(want)
    assert torch.equal(s.p[bad], before[bad])
    good = np.setdiff1d(np.arange(1500), bad)
    assert bool((s.p[good] != before[good]).all()) and bool(torch.isfinite(s.p).all())
    mc, vc = s.codes()
    assert set(np.flatnonzero(mc & 0x7F == 0x7F)) == {5, 6, *range(512, 768)}
    assert set(np.flatnonzero(vc & 0x7F == 0x7F)) == {300, *range(768, 1024)}


@pytest.mark.parametrize("rounding", ["rne", "sr"])
def test_kept_moments_are_encoded_with_the_blocks_new_scale(rounding):
    """Gradients that are not finite beside one that raises the block's scales
    by many powers of two: every code and scale as the definition has it."""
    say("adamw, kept moments beside a new maximum, %s" % rounding)
    s = Eight(1100, 4)
    bad = np.array([0, 7, 255, 260, 700, 1099])
    s.g[bad] = torch.tensor([float("nan"), float("inf"), float("-inf"), 1e30, float("nan"), -1e25], device="cuda")
    s.g[20], s.g[300], s.g[1090] = 0.5, 30.0, -4.0
    before, kept = s.p.clone(), [c[bad] for c in s.codes()]
    want = s.expect(bad, 7, rounding, 11)
    assert any((w[0][bad] != k).any() for w, k in zip(want, kept))  # the case is met
    s.step(7, rounding, 11)
    _reported()
    s.check(want)
    assert torch.equal(s.p[bad], before[bad])
    r = adamw.decode(s.codes()[1], s.scales()[1])
    assert ((r[bad] > 0) == (kept[1] > 0)).all()


def test_autograd_sees_the_write():
    """A graph that saved a parameter refuses its backward pass after a step,
    as after any write in place."""
    p = torch.nn.Parameter(torch.ones(5, device="cuda"))
    opt = optim.AdamW([p], state_bits=32)
    for _ in range(2):  # the first step makes the states, the second finds them
        loss = (p * p).sum()
        p.grad = torch.ones(5, device="cuda")
        opt.step()
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    q = torch.ones(5, device="cuda")
    m, v, _, _ = metis.adamw_state(5, 32)
    before = q._version
    metis.adamw_step([q], [torch.ones(5, device="cuda")], [m], [v], lr=0.1, step=1)
    assert q._version == before + 1
    with torch.inference_mode():
        r = torch.ones(5, device="cuda")
    metis.adamw_step([r], [torch.ones(5, device="cuda")], [m], [v], lr=0.1, step=2)  # has no versions
    metis.status_sync()
    assert bool((r < 1).all())


@pytest.mark.parametrize("capturable", [False, True])
def test_norms_kept_over_steps(capturable):
    """Each step's norm is a tensor of its own; with capturable, one that every step writes."""
    p = torch.nn.Parameter(torch.zeros(9, device="cuda"))
    opt = optim.AdamW([p], max_norm=1.0, state_bits=32, capturable=capturable)
    norms = []
    for t in range(1, 4):
        p.grad = torch.full((9,), float(t), device="cuda")
        opt.step()
        norms.append(opt.grad_norm)
    assert [n.item() for n in norms] == ([9.0] * 3 if capturable else [3.0, 6.0, 9.0])
    metis.status_sync()
