"""Layer norm at the ends of its ranges."""

import pytest
import torch

from spectral_split_quantized_amd import metis

from gpu_helpers import say

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X; none is visible")
    metis.load()
    torch.cuda.set_device(0)
    metis.init_device()


def _signs(cols, block):
    """Ones whose sign changes every `block` columns."""
    full = -(-cols // (2 * block))
    return torch.tensor([1.0, -1.0], device="cuda").to(BF).repeat_interleave(block).repeat(full)[:cols].clone().view(1, cols)


def test_rows_of_more_columns_than_a_launch_has_work_items_for():
    """2^28 + 77 columns: sums of dweight and dbias over more workgroups' columns than one launch takes."""
    cols = (1 << 28) + 77
    say("layer norm of %d columns" % cols)
    x, dy = _signs(cols, 1024), _signs(cols, 2048)
    y, mean, rstd = metis.layernorm(x)
    # sums of ones of both signs are exact, and the mean is below 2^-17; so are squares within 2^-16 of one
    assert mean.abs().item() < 2.0 ** -17 and abs(rstd.item() - 1) < 2.0 ** -15
    assert torch.equal(y, x)  # (a value is off by less than bf16's step, and rounds to 1)
    dx, dw, db = metis.layernorm_bwd(dy, x, mean, rstd)
    say("backward done")
    assert torch.equal(db.view_as(dy), dy.float())
    h = (x.float() - mean) * rstd
    assert ((dw - (h * dy.float()).view(-1)).abs().max() <= 2.0 ** -22)  # one rounding, and that of the centred value
    assert torch.equal(dx, dy)


def test_rows_of_the_longest_length():
    """2^31 - 1 columns."""
    cols = (1 << 31) - 1
    say("layer norm of %d columns" % cols)
    x, dy = _signs(cols, 1024), _signs(cols, 2048)
    y, mean, rstd = metis.layernorm(x)
    assert mean.abs().item() < 2.0 ** -17 and abs(rstd.item() - 1) < 2.0 ** -15
    assert torch.equal(y, x)
    del y
    say("forward done")
    dx, dw, db = metis.layernorm_bwd(dy, x, mean, rstd)
    say("backward done")
    assert torch.equal(dx, dy)
    assert bool((db.view_as(dy) == dy).all())
    dw.abs_()
    assert dw.min() > 1 - 2.0 ** -14 and dw.max() < 1 + 2.0 ** -14
