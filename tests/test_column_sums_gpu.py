"""Gradients of the norms' per-column weights where one row is 2^24 of the
others: a sum over rows loses none of them, and is rounded once (2^-24)."""
import pytest
import torch

from sequence_ref import far

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
BIG = 2.0 ** 24


@needs_gpu
@pytest.mark.parametrize("rows,D", [(1000, 100), (1023, 37)])
def test_scale_of_a_residual(rows, D):
    """dscale = sum over rows of y, where only x' is used."""
    import recurrent_state_update_amd as rsu
    x = torch.zeros(rows, D, device="cuda")
    y = torch.ones(rows, D, device="cuda")
    y[5] = BIG
    scale = torch.ones(D, device="cuda", requires_grad=True)
    out, _ = rsu.residual_norm(x, y, scale)
    (got,) = torch.autograd.grad(out.sum(), scale)
    assert far(got, torch.full((D,), BIG + rows - 1, dtype=torch.float64)) <= 2.0 ** -24


@needs_gpu
def test_weight_of_a_residual_norm():
    """dweight = sum over rows of dh rms(x): x = 1 and eps below its rounding,
    so rms(x) = 1."""
    import recurrent_state_update_amd as rsu
    rows, D = 1000, 64
    x = torch.ones(rows, D, device="cuda")
    dh = torch.ones(rows, D, device="cuda")
    dh[7] = BIG
    weight = torch.ones(D, device="cuda", requires_grad=True)
    _, h = rsu.residual_norm(x, weight=weight, eps=1e-12, dtype=torch.float32)
    (got,) = torch.autograd.grad(h, weight, dh)
    assert far(got, torch.full((D,), BIG + rows - 1, dtype=torch.float64)) <= 2.0 ** -24
