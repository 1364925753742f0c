"""Scales of residual_norm_fp8 for what holds zeros only: tiny, above zero and finite,
whatever the rest of the row and eps are, so that a division by them stays finite.  The
scales of other groups are within the roundings that test_norm_fp8_gpu.py counts (80 of
2^-24 of a row's largest)."""
import pytest
import torch

from layer_ref import UNIT, norm_ref

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")


def norm(x, eps=1e-6, **kw):
    import recurrent_state_update_amd as rsu
    _, h, s = rsu.residual_norm_fp8(x.cuda(), eps=eps, **kw)
    return h.float().cpu(), s.cpu()


def tiny(s):
    return bool(((s > 0) & (s < 1e-28)).all())


@needs_gpu
@pytest.mark.parametrize("D", [256, 512, 2048, 4096, 8192, 16384])
def test_groups_of_zeros_in_large_rows(D):
    big = torch.tensor([1e-20, 1.0, 1e12, 3e12, 5e12, 1e15, 1e16])
    x = big[:, None] * torch.randn(len(big), D, generator=torch.Generator().manual_seed(D))
    x[:, :128] = 0
    x[3, -128:] = 0
    h, s = norm(x, group=128)
    assert tiny(s[:, 0]) and tiny(s[3, -1])
    assert not h[:, :128].any() and not h[3, -128:].any()
    want = norm_ref(x, None, None, None, 1e-6)[1].unflatten(-1, (-1, 128)).abs().amax(-1)
    live = want > 0
    assert ((s.double() * 448 - want).abs() <= 80 * UNIT * want.amax(1, keepdim=True))[live].all()


@needs_gpu
@pytest.mark.parametrize("D,group", [(256, 128), (256, None), (100, None), (1531, None), (4096, 128), (16384, None)])
@pytest.mark.parametrize("eps", [1e-30, 1e-6, 1.0, 1e20, 1e28])
def test_rows_of_zeros(D, group, eps):
    x = torch.zeros(3, D)
    x[1] = 1
    h, s = norm(x, eps=eps, group=group)
    assert not h[0].any() and not h[2].any() and torch.isfinite(s).all()
    assert ((s[0] > 0) & (s[2] > 0)).all()


@needs_gpu
def test_beside_infinities_and_nan():
    x = torch.zeros(4, 512)
    x[0, 300], x[1, 300], x[2, 300], x[3, 300] = float("inf"), -float("inf"), float("nan"), 1e30
    h, s = norm(x, group=128)
    zeros = [0, 1, 3]  # (column 300 is in the third group)
    for r in (0, 1, 3):
        assert tiny(s[r, zeros]), r
    assert torch.isnan(s[:2, 2]).all() and torch.isnan(s[2]).all() and torch.isnan(h[2]).all()
