"""Full forgetting and strong decays where the scan takes them another way:
wide keys, whose pairs are formed in two passes, and sequences that are cut
into segments.  Tolerances of test_scan_gpu.py."""
import pytest
import torch

from test_scan_gpu import OPS, compare, inputs

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")


def decays(kind):
    def change(ld, g):
        r = torch.rand(ld.shape, generator=g)
        if kind == "erase":
            return torch.where(r < 0.02, -torch.inf, ld)
        if kind == "erase often":
            return torch.where(r < 0.5, -torch.inf, ld)
        if kind == "one half of the keys":  # strong in one pass of keys only
            half = torch.arange(ld.shape[-1]) < ld.shape[-1] // 2
            return torch.where(half, -20 * r, ld)
        if kind == "the other half":
            half = torch.arange(ld.shape[-1]) < ld.shape[-1] // 2
            return torch.where(half, ld, -20 * r)
        if kind == "no more than once":  # one row forgets everything
            ld = ld.clone()
            ld[len(ld) // 2] = -torch.inf
            return ld
        assert kind == "mixed"
        return torch.where(r < 0.3, -40 * r, torch.where(r < 0.6, torch.zeros_like(ld), ld))
    return change


@needs_gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["erase", "erase often", "one half of the keys", "the other half", "mixed"])
def test_wide_keys(op, dtype, kind):
    x, cu, do, ds = inputs(op, [150, 20], 2, 128, 32, dtype, seed=5, decay=decays(kind))
    compare(op, x, cu, do, ds, dtype)


@needs_gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("kind", ["erase", "no more than once", "mixed"])
def test_segments(op, kind):
    x, cu, do, ds = inputs(op, [2700], 2, 32, 32, torch.float32, seed=6, decay=decays(kind))
    compare(op, x, cu, do, ds, torch.float32)
