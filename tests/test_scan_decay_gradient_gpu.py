"""The log-decay's gradient, channel by channel, where decays are strong: it
scales with e^ell, and no channel or row may carry the rounding of others that
are larger.

Tolerance: that of dlog_decay in test_scan_gpu.py (ten times FP32, for terms
that partly cancel), for every channel by itself, as |x - ref| / |ref| in the
2-norm over its rows (GDN: a head; else a key of a head)."""
import pytest
import torch

from test_scan_gpu import LD, OPS, gpu_run, inputs, ref_run

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")


def decays(kind):
    """A map of log-decays, and the rows to compare apart (none: all as one)."""
    strong = {}

    def change(ld, g):
        r = torch.rand(ld.shape, generator=g)
        if isinstance(kind, float):
            return kind * (1 + 0.05 * r)
        weak = -0.1 * r
        if kind == "channels":  # one in three
            c = torch.arange(ld.shape[-1]) % 3 == 1
            return torch.where(c, -12 - r, weak)
        if kind == "blocks":  # stretches of rows
            rows = torch.arange(len(ld)) // 10 % 2 == 1
        else:
            rows = torch.arange(len(ld)) % 7 == 3
        strong["rows"] = rows
        return torch.where(rows.view(-1, *[1] * (ld.dim() - 1)), -12 - 2 * r, weak)
    return change, strong


def worst(got, want, rows):
    """The largest relative distance of a channel, over the given rows."""
    got, want = got.double().cpu()[rows], want.detach()[rows]
    assert torch.isfinite(got).all()
    d, n = (got - want).norm(dim=0), want.norm(dim=0)
    assert (n > 0).all()
    return float((d / n).max())


@needs_gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dk,dtype", [(32, torch.float32), (128, torch.float32), (128, torch.bfloat16)],
                         ids=["32-f32", "128-f32", "128-bf16"])
@pytest.mark.parametrize("kind", [-8.0, -12.0, -16.0, "channels", "rows", "blocks"])
def test_channels(op, dk, dtype, kind):
    change, strong = decays(kind)
    x, cu, do, ds = inputs(op, [150, 70], 3, dk, 32, dtype, seed=11, decay=change)
    got, want = gpu_run(op, x, cu, do, ds)["dlog_decay"], ref_run(op, x, cu, do, ds)["dlog_decay"]
    rows = strong.get("rows")
    parts = [slice(None)] if rows is None else [rows, ~rows]
    errs = [worst(got, want, part) for part in parts]
    print(f"[scan {op}] dlog_decay, worst channel:", " ".join(f"{e:.1e}" for e in errs), flush=True)
    assert max(errs) <= LD
