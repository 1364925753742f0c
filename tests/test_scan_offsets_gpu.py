"""Packed sequences that do not fill their tensors, and offsets that are no
offsets."""
import pytest
import torch

import recurrent_state_update_amd as rsu
from test_scan_gpu import OPS, gpu_run, inputs

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")


def guarded(rows, *shape, dtype=torch.float32):
    """A tensor with a guard row of fives on either side, fives itself."""
    return torch.full((rows + 2, *shape), 5.0, dtype=dtype, device="cuda")


def both_passes(op, x, cu, T, H, d, do, ds):
    """dl_scan and dl_scan_backward over outputs that hold fives; checks every
    guard and returns the outputs."""
    x = {n: None if t is None else t.cuda() for n, t in x.items()}
    p = {n: None if t is None else t.data_ptr() for n, t in x.items()}
    N, delta = len(cu) - 1, op != "rwkv6"
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    desc = rsu.dl_scan_desc(rsu.OPS[op], 0, T, N, H, d, d, 0, 0, 0, cut.data_ptr(), p["q"], p["k"], p["v"], p["beta"],
                            p["log_decay"], p["u"])
    sizes = [rsu.dl_scan_workspace_bytes(desc), rsu.dl_scan_saved_bytes(desc), rsu.dl_scan_backward_workspace_bytes(desc)]
    ws, saved, ws2 = (torch.full((n + 512,), 7, dtype=torch.uint8, device="cuda") for n in sizes)
    out = dict(o=guarded(T, H, d), state=guarded(N, H, d, d), dq=guarded(T, H, d), dk=guarded(T, H, d), dv=guarded(T, H, d),
               dbeta=guarded(T, H) if delta else None, dlog_decay=guarded(T, H) if op == "gdn" else guarded(T, H, d),
               du=None if delta else guarded(H, d), dinitial_state=guarded(N, H, d, d))
    a = {n: None if t is None else t[1:-1] for n, t in out.items()}
    assert rsu.dl_scan(desc, x["initial_state"], a["state"], None, 0, a["o"], saved, ws) == 0
    assert rsu.dl_scan_backward(desc, saved, do.cuda(), ds.cuda(), a["dq"], a["dk"], a["dv"], a["dbeta"], a["dlog_decay"],
                                a["du"], a["dinitial_state"], ws2) == 0
    torch.cuda.synchronize()
    for n, t in out.items():
        assert t is None or ((t[0] == 5).all() and (t[-1] == 5).all()), n
    for b, n in zip((ws, saved, ws2), sizes):
        assert (b[n:] == 7).all()
    return {n: t for n, t in a.items() if t is not None}


@needs_gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("before,lens,tail", [(1, [5], 0), (37, [63, 50], 10), (64, [64], 0), (130, [0, 70, 0], 3), (200, [0], 0)])
def test_rows_ahead_of_the_first_sequence(op, before, lens, tail):
    """They take no part, whatever they hold, and are zero in every output."""
    T, H, d = before + sum(lens) + tail, 2, 16
    x, cu, do, ds = inputs(op, lens, H, d, d, torch.float32, seed=before, tail=tail)
    want = gpu_run(op, x, cu, do, ds)
    y = {n: t if t is None or n in ("u", "initial_state") else
         torch.cat([torch.full((before, *t.shape[1:]), float("nan")), t]) for n, t in x.items()}
    got = both_passes(op, y, [before + c for c in cu], T, H, d, torch.cat([torch.full((before, H, d), float("nan")), do]), ds)
    assert set(got) == set(want)
    for n, t in got.items():
        if n in ("state", "dinitial_state", "du"):
            assert torch.equal(t, want[n]), n
        else:
            assert not t[:before].any() and torch.equal(t[before:], want[n]), n


@needs_gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("T,sets", [
    (100, ([0, 70, 30, 100], [0, 200, 300, 400], [-50, -20, 40, 1 << 30], [100, 0, 0, 0])),
    # cut into segments
    (6400, ([0, 6000, 200, 6400], [-5, 1 << 30, -7, 3000], [6400, 0, 6400, 0], [6000, 100, 9000, 6400]))], ids=["short", "long"])
def test_bad_offsets_in_both_passes(op, T, sets):
    """Offsets out of order or out of range: meaningless results, no access
    outside the tensors."""
    H, d = 2, 32
    x, _, do, _ = inputs(op, [T], H, d, d, torch.float32, init=False)
    for cu in sets:
        both_passes(op, x, cu, T, H, d, do, torch.zeros(len(cu) - 1, H, d, d))
