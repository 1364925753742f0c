"""Offsets that are no offsets, and packed sequences that do not fill their tensors, in
the state space layer's operators: nothing is written outside outputs, saved states and
workspaces, which lie between guards here."""
import pytest
import torch

import recurrent_state_update_amd as rsu
from test_short_conv_gpu import inputs as conv_inputs, run as conv_run
from test_ssm_gpu import inputs as ssm_inputs, run as ssm_run

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
GUARD = 4096  # elements (bytes) on either side: every output stays on its boundary


class Guards:
    """Outputs and workspaces between guards of fives."""

    def __init__(self):
        self.all = {}

    def out(self, name, *shape, dtype=torch.float32):
        n = int(torch.Size(shape).numel())
        t = self.all[name] = torch.full((n + 2 * GUARD,), 5, dtype=dtype, device="cuda")
        return t[GUARD:GUARD + n].view(shape)

    def bytes(self, name, n):
        return self.out(name, n, dtype=torch.uint8)

    def whole(self):
        torch.cuda.synchronize()
        for n, t in self.all.items():
            assert (t[:GUARD] == 5).all() and (t[-GUARD:] == 5).all(), n


def offsets(cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def conv_passes(x, cu, dy, dend):
    """dl_short_conv and its backward pass; the outputs, as `run` of test_short_conv_gpu.py
    names them."""
    v = {n: t.cuda() for n, t in x.items()}
    (T, C), W, N, dt = v["x"].shape, v["weight"].shape[1], len(cu) - 1, v["x"].dtype
    off, g = offsets(cu), Guards()
    d = rsu.dl_conv_desc(rsu.DTYPES[dt], T, N, C, W, 1, 0, off.data_ptr(), v["x"].data_ptr(), v["weight"].data_ptr(),
                         v["bias"].data_ptr())
    o = dict(y=g.out("y", T, C, dtype=dt), end=g.out("end", N, W - 1, C, dtype=dt), dx=g.out("dx", T, C, dtype=dt),
             dweight=g.out("dweight", C, W), dbias=g.out("dbias", C), dinitial=g.out("dinitial", N, W - 1, C, dtype=dt))
    ws = g.bytes("workspace", rsu.dl_short_conv_workspace_bytes(d))
    dy, dend = dy.cuda(), dend.cuda()
    assert rsu.dl_short_conv(d, v["initial"], o["end"], o["y"]) == 0
    assert rsu.dl_short_conv_backward(d, v["initial"], dy, dend, o["dx"], o["dweight"], o["dbias"], o["dinitial"], ws) == 0
    g.whole()
    return o


def ssm_passes(x, cu, dy, dend):
    """dl_ssm_scan and its backward pass; the outputs, as `run` of test_ssm_gpu.py names
    them."""
    v = {n: t.cuda() for n, t in x.items()}
    (T, C), S, N, dt = v["x"].shape, v["A"].shape[1], len(cu) - 1, v["x"].dtype
    G = v["B"].shape[1] if v["B"].dim() == 3 else 1
    off, g = offsets(cu), Guards()
    p = {n: t.data_ptr() for n, t in v.items()}
    d = rsu.dl_ssm_desc(rsu.DTYPES[dt], T, N, C, S, G, 1, 0, 0, 0, 0, 0, off.data_ptr(), p["x"], p["dt"], p["z"], p["B"],
                        p["C"], p["A"], p["D"], p["dt_bias"])
    rows = dict(dtype=dt)
    o = dict(y=g.out("y", T, C, **rows), end=g.out("end", N, C, S), dx=g.out("dx", T, C, **rows),
             ddt=g.out("ddt", T, C, **rows), dA=g.out("dA", C, S), dB=g.out("dB", *v["B"].shape, **rows),
             dC=g.out("dC", *v["B"].shape, **rows), dD=g.out("dD", C), dz=g.out("dz", T, C, **rows),
             ddt_bias=g.out("ddt_bias", C), dinitial=g.out("dinitial", N, C, S))
    ws, saved, ws2 = (g.bytes(n, f(d)) for n, f in (
        ("workspace", rsu.dl_ssm_workspace_bytes), ("saved", rsu.dl_ssm_saved_bytes),
        ("backward workspace", rsu.dl_ssm_backward_workspace_bytes)))
    dy, dend = dy.cuda(), dend.cuda()
    assert rsu.dl_ssm_scan(d, v["initial"], o["end"], o["y"], saved, ws) == 0
    assert rsu.dl_ssm_scan_backward(d, saved, dy, dend, o["dx"], o["ddt"], o["dz"], o["dB"], o["dC"], o["dA"], o["dD"],
                                    o["ddt_bias"], o["dinitial"], ws2) == 0
    g.whole()
    return o


CONV = [(16, 4, "f32"), (13, 3, "bf16"), (40, 2, "bf16")]          # channels, taps
SSM = [(16, 16, 1, "f32"), (36, 20, 2, "bf16"), (24, 64, 1, "bf16")]  # channels, states, groups


def bad(T):
    sets = [[0, 5 * T // 6, T // 3, T], [-5, T // 2, 3 * T // 2, T], [T, 2 * T // 3, T // 3, 0], [0, 2 ** 31 - 1, T // 6, T],
            [-2 ** 31, 5, 5, 7 * T // 6], [T] * 4, [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, -2 ** 31], [-1] * 4]
    g = torch.Generator().manual_seed(T)
    for n in (2, 8, 40):  # anywhere, most of them out of order
        sets.append(torch.randint(-T // 4, T + T // 4, (n,), generator=g).tolist())
    return sets


@needs_gpu
@pytest.mark.parametrize("T", [7, 60, 2400])
@pytest.mark.parametrize("shape", CONV, ids=str)
def test_conv_bad_offsets(shape, T):
    C, W, dtype = shape
    for cu in bad(T):
        x, _, dy, _ = conv_inputs([T], C, W, dtype)
        n = len(cu) - 1
        x["initial"] = torch.ones(n, W - 1, C, dtype=DT[dtype])
        conv_passes(x, cu, dy, torch.ones(n, W - 1, C, dtype=DT[dtype]))


@needs_gpu
@pytest.mark.parametrize("T", [7, 60, 2400])  # the last in segments, both ways
@pytest.mark.parametrize("shape", SSM, ids=str)
def test_scan_bad_offsets(shape, T):
    C, S, G, dtype = shape
    for cu in bad(T):
        x, _, dy, _ = ssm_inputs([T], C, S, G, dtype)
        n = len(cu) - 1
        x["initial"] = torch.ones(n, C, S)
        ssm_passes(x, cu, dy, torch.ones(n, C, S))


SETS = [([5], 3, 0), ([0, 33, 0, 20], 0, 9), ([1, 70], 40, 30), ([900, 0, 700], 17, 100)]  # lengths, rows ahead and behind


@needs_gpu
@pytest.mark.parametrize("lens,first,tail", SETS, ids=str)
@pytest.mark.parametrize("shape", CONV, ids=str)
def test_conv_between_guards(shape, lens, first, tail):
    C, W, dtype = shape
    x, cu, dy, dend = conv_inputs(lens, C, W, dtype, first=first, tail=tail)
    got, want = conv_passes(x, cu, dy, dend), conv_run(x, cu, dy, dend)
    assert set(got) == set(want)
    for n in want:
        assert torch.equal(got[n], want[n]), n


@needs_gpu
@pytest.mark.parametrize("lens,first,tail", SETS, ids=str)
@pytest.mark.parametrize("shape", SSM, ids=str)
def test_scan_between_guards(shape, lens, first, tail):
    C, S, G, dtype = shape
    x, cu, dy, dend = ssm_inputs(lens, C, S, G, dtype, first=first, tail=tail)
    got, want = ssm_passes(x, cu, dy, dend), ssm_run(x, cu, dy, dend)
    assert set(got) == set(want)
    for n in want:
        assert torch.equal(got[n], want[n].reshape(got[n].shape)), n
