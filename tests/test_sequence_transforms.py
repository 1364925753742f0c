"""Transforms that would take a call of the library for no operation are
refused: forward-mode derivatives (they would be zero) and tracing (the traced
function would return memory that nothing has written).  Refused before the
device is looked at, so without a GPU."""
import pytest
import torch
import torch.autograd.forward_ad as fwd
from torch.fx.experimental.proxy_tensor import make_fx

import recurrent_state_update_amd as rsu
from recurrent_state_update_amd.sequence import _prefill

T, H, D = 4, 2, 16
DEVICES = ["cpu", pytest.param("cuda", marks=[
    pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")])]


def calls(device):
    """Each operator as a function of its tensors, and those."""
    q, beta, ld = torch.randn(T, H, D, device=device), torch.rand(T, H, device=device), -torch.rand(T, H, device=device)
    u, s, w = torch.rand(H, D, device=device), torch.randn(1, H, D, D, device=device), torch.rand(D, device=device)
    return {
        "gdn": (lambda q, k, v, beta, ld, s: rsu.scan("gdn", q, k, v, beta, ld, initial_state=s)[0], [q, q + 1, q + 2, beta, ld, s]),
        "rwkv6": (lambda q, k, v, ld, u: rsu.scan("rwkv6", q, k, v, None, ld, u)[0], [q, q + 1, q + 2, -q.abs(), u]),
        "prefill": (lambda *a: _prefill(None, *a, None, None, None), [q, q + 1, q + 2, beta, ld]),
        "gated_norm": (lambda o, g, w: rsu.gated_norm(o, g, w), [q, q + 1, w]),
        "residual_norm": (lambda x, y, s, w: rsu.residual_norm(x, y, s, w)[1], [q, q + 1, w, w + 1]),
    }


NAMES = list(calls("cpu"))


@pytest.mark.parametrize("device", DEVICES)
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("no_grad", [False, True])
def test_forward_mode(name, device, no_grad):
    f, args = calls(device)[name]
    with torch.set_grad_enabled(not no_grad):
        for i, t in enumerate(args):
            with fwd.dual_level():
                duals = [fwd.make_dual(a, torch.ones_like(a)) if j == i else a for j, a in enumerate(args)]
                with pytest.raises(NotImplementedError, match="forward-mode"):
                    f(*duals)


@pytest.mark.parametrize("device", DEVICES)
@pytest.mark.parametrize("name", NAMES)
def test_tracing(name, device):
    f, args = calls(device)[name]
    with pytest.raises(NotImplementedError, match="traced"):
        torch.jit.trace(f, tuple(args), check_trace=False)
    for mode in ("real", "fake"):
        with pytest.raises(NotImplementedError, match="traced"):
            make_fx(f, tracing_mode=mode)(*args)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
@pytest.mark.parametrize("name", [n for n in NAMES if n != "prefill"])
def test_calls_beside_a_transform(name):
    """Tensors without tangents within a dual level, and calls after a refused
    trace, are as ever."""
    f, args = calls("cuda")[name]

    want = f(*args)
    with pytest.raises(NotImplementedError):
        torch.jit.trace(f, tuple(args), check_trace=False)
    with fwd.dual_level():
        fwd.make_dual(torch.ones(1), torch.ones(1))
        assert torch.equal(f(*args), want)
    assert torch.equal(f(*args), want)
