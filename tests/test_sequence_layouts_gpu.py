"""The sequence operators on tensors laid out as other code leaves them: the
results are those of contiguous copies, to the bit."""
import pytest
import torch

from test_scan_gpu import OPS, inputs

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
NAMES = ("q", "k", "v", "beta", "log_decay", "u", "initial_state")


def run(op, x):
    import recurrent_state_update_amd as rsu
    return rsu.scan(op, *(x[n] for n in NAMES))


def off_by_one(t):
    """The values of t in a contiguous view, one element behind a boundary."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    view = flat[1:].view(t.shape)
    view.copy_(t.detach())
    assert view.is_contiguous() and view.data_ptr() % 16 == t.element_size()
    return view


@needs_gpu
@pytest.mark.parametrize("op", OPS)
def test_states_off_the_boundary(op):
    """An initial state cut from a flat cache, and an end state's gradient as
    torch.cat's backward pass gives it: a narrow view."""
    x = {n: None if t is None else t.cuda() for n, t in inputs(op, [70], 2, 16, 32, torch.float32, seed=1)[0].items()}
    grads = []
    for view in (False, True):
        leaves = {n: None if t is None else t.clone().requires_grad_() for n, t in x.items()}
        if view:
            leaves["initial_state"] = off_by_one(x["initial_state"]).requires_grad_()
        o, end = run(op, leaves)
        w = torch.linspace(-1, 1, 1 + end.numel(), device="cuda")
        parts = [o.sum().view(1), end.flatten()]
        loss = (torch.cat(parts) * w).sum() if view else (parts[0] * w[:1]).sum() + (parts[1] * w[1:]).sum()
        loss.backward()
        grads.append([t.grad for t in leaves.values() if t is not None])
    for a, b in zip(*grads):
        assert torch.equal(a, b)
    with torch.no_grad():
        want = run(op, x)
        got = run(op, {**x, "initial_state": off_by_one(x["initial_state"])})
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@needs_gpu
@pytest.mark.parametrize("op", OPS)
def test_rows_far_apart(op):
    """One batch entry of [T,B,W] tensors: rows further apart than the library
    takes them."""
    T, H, dk, dv, W = 6, 2, 16, 32, 1 << 22
    x = {n: None if t is None else t.cuda() for n, t in inputs(op, [T], H, dk, dv, torch.bfloat16, seed=2)[0].items()}
    wide = torch.zeros(T, 2, W, dtype=torch.bfloat16, device="cuda")
    y, at = dict(x), 0
    for n in "qkv":
        d = x[n].shape[-1]
        y[n] = wide[:, 1, at:at + H * d].unflatten(1, (H, d))
        y[n].copy_(x[n])
        at += H * d
    assert all(torch.equal(a, b) for a, b in zip(run(op, y), run(op, x)))


@needs_gpu
def test_gate_rows_far_apart():
    import recurrent_state_update_amd as rsu
    T, H, d, W = 6, 2, 16, 1 << 22
    g = torch.Generator().manual_seed(3)
    o, gate = (torch.randn(T, H, d, generator=g).bfloat16().cuda() for _ in range(2))
    wide = torch.zeros(T, 2, W, dtype=torch.bfloat16, device="cuda")
    far = wide[:, 1, :H * d].unflatten(1, (H, d))
    far.copy_(gate)
    assert torch.equal(rsu.gated_norm(o, far), rsu.gated_norm(o, gate))
