"""The sequence operators' gradients where autograd does not keep what they
saved but makes it again: checkpoints run the forward pass a second time, and
offloaded tensors come back elsewhere and contiguous.  Same kernels, same
inputs: the gradients are the same to the bit."""
import pytest
import torch
import torch.utils.checkpoint

from recurrent_state_update_amd import gated_norm, residual_norm, scan

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")


def layer(op, x, w, beta, log_decay, u):
    """Slices of one projection through all three operators."""
    H, d = beta.shape[1], w.shape[1] // (4 * beta.shape[1])
    q, k, v, g = (x @ w).view(len(x), 4, H, d).unbind(1)
    o, end = scan(op, q * 0.3, k * 0.3, v, None if op == "rwkv6" else beta, log_decay, u)
    y = gated_norm(o, g, torch.ones(d, device="cuda"))
    x, h = residual_norm(x, y.flatten(1)[:, :x.shape[1]], torch.full((x.shape[1],), 0.5, device="cuda"))
    return x.square().mean() + h.tanh().mean() + end.square().mean()


@needs_gpu
@pytest.mark.parametrize("kept", ["checkpoint", "offload"])
@pytest.mark.parametrize("op", ["gdn", "kda", "rwkv6"])
def test_saved_elsewhere(op, kept):
    T, H, d = 150, 3, 32
    g = torch.Generator().manual_seed(5)
    normal = lambda *s: torch.randn(*s, generator=g)
    args = [normal(T, 48), normal(48, 4 * H * d) / 7, torch.sigmoid(normal(T, H)),
            -torch.rand(*((T, H) if op == "gdn" else (T, H, d)), generator=g)]
    args = [a.cuda().requires_grad_() for a in args] + [normal(H, d).cuda().requires_grad_() if op == "rwkv6" else None]
    leaves = [a for i, a in enumerate(args) if a is not None and not (op == "rwkv6" and i == 2)]

    def grads(how):
        if how == "checkpoint":
            loss = torch.utils.checkpoint.checkpoint(layer, op, *args, use_reentrant=False)
        elif how == "offload":
            with torch.autograd.graph.save_on_cpu():
                loss = layer(op, *args)
        else:
            loss = layer(op, *args)
        spoil = [torch.full((1 << 18,), float("nan"), device="cuda") for _ in range(64)]  # over what was freed
        del spoil
        return torch.autograd.grad(loss, leaves)

    want = grads(None)
    assert all(w.isfinite().all() and w.abs().max() > 0 for w in want)
    for got, w in zip(grads(kept), want):
        assert torch.equal(got, w)
