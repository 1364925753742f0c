"""Gradients of the short convolution's weight and bias over thousands of runs of tokens
where one token is 2^24 of the others: a sum over runs loses none of them, and is
rounded once (2^-24).  (Within its run, of at most 128 tokens and in 32 bits, it is
alone.)"""
import pytest
import torch

from sequence_ref import far

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
BIG = 2.0 ** 24


@needs_gpu
@pytest.mark.parametrize("T,C", [(20000, 4), (20001, 3), (9000, 20), (1 << 20, 16)])
@pytest.mark.parametrize("wants", ["weight", "bias", "both"])
def test_many_runs(T, C, wants):
    import recurrent_state_update_amd as rsu
    W, at = 3, T // 2
    x = torch.ones(T, C, device="cuda")
    dy = torch.ones(T, C, device="cuda")
    dy[at - 130:at + 131] = 0
    dy[at] = BIG
    live = T - 261 + BIG
    weight = torch.ones(C, W, device="cuda", requires_grad=wants != "bias")
    bias = torch.zeros(C, device="cuda", requires_grad=wants != "weight")
    y, _ = rsu.short_conv(x, weight, bias, silu=False)
    leaves = [t for t in (weight, bias) if t.requires_grad]
    grads = dict(zip([t.dim() for t in leaves], torch.autograd.grad(y, leaves, dy)))
    if 2 in grads:  # tap j misses the first W - 1 - j tokens
        want = torch.tensor([live - 2, live - 1, live], dtype=torch.float64).expand(C, W)
        assert far(grads[2], want) <= 2.0 ** -24
    if 1 in grads:
        assert far(grads[1], torch.full((C,), live, dtype=torch.float64)) <= 2.0 ** -24
