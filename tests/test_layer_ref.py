"""The 64-bit forms that the state space layer's tests hold the kernels to:
their hand-written adjoints against autograd, and what they call the size of an
output against the output (no GPU needed)."""
import pytest
import torch

from layer_ref import conv_ref, offsets, silu, ssm_ref


def normal(g, *s):
    return torch.randn(*s, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_adjoint(act, W):
    g, C, cu = torch.Generator().manual_seed(W), 3, offsets([5, 0, 2, 1], 1)
    T, N = cu[-1] + 1, 4
    x = dict(x=normal(g, T, C), weight=normal(g, C, W), bias=normal(g, C), initial=normal(g, N, W - 1, C))
    dy, dend = normal(g, T, C), normal(g, N, W - 1, C)
    leaves = {n: t.clone().requires_grad_(True) for n, t in x.items()}
    loss = 0
    for n in range(N):
        seen = torch.cat([leaves["initial"][n], leaves["x"][cu[n]:cu[n + 1]]])
        L = cu[n + 1] - cu[n]
        s = torch.nn.functional.conv1d(seen.t()[None], leaves["weight"][:, None], leaves["bias"], groups=C)[0].t()[:L] \
            if L else seen[:0]
        loss = loss + ((silu(s) if act else s) * dy[cu[n]:cu[n + 1]]).sum() + (seen[L:] * dend[n]).sum()
    want = dict(zip(x, torch.autograd.grad(loss, list(leaves.values()))))
    got = conv_ref(*x.values(), cu, act, dy, dend)
    size = conv_ref(*x.values(), cu, act, dy, dend, size=True)
    for n in x:
        assert torch.allclose(got["d" + n], want[n], rtol=1e-12, atol=1e-12), n
    for n in got:
        assert (got[n].abs() <= size[n] * (1 + 1e-9) + 1e-12).all(), n


@pytest.mark.parametrize("gate,softplus", [(True, True), (False, False)])
def test_ssm_adjoint(gate, softplus):
    g, C, N, G, cu = torch.Generator().manual_seed(1), 4, 3, 2, offsets([5, 0, 3], 1)
    T = cu[-1] + 1
    x = dict(x=normal(g, T, C), dt=normal(g, T, C) * 0.5, A=-normal(g, C, N).exp(), B=normal(g, T, G, N),
             C=normal(g, T, G, N), D=normal(g, C), z=normal(g, T, C) if gate else None, dt_bias=normal(g, C),
             initial=normal(g, 3, C, N))
    dy, dend = normal(g, T, C), normal(g, 3, C, N)
    leaves = {n: None if t is None else t.clone().requires_grad_(True) for n, t in x.items()}
    l = leaves
    raw = l["dt"] + l["dt_bias"]
    delta = torch.nn.functional.softplus(raw) if softplus else raw
    loss = 0
    for n in range(3):
        h = l["initial"][n]
        for t in range(cu[n], cu[n + 1]):
            wide = [l[k][t].repeat_interleave(C // G, 0) for k in ("B", "C")]
            h = torch.exp(delta[t, :, None] * l["A"]) * h + (delta[t] * l["x"][t])[:, None] * wide[0]
            y = (h * wide[1]).sum(1) + l["D"] * l["x"][t]
            loss = loss + ((y * silu(l["z"][t]) if gate else y) * dy[t]).sum()
        loss = loss + (h * dend[n]).sum()
    wrt = [n for n in x if x[n] is not None]
    want = dict(zip(wrt, torch.autograd.grad(loss, [l[n] for n in wrt])))
    got = ssm_ref(*x.values(), cu, softplus, dy, dend)
    size = ssm_ref(*x.values(), cu, softplus, dy, dend, size=True)
    for n in wrt:
        assert torch.allclose(got["d" + n], want[n], rtol=1e-11, atol=1e-12), n
    for n in got:
        assert (got[n].abs() <= size[n] * (1 + 1e-9) + 1e-12).all(), n


def test_ssm_adjoint_against_differences():
    """One number of each input moved: the loss moves as the gradient says."""
    g, cu = torch.Generator().manual_seed(2), [0, 4]
    x = dict(x=normal(g, 4, 2), dt=normal(g, 4, 2), A=-normal(g, 2, 2).exp(), B=normal(g, 4, 1, 2), C=normal(g, 4, 1, 2),
             D=normal(g, 2), z=normal(g, 4, 2), dt_bias=normal(g, 2), initial=normal(g, 1, 2, 2))
    dy, dend = normal(g, 4, 2), normal(g, 1, 2, 2)

    def loss(v):
        o = ssm_ref(*v.values(), cu)
        return float((o["y"] * dy).sum() + (o["end"] * dend).sum())
    grads = ssm_ref(*x.values(), cu, True, dy, dend)
    for n in x:
        step = 1e-6
        up, down = ({**x, n: x[n].clone()} for _ in range(2))
        up[n].view(-1)[-1] += step
        down[n].view(-1)[-1] -= step
        slope = (loss(up) - loss(down)) / (2 * step)
        assert abs(slope - float(grads["d" + n].view(-1)[-1])) < 1e-7 * (1 + abs(slope)), n
