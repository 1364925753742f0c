"""Plain 64-bit forms of the sequence operators for the tests, on the CPU: the
recurrence token by token as the decode step defines it, and the norms from
their formulas.  Gradients come from autograd over these plain forms."""
import torch

FLOOR = -112.0  # log-decays below act as this


def scan_ref(op, q, k, v, beta, ld, u=None, initial=None, cu=None):
    """Packed [T,H,.] fp64 tensors; cu a list of offsets.  Returns o, states."""
    T, H, dk = q.shape
    dv = v.shape[-1]
    cu = [0, T] if cu is None else list(cu)
    rows, states = [None] * T, []
    for n in range(len(cu) - 1):
        X = torch.zeros(H, dk, dv, dtype=torch.float64) if initial is None else initial[n]
        for t in range(cu[n], cu[n + 1]):
            D = torch.clamp(ld[t], min=FLOOR).exp().reshape(H, -1, 1)
            if op == "rwkv6":
                s = (q[t] * u * k[t]).sum(-1, keepdim=True)
                rows[t] = (X * q[t].unsqueeze(-1)).sum(1) + s * v[t]
                X = D * X + k[t].unsqueeze(-1) * v[t].unsqueeze(1)
            else:
                X = D * X
                b = beta[t].unsqueeze(-1) * (v[t] - (X * k[t].unsqueeze(-1)).sum(1))
                X = X + k[t].unsqueeze(-1) * b.unsqueeze(1)
                rows[t] = (X * q[t].unsqueeze(-1)).sum(1)
        states.append(X)
    zero = torch.zeros(H, dv, dtype=torch.float64)
    o = torch.stack([zero if r is None else r for r in rows]) if T else torch.zeros(0, H, dv, dtype=torch.float64)
    return o, torch.stack(states)


def rms_ref(x, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def gated_norm_ref(o, gate, weight, eps):
    y = rms_ref(o, eps) * torch.nn.functional.silu(gate)
    return y if weight is None else y * weight


def residual_norm_ref(x, y, scale, weight, eps):
    if y is not None:
        x = x + (y if scale is None else y * scale)
    h = rms_ref(x, eps)
    return x, h if weight is None else h * weight


def f64(t, grad=True):
    """A tensor's values in 64 bits on the CPU, as a leaf."""
    return None if t is None else t.detach().double().cpu().requires_grad_(grad)


def far(x, ref):
    """|x - ref| / |ref| in the 2-norm; inf where x is not finite though ref is."""
    x, ref = x.detach().double().cpu(), ref.detach().double()
    assert x.shape == ref.shape, (x.shape, ref.shape)
    if not torch.isfinite(x).all():
        return float("inf")
    n = float(ref.norm())
    d = float((x - ref).norm())
    return d / n if n else (0.0 if d == 0.0 else float("inf"))
