"""Plain 64-bit forms of a state space layer's operators for the tests, on the CPU:
token by token, from the formulas.  Each can also be run on absolute values
(`size`): what it then gives, the sum of the absolute values of all terms of an
output, is what the output's rounding errors are proportional to."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float64: 0.0}  # half a step, relative
UNIT = 2.0 ** -24


def within(got, want, size, units):
    """Whether |got - want| is at most `units` roundings of 32 bits of `size`, and
    one rounding to got's type.  Returns the worst share of that bound."""
    got_, want, size = got.detach().cpu().double(), want.detach(), size.detach()
    assert got_.shape == want.shape, (got_.shape, want.shape)
    assert torch.equal(torch.isfinite(got_), torch.isfinite(want)), "finite in other places"
    if not want.numel():
        return 0.0
    err = units * UNIT * size
    bound = err + HALF[got.dtype] * (want.abs() + err) + 1e-37  # (the last for what underflows)
    return float(((got_ - want).abs() / bound).nan_to_num(0.0).max())


def check(got, want, size, units):
    """`within` of every output by name."""
    bad = {}
    for n, w in want.items():
        share = within(got[n], w, size[n], units[n] if isinstance(units, dict) else units)
        print(f"{n}={share:.2g}", end=" ", flush=True)
        if not share <= 1.0:
            bad[n] = share
    print(flush=True)
    assert not bad, bad


def silu(s):
    return s * torch.sigmoid(s)


def conv_ref(x, weight, bias, initial, cu, act=True, dy=None, dend=None, size=False):
    """x [T,C], cu a list of offsets.  A dict of y, end and, with dy and dend, the
    gradients; all fp64."""
    T, C = x.shape
    W, N = weight.shape[1], len(cu) - 1
    x, weight = x.double(), weight.double()
    bias = torch.zeros(C, dtype=torch.float64) if bias is None else bias.double()
    old = torch.zeros(N, W - 1, C, dtype=torch.float64) if initial is None else initial.double()
    y, end, dx, d0 = torch.zeros(T, C, dtype=torch.float64), [], torch.zeros(T, C, dtype=torch.float64), []
    dw, db = torch.zeros_like(weight), torch.zeros_like(bias)
    a = torch.abs if size else (lambda v: v)
    for n in range(N):
        b, L = cu[n], cu[n + 1] - cu[n]
        seen = torch.cat([old[n], x[b:b + L]])
        s, sbar = bias.expand(L, C), bias.abs().expand(L, C)
        for j in range(W):
            s = s + seen[j:j + L] * weight[:, j]
            sbar = sbar + (seen[j:j + L] * weight[:, j]).abs()
        # silu is at most 1.1 times as steep as its argument, its slope's slope at most 0.5
        y[b:b + L] = (1.1 * sbar if act else sbar) if size else silu(s) if act else s
        end.append(a(seen[L:]))
        if dy is None:
            continue
        g = a(dy[b:b + L].double())
        sig = torch.sigmoid(s)
        if act:
            g = g * (1.1 + 0.5 * sbar) if size else g * sig * (1 + s * (1 - sig))
        dseen = torch.zeros_like(seen)
        dseen[L:] += a(dend[n].double())
        for j in range(W):
            dseen[j:j + L] += g * a(weight[:, j])
            dw[:, j] += (g * a(seen[j:j + L])).sum(0)
        db += g.sum(0)
        dx[b:b + L] = dseen[W - 1:]
        d0.append(dseen[:W - 1])
    out = dict(y=y, end=torch.stack(end))
    if dy is not None:
        out.update(dx=dx, dweight=dw, dbias=db, dinitial=torch.stack(d0))
    return out


def ssm_ref(x, dt, A, B, C, D, z, dt_bias, initial, cu, softplus=True, dy=None, dend=None, size=False):
    """x [T,ch], A [ch,N], B, C [T,G,N], cu a list of offsets.  As conv_ref."""
    T, ch = x.shape
    N, G, n_seq = A.shape[1], B.shape[1], len(cu) - 1
    a = torch.abs if size else (lambda v: v)
    x, dt, A, B, C = a(x.double()), dt.double(), A.double(), a(B.double()), a(C.double())
    D = torch.zeros(ch, dtype=torch.float64) if D is None else a(D.double())
    raw = dt if dt_bias is None else dt + dt_bias.double()
    delta = torch.nn.functional.softplus(raw, threshold=1e9) if softplus else raw
    slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    gate = torch.ones_like(x) if z is None else a(silu(z.double()))
    sig = None if z is None else torch.sigmoid(z.double())
    # silu' = sig + z sig (1 - sig): two terms, which cancel at z = -1.278; each is rounded, so
    # the size is |sig| + |z| sig (1 - sig), and not their sum's
    dgate = None if z is None else sig * (1 + a(z.double()) * (1 - sig))
    h0 = torch.zeros(n_seq, ch, N, dtype=torch.float64) if initial is None else a(initial.double())
    wide = lambda v: v.repeat_interleave(ch // G, 0)  # noqa: E731  [G,N] -> [ch,N]
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    y, end, before = zeros(T, ch), [], {}
    u = a(delta) * x
    for n in range(n_seq):
        h = h0[n]
        for t in range(cu[n], cu[n + 1]):
            before[t] = h
            h = torch.exp(delta[t, :, None] * A) * h + u[t, :, None] * wide(B[t])
            y[t] = (h * wide(C[t])).sum(1) + D * x[t]
        end.append(h)
    out = dict(y=y * gate, end=torch.stack(end))
    if dy is None:
        return out
    live = zeros(T, 1)
    for n in range(n_seq):
        live[cu[n]:cu[n + 1]] = 1
    dy = a(dy.double()) * live
    dz = None if z is None else dy * y * dgate
    dy = dy * gate
    dx, dd, dB, dC, dA, d0 = dy * D, zeros(T, ch), zeros(T, G, N), zeros(T, G, N), zeros(ch, N), []
    for n in range(n_seq):
        g = a(dend[n].double())
        for t in reversed(range(cu[n], cu[n + 1])):
            d, b = torch.exp(delta[t, :, None] * A), wide(B[t])
            h = d * before[t] + u[t, :, None] * b
            g = g + dy[t, :, None] * wide(C[t])
            dC[t] = (dy[t, :, None] * h).reshape(G, -1, N).sum(1)
            dB[t] = (u[t, :, None] * g).reshape(G, -1, N).sum(1)
            q, moved = (g * b).sum(1), d * g * before[t]
            dx[t] += q * a(delta[t])
            dd[t] = q * x[t] + torch.nan_to_num(moved * a(A), nan=0.0).sum(1)
            dA += a(delta[t, :, None]) * moved
            g = d * g
        d0.append(g)
    ddt = dd * slope * live
    out.update(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(dy * x).sum(0), ddt_bias=ddt.sum(0), dinitial=torch.stack(d0))
    if z is not None:
        out["dz"] = dz
    return out


def norm_ref(x, y, scale, weight, eps):
    """x' and rms(x') * weight."""
    x = x.double()
    if y is not None:
        x = x + (y.double() if scale is None else y.double() * scale.double())
    h = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x, h if weight is None else h * weight.double()


def offsets(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu
