"""GPU checks of gated_norm and residual_norm against their formulas in 64 bits
and autograd's gradients of them.

Tolerances (2-norm, relative): a row's outputs take one sum of up to D <= 16384
squares in fp32, at most 128 of them in a row per lane (the rest is a tree), so
about sqrt(128) 2^-24 = 7e-7, and a handful of further roundings (the
exponential and the square root are good to 2 units): FP32 = 2e-6.  The column
sums over rows run to a few hundred terms per thread: the same.  bf16 outputs
add their rounding, at most 2^-8 of each value."""
import pytest
import torch

from sequence_ref import f64, far, gated_norm_ref, residual_norm_ref

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
FP32 = 2e-6
BF16 = 2.0 ** -8
EPS = 1e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def check(got, want, types):
    errs = {n: far(got[n], want[n]) for n in want}
    print(" ".join(f"{n}={e:.1e}" for n, e in errs.items()), flush=True)
    bad = {n: e for n, e in errs.items() if not e <= FP32 + (BF16 if types.get(n) == torch.bfloat16 else 0.0)}
    assert not bad, bad


def normal(g, *s):
    return torch.randn(*s, generator=g)


@needs_gpu
@pytest.mark.parametrize("ot", ["f32", "bf16"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("lead,H,d", [((1,), 1, 16), ((7,), 3, 32), ((5, 13), 5, 64), ((300,), 2, 128), ((0,), 2, 16),
                                      ((2100,), 9, 16)])
@pytest.mark.parametrize("weighted", [True, False])
def test_gated_norm(ot, t, lead, H, d, weighted):
    import recurrent_state_update_amd as rsu
    g = torch.Generator().manual_seed(d + H)
    x = dict(o=normal(g, *lead, H, d).to(DT[ot]), gate=(2 * normal(g, *lead, H, d)).to(DT[t]),
             weight=1 + 0.3 * normal(g, d) if weighted else None)
    dy = normal(g, *lead, H, d).to(DT[t])
    a = {n: None if v is None else v.cuda().requires_grad_(True) for n, v in x.items()}
    b = {n: f64(v) for n, v in x.items()}
    y, ref = rsu.gated_norm(a["o"], a["gate"], a["weight"], eps=EPS), gated_norm_ref(*b.values(), EPS)
    assert y.dtype == DT[t]
    wrt = [n for n in x if x[n] is not None]
    got = torch.autograd.grad(y, [a[n] for n in wrt], dy.cuda())
    want = torch.autograd.grad(ref, [b[n] for n in wrt], f64(dy, False))
    check({"y": y, **dict(zip(wrt, got))}, {"y": ref, **dict(zip(wrt, want))},
          {"y": DT[t], "o": DT[ot], "gate": DT[t]})


@needs_gpu
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_gated_norm_slices(shift):
    """The gate as a slice of a projection at any alignment, and o off a
    16-byte boundary: the same results."""
    import recurrent_state_update_amd as rsu
    g = torch.Generator().manual_seed(3)
    rows, H, d = 37, 3, 32
    o, gate = normal(g, rows, H, d), normal(g, rows, H, d).bfloat16()
    p = torch.zeros(rows, shift + H * d + 5, dtype=torch.bfloat16, device="cuda")
    view = p[:, shift:shift + H * d]
    view.copy_(gate.reshape(rows, -1))
    ob = torch.zeros(rows * H * d + shift, device="cuda")[shift:].view(rows, H, d)
    ob.copy_(o)
    a = rsu.gated_norm(o.cuda(), gate.cuda())
    b = rsu.gated_norm(ob, view.unflatten(1, (H, d)))
    assert torch.equal(a, b)


@needs_gpu
def test_gated_norm_extremes():
    """Zero rows, gates whose exponential overflows, and values whose squares
    are far from one."""
    import recurrent_state_update_amd as rsu
    o = torch.zeros(4, 1, 16)
    o[1], o[2], o[3] = 1.0, 1e12, 1e-12
    gate = torch.zeros(4, 1, 16)
    gate[..., :4], gate[..., 4:8], gate[..., 8:12] = -200.0, 200.0, -3.0
    a = [t.cuda().requires_grad_(True) for t in (o, gate)]
    b = [f64(t) for t in (o, gate)]
    y, ref = rsu.gated_norm(*a), gated_norm_ref(*b, None, EPS)
    dy = torch.ones_like(ref)
    got = torch.autograd.grad(y, a, dy.float().cuda())
    want = torch.autograd.grad(ref, b, dy)
    for i in range(4):
        for x, w in ((y, ref), (got[0], want[0]), (got[1], want[1])):
            if float(w[i].abs().max()) > 1e-10:  # smaller ones are what rounding leaves of an exact zero
                assert far(x[i], w[i]) <= FP32 or float((x[i].detach().cpu().double() - w[i]).abs().max()) <= 1e-6 * float(
                    w.abs().max()), i
        assert torch.isfinite(y[i]).all() and torch.isfinite(got[0][i]).all() and torch.isfinite(got[1][i]).all()


@needs_gpu
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("lead,D", [((1,), 1), ((3,), 7), ((2, 5), 64), ((70,), 511), ((9,), 512), ((33,), 513),
                                    ((64,), 2048), ((5,), 2050), ((6,), 4096), ((3,), 8000), ((2,), 16384), ((0,), 32),
                                    ((1500,), 40)])
@pytest.mark.parametrize("scaled,weighted", [(True, True), (False, False), (True, False)])
def test_residual_norm(t, lead, D, scaled, weighted):
    import recurrent_state_update_amd as rsu
    g = torch.Generator().manual_seed(D)
    x = dict(x=2 * normal(g, *lead, D), y=normal(g, *lead, D).to(DT[t]),
             scale=0.5 + 0.2 * normal(g, D) if scaled else None, weight=1 + 0.2 * normal(g, D) if weighted else None)
    dx, dh = normal(g, *lead, D), normal(g, *lead, D).to(DT[t])
    a = {n: None if v is None else v.cuda().requires_grad_(True) for n, v in x.items()}
    b = {n: f64(v) for n, v in x.items()}
    xo, h = rsu.residual_norm(a["x"], a["y"], a["scale"], a["weight"], eps=EPS)
    rx, rh = residual_norm_ref(*b.values(), EPS)
    assert h.dtype == DT[t] and xo.dtype == torch.float32
    wrt = [n for n in x if x[n] is not None]
    got = torch.autograd.grad([xo, h], [a[n] for n in wrt], [dx.cuda(), dh.cuda()])
    want = torch.autograd.grad([rx, rh], [b[n] for n in wrt], [f64(dx, False), f64(dh, False)])
    check({"x_out": xo, "h": h, **dict(zip(wrt, got))}, {"x_out": rx, "h": rh, **dict(zip(wrt, want))},
          {"h": DT[t], "y": DT[t]})


@needs_gpu
@pytest.mark.parametrize("D", [40, 41, 3000])
def test_norm_alone(D):
    import recurrent_state_update_amd as rsu
    g = torch.Generator().manual_seed(1)
    x, w, dh = normal(g, 19, D), 1 + 0.1 * normal(g, D), normal(g, 19, D).bfloat16()
    a, b = [t.cuda().requires_grad_(True) for t in (x, w)], [f64(t) for t in (x, w)]
    same, h = rsu.residual_norm(a[0], weight=a[1])
    assert same is a[0]
    _, ref = residual_norm_ref(b[0], None, None, b[1], EPS)
    got = torch.autograd.grad(h, a, dh.cuda())
    want = torch.autograd.grad(ref, b, f64(dh, False))
    check(dict(h=h, x=got[0], w=got[1]), dict(h=ref, x=want[0], w=want[1]), dict(h=torch.bfloat16))


@needs_gpu
def test_norms_graph_replays_and_one_cotangent():
    """Forward and backward of both captured, replayed on new inputs; and
    gradients from one cotangent alone."""
    import recurrent_state_update_amd as rsu
    g = torch.Generator().manual_seed(4)
    o, gate, w = (t.cuda().requires_grad_(True) for t in (normal(g, 50, 2, 16), normal(g, 50, 2, 16), normal(g, 16)))
    x, s = (t.cuda().requires_grad_(True) for t in (normal(g, 50, 32), normal(g, 32)))
    dx, dh = normal(g, 50, 32).cuda(), normal(g, 50, 32).cuda()

    def step():
        y = rsu.gated_norm(o, gate, w)
        xo, h = rsu.residual_norm(x, y.reshape(50, 32), s)
        return [y, xo, h, *torch.autograd.grad([xo, h], [o, gate, w, x, s], [dx, dh])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [t.detach() for t in step()]
    for i in range(3):
        with torch.no_grad():
            for t in (o, gate, w, x, s, dx, dh):
                t.copy_(normal(g, *t.shape))
        graph.replay()
        got = [t.clone() for t in outs]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
    xo, h = rsu.residual_norm(x, rsu.gated_norm(o, gate, w).reshape(50, 32), s)
    both = torch.autograd.grad([xo, h], [x, s], [dx, dh], retain_graph=True)
    parts = [torch.autograd.grad(t, [x, s], c, retain_graph=True) for t, c in ((xo, dx), (h, dh))]
    for i in range(2):
        assert far(parts[0][i] + parts[1][i], both[i].double().cpu()) <= 4 * FP32


@needs_gpu
def test_rows_past_an_int_are_refused():
    import recurrent_state_update_amd as rsu
    many = torch.zeros(1, device="cuda").expand(1 << 31, 1)
    with pytest.raises(ValueError):
        rsu.residual_norm(many)
    heads = torch.zeros(16, device="cuda").expand(1 << 31, 1, 16)
    with pytest.raises(ValueError):
        rsu.gated_norm(heads, heads)


@needs_gpu
@pytest.mark.parametrize("t,n", [("f32", 18_000_000), ("bf16", 24_000_000)])
@pytest.mark.parametrize("D", [128, 2000, 4096, 8000, 16384])
def test_residual_norm_beyond_the_caches(t, n, D):
    """More data than the last-level cache holds, against the same rows in two
    halves that it does hold: rows bit for bit, the column sums (up to 190 terms
    per thread, so some 4e-7 of rounding either way) within FP32 twice over."""
    import recurrent_state_update_amd as rsu
    rows = n // D // 2 * 2
    g = torch.Generator("cuda").manual_seed(D)
    x, y, dx, dh = (torch.randn(rows, D, generator=g, device="cuda") for _ in range(4))
    y, dh = y.to(DT[t]), dh.to(DT[t])
    s, w = (1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2))

    def run(a, b):
        leaves = [v.requires_grad_() for v in (x[a:b].clone(), y[a:b].clone(), s.clone(), w.clone())]
        out = rsu.residual_norm(*leaves)
        return [*out, *torch.autograd.grad(out, leaves, [dx[a:b], dh[a:b]])]
    whole, one, two = run(0, rows), run(0, rows // 2), run(rows // 2, rows)
    for a, b, c in list(zip(whole, one, two))[:4]:
        assert torch.equal(a[:rows // 2], b) and torch.equal(a[rows // 2:], c)
    for a, b, c in list(zip(whole, one, two))[4:]:
        assert far(a, (b.double() + c.double()).cpu()) <= 2 * FP32
