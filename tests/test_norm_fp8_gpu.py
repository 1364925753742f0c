"""GPU checks of residual_norm_fp8 against its formulas in 64 bits.

Tolerances.  x' is one product and one sum: 2 roundings of 32 bits (2^-24).  The
scale takes the row's sum of squares (at most 128 in a row per lane, the rest a tree:
140), half of which the square root leaves, and six more operations, of the
exponent's one largest value: 80 roundings.  h * scale is off from rms(x') weight by
e4m3's rounding, at most 2^-4 of the value or, below its smallest normal value 2^-6,
half of its step 2^-9, and by 160 roundings."""
import pytest
import torch

from layer_ref import UNIT, norm_ref

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def inputs(lead, D, dtype, y=True, scaled=True, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g)
    return dict(x=2 * normal(*lead, D), y=normal(*lead, D).to(DT[dtype]) if y else None,
                scale=0.5 + 0.1 * normal(D) if scaled and y else None, weight=1 + 0.3 * normal(D) if scaled else None)


def gpu(v, group):
    import recurrent_state_update_amd as rsu
    return rsu.residual_norm_fp8(*(None if t is None else t.cuda() for t in v.values()), eps=EPS, group=group)


def verify(v, out, group):
    x, h, s = (t.cpu().double() for t in out)
    rx, rh = norm_ref(*v.values(), EPS)
    D = rx.shape[-1]
    size = rx.abs() if v["y"] is None else v["x"].abs() + (v["y"].double() * (1 if v["scale"] is None else v["scale"])).abs()
    assert ((x - rx).abs() <= 2 * UNIT * size).all()
    most = rh.unflatten(-1, (-1, group or D)).abs().amax(-1)
    # (where a sum nearly cancels, what it keeps of its terms' rounding counts)
    assert ((s.reshape(most.shape) * 448 - most).abs() <= 80 * UNIT * most + 4 * UNIT * most.max()).all()
    step = s.reshape(most.shape).unsqueeze(-1)
    h = h.unflatten(-1, (-1, group or D))
    rh = rh.unflatten(-1, (-1, group or D))
    assert torch.isfinite(h).all() and (h.abs().amax(-1) == 448).all()
    assert ((h * step - rh).abs() <= 2.0 ** -4 * rh.abs() + 2.0 ** -10 * step + 160 * UNIT * (rh.abs() + most[..., None])).all()


@needs_gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lead,D,group", [
    ((1,), 128, 128), ((1,), 1, None), ((7,), 48, None), ((5, 3), 512, 128), ((65,), 2048, None), ((65,), 2048, 128),
    ((33,), 1531, None), ((9,), 4096, 128), ((5,), 4224, 128), ((5,), 8192, None), ((3,), 16384, 128), ((3,), 16383, None),
    ((2500,), 384, 128), ((2500,), 130, None)])
@pytest.mark.parametrize("form", ["plain", "scaled", "first"])
def test_against_64_bits(lead, D, group, dtype, form):
    v = inputs(lead, D, dtype, y=form != "first", scaled=form != "plain", seed=D)
    x, h, s = gpu(v, group)
    assert h.dtype == torch.float8_e4m3fn and h.shape == v["x"].shape
    assert s.shape == ((*lead, D // 128) if group else lead)
    verify(v, (x, h, s), group)


@needs_gpu
@pytest.mark.parametrize("rows,D,group", [(8300, 130, None), (8300, 256, 128), (2200, 641, None), (2200, 640, 128),
                                          (1100, 2176, 128), (1100, 2051, None), (600, 4224, 128), (600, 8200, None)])
def test_many_rows(rows, D, group):
    """More rows than workgroups: each takes several."""
    v = inputs((rows,), D, "bf16", seed=D)
    verify(v, gpu(v, group), group)


@needs_gpu
def test_agrees_with_residual_norm():
    """x' is bit for bit residual_norm's, and h its h to e4m3's rounding."""
    import recurrent_state_update_amd as rsu
    v = inputs((40,), 1024, "f32")
    a = [t.cuda() for t in v.values()]
    x, h = rsu.residual_norm(*a, eps=EPS)
    x8, h8, s = rsu.residual_norm_fp8(*a, eps=EPS)
    assert torch.equal(x, x8)
    d = h8.float() * s[:, None] - h
    assert (d.abs() <= (2.0 ** -4 + 1e-5) * h.abs() + 2.0 ** -10 * s[:, None] * 1.001).all()


@needs_gpu
@pytest.mark.parametrize("group", [None, 128])
def test_off_a_boundary(group):
    """Tensors off a 16-byte boundary, and rows that are not contiguous: the same results."""
    import recurrent_state_update_amd as rsu
    v = inputs((10,), 256, "bf16")
    want = gpu(v, group)

    def off(t):
        return torch.cat([torch.zeros(1, dtype=t.dtype), t.reshape(-1)]).cuda()[1:].view(t.shape)
    got = rsu.residual_norm_fp8(*(off(t) for t in v.values()), eps=EPS, group=group)
    # whole rows take another path there, with other sums: the scale's last bits
    assert torch.equal(got[0], want[0])
    assert ((got[2] - want[2]).abs() <= 100 * UNIT * want[2]).all()
    verify(v, got, group)
    wide = torch.zeros(10, 600, device="cuda")
    wide[:, 100:356] = v["x"].cuda()
    got = rsu.residual_norm_fp8(wide[:, 100:356], *(t.cuda() for t in list(v.values())[1:]), eps=EPS, group=group)
    assert all(torch.equal(a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a,
                           b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b) for a, b in zip(got, want))


@needs_gpu
@pytest.mark.parametrize("group", [None, 128])
def test_extremes(group):
    """Rows of zeros, groups of zeros, tiny and huge rows, NaNs and infinities."""
    x = torch.zeros(8, 256)
    x[1, 3] = 1.0
    x[2] = 1e-25 * torch.randn(256, generator=torch.Generator().manual_seed(1))
    x[3] = 1e15 * torch.randn(256, generator=torch.Generator().manual_seed(2))
    x[4] = 1.0
    x[5, 7] = float("nan")
    x[6, 200] = float("inf")
    x[7] = -2.0
    _, h, s = gpu(dict(x=x, y=None, scale=None, weight=None), group)
    h, s = h.float().cpu(), s.cpu().reshape(8, -1)
    assert (h[0] == 0).all() and torch.isfinite(s[:5]).all() and (s[:5] > 0).all()
    assert h[1, 3] == 448 and (h[1].abs().sum() == 448)
    assert (h[4] == 448).all() and (h[7] == -448).all()
    want = norm_ref(x[2:4], None, None, None, EPS)[1]
    got = (h.unflatten(1, (s.shape[1], -1)) * s[..., None]).flatten(1)[2:4].double()
    assert ((got - want).abs() <= 2.0 ** -4 * 1.001 * want.abs() + 2.0 ** -10 * 1.001 * s[2:4].amax(1, keepdim=True)).all()
    assert torch.isnan(s[5]).all() and torch.isnan(h[5]).all()
    assert torch.isnan(s[6, -1])


@needs_gpu
def test_empty_streams_and_graph():
    import recurrent_state_update_amd as rsu
    x, h, s = rsu.residual_norm_fp8(torch.zeros(0, 128, device="cuda"))
    assert h.shape == (0, 128) and s.shape == (0,)
    v = [t.cuda() for t in inputs((70,), 512, "bf16").values()]
    want = rsu.residual_norm_fp8(*v)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = rsu.residual_norm_fp8(*v, stream=st)
    torch.cuda.synchronize()

    def same(a, b):
        return all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))
    assert same(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = rsu.residual_norm_fp8(*v)
    for _ in range(3):
        v[0].normal_()
        g.replay()
        torch.cuda.synchronize()
        assert same(out, rsu.residual_norm_fp8(*v))
