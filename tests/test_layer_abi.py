"""Host-side checks of the state space layer's operators (no GPU needed): bad
arguments are reported by the documented status before any HIP call, sizes of
buffers, and the torch entry points' refusals.  No call here reaches a kernel
launch: addresses are fake and every call is invalid, or returns before launching."""
import pytest
import torch
import torch.autograd.forward_ad as fwd
from torch.fx.experimental.proxy_tensor import make_fx

import recurrent_state_update_amd as rsu

OK, INVALID, SHAPE, ALIGN = range(4)
F32, BF16 = 0, 1
A = [0x7f0000000000 + 0x10000000 * i for i in range(32)]  # aligned, far apart, never dereferenced


def conv(dt=BF16, T=128, N=2, C=96, W=4, silu=1, xs=0, cu=A[0], x=A[1], w=A[2], b=A[3]):
    return rsu.dl_conv_desc(dt, T, N, C, W, silu, xs, cu, x, w, b)


def conv_forward(d, initial=A[4], final=A[5], y=A[6]):
    return rsu.dl_short_conv(d, initial, final, y, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), INVALID), (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(C=0), INVALID), (dict(W=1), SHAPE),
    (dict(W=5), SHAPE), (dict(C=1 << 21), SHAPE), (dict(T=(1 << 30) + 1), SHAPE), (dict(T=1 << 25, C=1024), SHAPE),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(xs=95), INVALID), (dict(xs=(1 << 22) + 1), SHAPE),
    (dict(cu=None, T=127), INVALID), (dict(x=A[1] + 1), ALIGN), (dict(w=A[2] + 2), ALIGN), (dict(b=A[3] + 1), ALIGN),
    (dict(cu=A[0] + 2), ALIGN)])
def test_conv_refuses_inputs(kw, status):
    assert conv_forward(conv(**kw)) == status
    assert rsu.dl_short_conv_backward(conv(**kw), A[4], A[5], A[6], A[7], A[8], A[9], A[10], A[11], stream=0) == status
    if not {"cu", "N"} & set(kw):
        assert rsu.dl_short_conv_step(conv(**kw), A[4], None, 1 << 20, A[6], stream=0) == status


def test_conv_refuses_outputs():
    d = conv()
    assert conv_forward(d, y=None) == INVALID and conv_forward(d, y=A[6] + 1) == ALIGN
    assert conv_forward(d, y=A[1]) == INVALID and conv_forward(d, y=A[1] + 128 * 96 * 2 - 2) == INVALID
    assert conv_forward(d, initial=A[5]) == INVALID and conv_forward(d, final=A[2]) == INVALID
    assert conv_forward(conv(xs=1000), y=A[1] + 2 * 1000 * 100) == INVALID  # inside x's strided span
    names = ["initial", "dy", "d_final", "dx", "dw", "db", "d0", "ws"]
    good = dict(zip(names, A[4:12]))

    def back(**kw):
        x = {**good, **kw}
        return rsu.dl_short_conv_backward(d, *(x[n] for n in names), stream=0)
    assert back(dx=None) == INVALID and back(ws=None) == INVALID
    assert back(ws=good["ws"] + 4) == ALIGN and back(dw=good["dw"] + 2) == ALIGN and back(d0=good["d0"] + 1) == ALIGN
    assert back(dx=A[1]) == INVALID and back(dx=good["dy"]) == INVALID and back(d0=good["d_final"]) == INVALID
    assert back(db=good["dw"]) == INVALID and back(ws=good["dx"]) == INVALID
    assert rsu.dl_short_conv_workspace_bytes(d) >= 96 * 5 * 4 and rsu.dl_short_conv_workspace_bytes(conv(W=5)) == 0

    def step(T=128, state=A[4], rows=A[5], n=200, y=A[6]):
        return rsu.dl_short_conv_step(conv(T=T), state, rows, n, y, stream=0)
    assert step(T=0) == OK and step(y=None) == INVALID and step(state=None) == INVALID and step(n=0) == INVALID
    assert step(rows=None, n=127) == INVALID  # fewer rows than tokens
    assert step(state=A[4] + 1) == ALIGN and step(rows=A[5] + 2) == ALIGN
    assert step(state=A[1]) == INVALID and step(y=A[4] + 2) == INVALID and step(rows=A[4]) == INVALID


def ssm(dt=BF16, T=128, N=2, C=96, S=16, G=2, soft=1, xs=0, dts=0, zs=0, bs=0, cs=0, cu=A[0], x=A[1], delta=A[2], z=A[3],
        b=A[4], c=A[5], a=A[6], d=A[7], bias=A[8]):
    return rsu.dl_ssm_desc(dt, T, N, C, S, G, soft, xs, dts, zs, bs, cs, cu, x, delta, z, b, c, a, d, bias)


def scan(d, initial=A[9], final=A[10], y=A[11], saved=None, ws=A[12]):
    return rsu.dl_ssm_scan(d, initial, final, y, saved, ws, stream=0)


BACK = ["saved", "dy", "d_final", "dx", "ddt", "dz", "db", "dc", "da", "dd", "dbias", "d0", "ws"]
GOOD = dict(zip(BACK, A[13:26]))


def back(d, **kw):
    x = {**GOOD, **kw}
    return rsu.dl_ssm_scan_backward(d, *(x[n] for n in BACK), stream=0)


SIZES = [dict(dt=2), dict(T=-1), dict(N=0), dict(C=0), dict(S=0), dict(G=0), dict(G=5), dict(S=65), dict(C=1 << 21),
         dict(N=1 << 20, C=1024, G=1), dict(T=1 << 29, C=16, G=1, S=64), dict(T=(1 << 30) + 1)]


@pytest.mark.parametrize("kw", SIZES, ids=str)
def test_ssm_refuses_sizes(kw):
    d = ssm(**kw)
    assert rsu.dl_ssm_workspace_bytes(d) == rsu.dl_ssm_saved_bytes(d) == rsu.dl_ssm_backward_workspace_bytes(d) == 0
    assert scan(d) in (INVALID, SHAPE) and back(d) in (INVALID, SHAPE)
    assert rsu.dl_ssm_step(d, A[9], None, 1 << 20, A[11], stream=0) in (INVALID, SHAPE)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(delta=None), INVALID), (dict(b=None), INVALID), (dict(c=None), INVALID),
    (dict(a=None), INVALID), (dict(xs=95), INVALID), (dict(zs=95), INVALID), (dict(bs=31), INVALID), (dict(cs=31), INVALID),
    (dict(dts=(1 << 22) + 1), SHAPE), (dict(cs=(1 << 22) + 1), SHAPE), (dict(cu=None, T=127), INVALID),
    (dict(x=A[1] + 1), ALIGN), (dict(z=A[3] + 1), ALIGN), (dict(a=A[6] + 2), ALIGN), (dict(bias=A[8] + 1), ALIGN),
    (dict(cu=A[0] + 2), ALIGN)])
def test_ssm_refuses_inputs(kw, status):
    assert scan(ssm(**kw)) == status and back(ssm(**kw)) == status
    if "cu" not in kw:
        assert rsu.dl_ssm_step(ssm(**kw), A[9], None, 200, A[11], stream=0) == status


def test_ssm_refuses_outputs():
    d = ssm()
    assert scan(d, y=None) == INVALID and scan(d, ws=None) == INVALID
    assert scan(d, ws=A[12] + 16) == ALIGN and scan(d, saved=A[13] + 16) == ALIGN and scan(d, final=A[10] + 2) == ALIGN
    assert scan(d, initial=A[10]) == INVALID and scan(d, y=A[3]) == INVALID and scan(d, ws=A[0]) == INVALID
    assert scan(d, saved=A[11]) == INVALID and scan(ssm(zs=1000), y=A[3] + 2 * 1000 * 100) == INVALID
    for n in ("saved", "dy", "dx", "ddt", "dz", "db", "dc", "da", "ws"):
        assert back(d, **{n: None}) == INVALID, n
    # gradients of what is not there
    assert back(ssm(z=None)) == INVALID and back(ssm(d=None)) == INVALID and back(ssm(bias=None)) == INVALID
    for n in ("saved", "ws", "da", "dd", "d0", "d_final"):
        assert back(d, **{n: GOOD[n] + 2}) == ALIGN, n
    assert back(d, dx=A[1]) == INVALID and back(d, dz=GOOD["dx"]) == INVALID and back(d, dc=GOOD["dy"]) == INVALID
    assert back(d, d0=GOOD["d_final"]) == INVALID and back(d, ws=GOOD["saved"]) == INVALID

    def step(T=128, state=A[9], rows=A[10], n=200, y=A[11]):
        return rsu.dl_ssm_step(ssm(T=T), state, rows, n, y, stream=0)
    assert step(T=0) == OK and step(y=None) == INVALID and step(state=None) == INVALID and step(n=0) == INVALID
    assert step(rows=None, n=127) == INVALID and step(state=A[9] + 2) == ALIGN and step(rows=A[10] + 1) == ALIGN
    assert step(state=A[6]) == INVALID and step(y=A[9]) == INVALID and step(rows=A[9]) == INVALID
    assert step(T=1 << 23, n=1 << 23) == SHAPE


def test_ssm_sizes():
    d = ssm()
    states = (128 // 16 + 2) * 96 * 16 * 4
    assert rsu.dl_ssm_saved_bytes(ssm(z=None)) == (states + 255) // 256 * 256
    assert rsu.dl_ssm_saved_bytes(d) == (states + 255) // 256 * 256 + 128 * 96 * 4
    for n in (rsu.dl_ssm_workspace_bytes(d), rsu.dl_ssm_backward_workspace_bytes(d)):
        assert n > 0 and n % 256 == 0
    # large shapes do not wrap around
    assert rsu.dl_ssm_saved_bytes(ssm(T=1 << 22, N=1, C=1 << 14, S=64, G=1)) > (1 << 18) * (1 << 14) * 64 * 4


def test_norm_refuses():
    def call(rows=4, D=256, t=BF16, x=A[0], y=A[1], s=A[2], w=A[3], eps=1e-6, xo=A[4], group=0, h=A[5], hs=A[6]):
        return rsu.dl_residual_norm_quant(rows, D, t, x, y, s, w, eps, xo, group, h, hs, stream=0)
    assert call(D=0) == SHAPE and call(D=16385) == SHAPE and call(rows=-1) == INVALID and call(t=2) == INVALID
    assert call(group=64) == SHAPE and call(group=128, D=200) == SHAPE
    assert call(eps=0.0) == INVALID and call(eps=float("nan")) == INVALID
    for n in ("x", "h", "hs", "xo", "y"):
        assert call(**{n: None}) == INVALID, n  # (x_out and scale go with y)
    assert call(x=A[0] + 2) == ALIGN and call(hs=A[6] + 1) == ALIGN and call(y=A[1] + 1) == ALIGN
    for n in ("x", "y", "xo", "h"):
        assert call(group=128, **{n: dict(x=A[0], y=A[1], xo=A[4], h=A[5])[n] + 8}) == ALIGN, n
    assert call(h=A[0]) == INVALID and call(hs=A[5]) == INVALID and call(xo=A[0] + 4) == INVALID and call(h=A[1]) == INVALID
    assert call(rows=0, x=None, h=None, hs=None) == OK


# ------------------------------------------------------- torch entry points --

T, C, N = 5, 8, 4


def calls():
    """Each operator as a function of its tensors, and those."""
    x, w, b = torch.randn(T, C), torch.randn(C, 4), torch.randn(C)
    bc, a = torch.randn(T, N), -torch.rand(C, N)
    return {
        "short_conv": (lambda *t: rsu.short_conv(*t)[0], [x, w, b, torch.randn(1, 3, C)]),
        "short_conv_step": (lambda *t: rsu.short_conv_step(*t), [x, torch.randn(T, 3, C), w, b]),
        "ssm_scan": (lambda *t: rsu.ssm_scan(*t)[0], [x, x + 1, a, bc, bc + 1, b, x + 2, b + 1]),
        "ssm_step": (lambda *t: rsu.ssm_step(*t), [x, x + 1, torch.randn(T, C, N), a, bc, bc + 1, b, x + 2, b + 1]),
        "residual_norm_fp8": (lambda *t: rsu.residual_norm_fp8(*t)[1], [x, x + 1, b, b + 1]),
    }


NAMES = list(calls())


@pytest.mark.parametrize("name", NAMES)
def test_refuses_cpu_tensors(name):
    f, args = calls()[name]
    with pytest.raises(ValueError, match="x: want a GPU tensor"):
        f(*args)
    with pytest.raises(ValueError):
        f(None, *args[1:])


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("no_grad", [False, True])
def test_refuses_forward_mode(name, no_grad):
    f, args = calls()[name]
    with torch.set_grad_enabled(not no_grad):
        for i in range(len(args)):
            with fwd.dual_level():
                duals = [fwd.make_dual(a, torch.ones_like(a)) if j == i else a for j, a in enumerate(args)]
                with pytest.raises(NotImplementedError, match="forward-mode"):
                    f(*duals)


@pytest.mark.parametrize("name", NAMES)
def test_refuses_tracing(name):
    f, args = calls()[name]
    with pytest.raises(NotImplementedError, match="traced"):
        torch.jit.trace(f, tuple(args), check_trace=False)
    for mode in ("real", "fake"):
        with pytest.raises(NotImplementedError, match="traced"):
            make_fx(f, tracing_mode=mode)(*args)


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on a GPU: the checks go by what tensors say,
    and every call here is refused before anything is read."""
    device = property(lambda self: torch.device("cuda:0"))
    is_cuda = True


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def good(name):
    x, w, b, bc, a = gpu(T, C), gpu(C, 4), gpu(C), gpu(T, N), gpu(C, N)
    return {"short_conv": dict(x=x, weight=w, bias=b, initial_state=gpu(1, 3, C)),
            "short_conv_step": dict(x=x, state=gpu(T, 3, C), weight=w, bias=b),
            "ssm_scan": dict(x=x, dt=x, A=a, B=bc, C=bc, D=b, z=x, dt_bias=b, initial_state=gpu(1, C, N)),
            "ssm_step": dict(x=x, dt=x, state=gpu(T, C, N), A=a, B=bc, C=bc, D=b, z=x, dt_bias=b),
            "residual_norm_fp8": dict(x=x, y=x, scale=b, weight=b)}[name]


BF = torch.bfloat16
I32 = torch.int32


@pytest.mark.parametrize("name,kw,what", [
    ("short_conv", dict(x=gpu(C)), "want \\[T,C\\]"), ("short_conv", dict(x=gpu(T, C, dtype=torch.float16)), "dtype|float16"),
    ("short_conv", dict(weight=gpu(C, 5)), "2 to 4 taps"), ("short_conv", dict(weight=gpu(C + 1, 4)), "weight"),
    ("short_conv", dict(weight=gpu(C, 4, dtype=BF)), "weight"), ("short_conv", dict(bias=gpu(C + 1)), "bias"),
    ("short_conv", dict(initial_state=gpu(2, 3, C)), "initial_state"), ("short_conv", dict(x=gpu(T, 0)), "channel"),
    ("short_conv", dict(initial_state=gpu(1, 3, C, dtype=BF)), "initial_state"),
    ("short_conv", dict(cu_seqlens=gpu(3)), "cu_seqlens"), ("short_conv", dict(cu_seqlens=gpu(1, dtype=I32)), "two offsets"),
    ("short_conv", dict(x=gpu(2, T, C), cu_seqlens=gpu(3, dtype=I32)), "packed"),
    ("short_conv", dict(x=gpu(0, T, C), initial_state=None), "one sequence"),
    ("short_conv_step", dict(x=gpu(1, T, C)), "want \\[B,C\\]"), ("short_conv_step", dict(state=gpu(T, 2, C)), "state"),
    ("short_conv_step", dict(state=gpu(T - 1, 3, C)), "name their rows"), ("short_conv_step", dict(state=None), "state"),
    ("short_conv_step", dict(state=gpu(T, C, 3).mT), "contiguous"), ("short_conv_step", dict(rows=gpu(T)), "rows"),
    ("short_conv_step", dict(rows=gpu(T + 1, dtype=I32)), "rows"),
    ("ssm_scan", dict(dt=gpu(T, C, dtype=BF)), "dt"), ("ssm_scan", dict(A=gpu(C, 65)), "64 states"),
    ("ssm_scan", dict(A=gpu(C, N, dtype=BF)), "A"), ("ssm_scan", dict(B=gpu(T, N + 1)), "B"),
    ("ssm_scan", dict(C=gpu(T, 1, N)), "C"), ("ssm_scan", dict(B=gpu(T, 3, N), C=gpu(T, 3, N)), "3 groups"),
    ("ssm_scan", dict(B=gpu(T, 0, N), C=gpu(T, 0, N)), "0 groups"), ("ssm_scan", dict(D=gpu(C, dtype=BF)), "D"),
    ("ssm_scan", dict(z=gpu(T, C + 1)), "z"), ("ssm_scan", dict(dt_bias=gpu(1)), "dt_bias"),
    ("ssm_scan", dict(initial_state=gpu(1, N, C)), "initial_state"), ("ssm_scan", dict(B=None), "B"),
    ("ssm_step", dict(state=gpu(T, N, C)), "state"), ("ssm_step", dict(state=gpu(T, C, N, dtype=BF)), "state"),
    ("ssm_step", dict(rows=gpu(T, dtype=torch.int64)), "rows"),
    ("residual_norm_fp8", dict(x=gpu(T, C, dtype=BF)), "x: want fp32"), ("residual_norm_fp8", dict(y=None), "scale goes with y"),
    ("residual_norm_fp8", dict(group=64), "group"), ("residual_norm_fp8", dict(group=128), "group"),
    ("residual_norm_fp8", dict(y=gpu(T, C + 1)), "y"), ("residual_norm_fp8", dict(weight=gpu(C + 1)), "weight"),
    ("residual_norm_fp8", dict(x=gpu(T, 16385)), "16384 columns")], ids=str)
def test_refuses_arguments(name, kw, what):
    with pytest.raises((ValueError, KeyError, TypeError), match=what):
        getattr(rsu, name)(**{**good(name), **kw})


@pytest.mark.parametrize("name,wants", [("short_conv_step", "weight"), ("ssm_step", "A"), ("residual_norm_fp8", "weight"),
                                        ("short_conv_step", "state"), ("ssm_step", "x")])
def test_operators_without_gradient_refuse_to_want_one(name, wants):
    args = good(name)
    args[wants] = args[wants].detach().requires_grad_(True)
    with pytest.raises(NotImplementedError, match="no gradient"):
        getattr(rsu, name)(**args)
