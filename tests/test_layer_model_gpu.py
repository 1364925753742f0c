"""A state space layer's operators together, as a model uses them, against 64 bits on
the CPU, and the short convolution in the synthetic decoder.

1. Serving: prompts packed through norm (8 bits), projection, convolution and scan,
   then tokens one at a time from the states that they leave, in a cache with more
   rows than requests.  The 64-bit model takes the norm's 8-bit values as they are
   (they are checked by themselves: a value next to a border may be rounded either
   way) and runs every request's tokens one after the other.
2. A training step: the gradients of every weight against autograd in 64 bits.
3. bench_decoder.py with a convolution: a prompt at once, and its tokens one by one.

Tolerances, in the 2-norm: fp32 throughout.  The operators are within 1e-6 of 64 bits
(fp32 cases of perf/more_operators.py) on sums like these, the projections' sums of up
to 64 columns add sqrt(64) 2^-24 = 5e-7 of their terms' norm each, and three follow each
other, with the next token's input: 1e-5.  Gradients take them twice, and sums over up to
60 tokens: 4e-5.  The decoder as its own tests: 2e-4 of the largest value."""
import numpy as np
import pytest
import torch

import synth
from layer_ref import conv_ref, norm_ref, offsets, ssm_ref

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
HID, C, N, R, W, EPS = 24, 40, 16, 8, 4, 1e-6


def far(a, b):
    return float((a.detach().cpu().double() - b.detach()).norm() / b.detach().norm())


def weights(g):
    def normal(*s, scale=1.0):
        return torch.randn(*s, generator=g) * scale
    return dict(gain=1 + 0.2 * normal(HID), W_in=normal(HID, 2 * C, scale=HID ** -0.5), conv=normal(C, W, scale=0.5),
                conv_bias=0.2 * normal(C), W_x=normal(C, R + 2 * N, scale=C ** -0.5), W_dt=normal(R, C, scale=R ** -0.5),
                dt_bias=normal(C) - 3, A=-torch.exp(normal(C, N)), D=normal(C), W_out=normal(C, HID, scale=C ** -0.5))


class Layer:
    """The layer on the GPU: sequences, or one token of each request."""

    def __init__(self, w):
        self.w = w

    def body(self, h, conv, scan):
        w = self.w
        x, z = (h @ w["W_in"]).split(C, dim=-1)
        x = conv(x)
        dt, B, Cs = (x @ w["W_x"]).split([R, N, N], dim=-1)
        return scan(x, dt @ w["W_dt"], B, Cs, z) @ w["W_out"]


def reference(w, h, cu, conv_state=None, ssm_state=None):
    """The same in 64 bits from the norm's output on, and the end states."""
    w = {n: t.double() for n, t in w.items()}
    x, z = (h @ w["W_in"]).split(C, dim=-1)
    c = conv_ref(x, w["conv"], w["conv_bias"], conv_state, cu)
    dt, B, Cs = (c["y"] @ w["W_x"]).split([R, N, N], dim=-1)
    s = ssm_ref(c["y"], dt @ w["W_dt"], w["A"], B[:, None], Cs[:, None], w["D"], z, w["dt_bias"], ssm_state, cu)
    return s["y"] @ w["W_out"], c["end"], s["end"]


@needs_gpu
def test_prompt_then_tokens():
    import recurrent_state_update_amd as rsu
    g = torch.Generator().manual_seed(7)
    w = weights(g)
    v = {n: t.cuda() for n, t in w.items()}
    layer = Layer(v)
    lens, rows, S, more = [17, 1, 33], [4, 0, 2], 6, 5
    cu = offsets(lens)
    T, n = cu[-1], len(lens)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    at = torch.tensor(rows, dtype=torch.int32, device="cuda")
    seen, state = torch.randn(S, W - 1, C, device="cuda"), torch.randn(S, C, N, device="cuda")
    untouched = [r for r in range(S) if r not in rows]
    before = seen[untouched].clone(), state[untouched].clone()
    x = torch.randn(T, HID, generator=g)

    def norm(x, y=None):
        x, h8, scale = rsu.residual_norm_fp8(x, y, weight=v["gain"], eps=EPS)
        return x, h8.float() * scale[:, None]

    with torch.no_grad():
        ends = {}

        def conv(t):
            y, ends["conv"] = rsu.short_conv(t, v["conv"], v["conv_bias"], cu_seqlens=off)
            return y

        def scan(x, dt, B, Cs, z):
            y, ends["ssm"] = rsu.ssm_scan(x, dt, v["A"], B, Cs, v["D"], z, v["dt_bias"], cu_seqlens=off)
            return y
        xs, h = norm(x.cuda())
        y = layer.body(h, conv, scan)
        seen[at.long()], state[at.long()] = ends["conv"], ends["ssm"]
        want, rconv, rssm = reference(w, h.cpu().double(), cu)
        assert far(y, want) < 1e-5 and far(ends["conv"], rconv) < 1e-5 and far(ends["ssm"], rssm) < 1e-5
        # token by token: the layer's output is the next input, through the residual
        last = torch.tensor(cu[1:]) - 1
        xt, yt = xs[last.cuda()], y[last.cuda()]
        for _ in range(more):
            xt, h = norm(xt, yt)
            yt = layer.body(h, lambda t: rsu.short_conv_step(t, seen, v["conv"], v["conv_bias"], rows=at),
                            lambda x, dt, B, Cs, z: rsu.ssm_step(x, dt, state, v["A"], B, Cs, v["D"], z, v["dt_bias"],
                                                                 rows=at))
            want, rconv, rssm = reference(w, h.cpu().double(), list(range(n + 1)), rconv, rssm)
            assert far(yt, want) < 1e-5
    assert far(seen[at.long()], rconv) < 1e-5 and far(state[at.long()], rssm) < 1e-5
    assert torch.equal(seen[untouched], before[0]) and torch.equal(state[untouched], before[1])


@needs_gpu
def test_training_step():
    import recurrent_state_update_amd as rsu
    g = torch.Generator().manual_seed(8)
    w, cu = weights(g), offsets([29, 3, 28])
    T = cu[-1]
    x, y0, dy = (torch.randn(T, HID, generator=g) for _ in range(3))
    v = {n: t.cuda().requires_grad_(True) for n, t in w.items()}
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    xn, h = rsu.residual_norm(x.cuda(), y0.cuda(), None, v["gain"], eps=EPS)
    y = Layer(v).body(h, lambda t: rsu.short_conv(t, v["conv"], v["conv_bias"], cu_seqlens=off)[0],
                      lambda x, dt, B, Cs, z: rsu.ssm_scan(x, dt, v["A"], B, Cs, v["D"], z, v["dt_bias"],
                                                           cu_seqlens=off)[0])
    got = torch.autograd.grad(((xn + y) * dy.cuda()).sum(), list(v.values()))
    r = {n: t.double().requires_grad_(True) for n, t in w.items()}
    _, h = norm_ref(x, y0, None, r["gain"], EPS)
    out, _, _ = reference(r, h, cu)
    want = torch.autograd.grad((out * dy.double()).sum(), list(r.values()))
    assert far(y, out) < 1e-5
    bad = {n: far(a, b) for n, a, b in zip(w, got, want)}
    print(bad)
    assert all(e < 4e-5 for e in bad.values()), bad


@needs_gpu
@pytest.mark.parametrize("path", ["deltalog", "eager"])
@pytest.mark.parametrize("fused", [False, True])
def test_decoder_with_convolution(path, fused):
    """A prompt of 9 tokens at once leaves what its tokens one by one leave, and the
    tokens behind it agree; captured steps go on from there."""
    from bench_decoder import SyntheticDecoder
    ds = synth.DecoderShape("gdn", 2, 3, 2, 32, 32, 4, 48, 64, gated=True, taps=4)
    X = torch.from_numpy(synth.decoder_prompt(ds, 9)).cuda()
    a = SyntheticDecoder(ds, path, torch.float32, fused=fused)
    b = SyntheticDecoder(ds, path, torch.float32, weights_from=a, fused=fused)
    out, x = a.prompt(X)
    for t in range(9):
        want, nxt = b.token(X[:, t].contiguous())
    assert float((out - want).abs().max() / want.abs().max()) < 2e-4
    for la, lb in zip(a.layers, b.layers):
        assert float((la["seen"] - lb["seen"]).abs().max() / lb["seen"].abs().max()) < 2e-4
    if path == "deltalog":  # a merge cycle begins where both stand alike
        for lay in b.layers:
            lay["st"].merge()
    nxt = nxt.clone()
    graph, outs = a.capture_cycle(x.contiguous())
    graph.replay()
    torch.cuda.synchronize()
    for m in range(ds.M):
        want, nxt = b.token(nxt)
        assert float((outs[m] - want).abs().max() / want.abs().max()) < 2e-4
    a.close()
    b.close()


@needs_gpu
def test_layers_without_convolution_are_as_before():
    """The weights drawn do not depend on the convolution's."""
    a = synth.decoder_layer(synth.DecoderShape("gdn", 1, 1, 1, 16, 16, 2, 8, 8, gated=True), 0)
    b = synth.decoder_layer(synth.DecoderShape("gdn", 1, 1, 1, 16, 16, 2, 8, 8, gated=True, taps=4), 0)
    assert all(np.array_equal(a[k], b[k]) for k in a if a[k] is not None) and "conv" not in a
