"""The sequence operators together, as a model uses them, against 64-bit models
on the CPU.

1. The synthetic decoder (bench_decoder.py) with a gated norm behind the step
   and its norms fused: a prompt as whole sequences, then decode steps from the
   states it leaves, against a model that runs every token through the
   oracle's eager step.
2. A training step of such a layer (projections, scan, gated norm, residual
   norm): loss and the gradients of every weight against autograd in 64 bits.

Tolerances: fp32 throughout, at the decoder tests' bar (2e-4 of the largest
value, which leaves two orders over the operators' own errors for the
projections' cancellation) and, for gradients in the 2-norm, 1e-4: the
operators' parts are within 1.1e-5 (10 times that for the log-decay), and the
projections' sums of up to 130 tokens x 48 columns add sqrt(6240) 2^-24 = 5e-6
of their terms' norm each."""
import numpy as np
import pytest
import torch

import synth
from gpu_harness import FP32_TOL, rel
from sequence_ref import f64, far, gated_norm_ref, residual_norm_ref, scan_ref

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")

EPS = 1e-6


def _rms(x):
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + EPS)


class CpuModel:
    """fp64 model of the gated decoder, token by token."""

    def __init__(self, ds, orc):
        self.ds, self.orc = ds, orc
        self.p = [{k: None if v is None else v.astype(np.float64) for k, v in synth.decoder_layer(ds, l).items()}
                  for l in range(ds.L)]

    def token(self, x):
        ds = self.ds
        B, H = ds.B, ds.H
        for p in self.p:
            h = _rms(x)
            q, k, v, zb, zd = np.split(h @ p["W_in"], np.cumsum(ds.proj_split)[:-1], axis=1)
            q, k, v = (t.reshape(B, H, -1) for t in (q, k, v))
            if ds.op != "rwkv6":
                q, k = (t / np.sqrt((t * t).sum(-1, keepdims=True) + ds.dk * EPS) for t in (q, k))
            beta = None if ds.op == "rwkv6" else 1 / (1 + np.exp(-zb))
            ld = -np.logaddexp(0, zd - 3.0)
            ld = ld.reshape(B, H) if ds.op == "gdn" else ld.reshape(B, H, ds.dk)
            o = self.orc.eager_step(ds.op, p["X0"], q, k, v, beta, ld, p["u"])
            if ds.gated:
                g = (h @ p["W_g"]).reshape(B, H, ds.dv)
                o = _rms(o) * p["g"] * g / (1 + np.exp(-g))
            x = x + o.reshape(B, -1) @ p["W_o"]
            g, u = np.split(_rms(x) @ p["W_gu"], 2, axis=1)
            x = x + (g / (1 + np.exp(-g)) * u) @ p["W_dn"]
        return x, _rms(x)


@needs_gpu
@pytest.mark.parametrize("op", ["gdn", "kda", "rwkv6"])
@pytest.mark.parametrize("path,gated,fused", [("deltalog", True, True), ("eager", True, False), ("deltalog", False, True)])
def test_prompt_then_decode(orc, op, path, gated, fused):
    from bench_decoder import SyntheticDecoder
    T = 70
    ds = synth.DecoderShape(op, L=2, B=2, H=2, dk=32, dv=64, M=4, hidden=64, ffn=96, seed=3, gated=gated)
    dec = SyntheticDecoder(ds, path, torch.float32, fused=fused)
    ref = CpuModel(ds, orc)
    X = synth.decoder_prompt(ds, T)
    for t in range(T):
        want = ref.token(X[:, t].astype(np.float64))
    got = dec.prompt(torch.from_numpy(X).cuda())
    worst = max(rel(a.cpu().numpy(), b) for a, b in zip(got, want))
    x, xr = got[1].contiguous(), want[1]
    for _ in range(ds.M + 2):
        out, x = dec.token(x)
        ref_out, xr = ref.token(xr)
        worst = max(worst, rel(out.cpu().numpy(), ref_out))
    print(f"[prompt {op} {path} gated={gated} fused={fused}] worst={worst:.2e}", flush=True)
    dec.close()
    assert worst < FP32_TOL


def layer(op, H, dk, dv, scan, gated_norm, residual_norm, x, w, cu, u, s0):
    """A recurrent layer over packed tokens x [T, D] and its loss: projections,
    the recurrence, the gated norm, the residual add and the next norm."""
    T = x.shape[0]
    _, h = residual_norm(x, None, None, w["norm"])
    q, k, v, zb, zd, gate = (h @ w["in"]).split([H * dk, H * dk, H * dv, H, H if op == "gdn" else H * dk, H * dv], dim=1)
    q, k, v = (t.reshape(T, H, -1) for t in (q, k, v))
    if op != "rwkv6":
        q, k = (t / (t * t).sum(-1, keepdim=True).sqrt() for t in (q, k))
    beta = None if op == "rwkv6" else torch.sigmoid(zb)
    ld = -torch.nn.functional.softplus(zd - 3)
    ld = ld if op == "gdn" else ld.reshape(T, H, dk)
    o, s = scan(op, q, k, v, beta, ld, u, s0, cu)
    y = gated_norm(o, gate.reshape(T, H, dv), w["gain"])
    x, h = residual_norm(x, y.reshape(T, H * dv) @ w["out"], w["scale"], w["norm2"])
    return (h * w["read"]).sum() + 0.1 * (x * x).sum() + 0.01 * (s * s).sum()


@needs_gpu
@pytest.mark.parametrize("op", ["gdn", "kda", "rwkv6"])
def test_training_step(op):
    import recurrent_state_update_amd as rsu
    H, dk, dv, D, lens = 2, 16, 32, 48, [70, 1, 59]
    g = torch.Generator().manual_seed(11)
    T = sum(lens)
    cu = [0, 70, 71, 130]

    def normal(*s, scale=1.0):
        return torch.randn(*s, generator=g) * scale
    width = 2 * H * dk + H * dv + H + (H if op == "gdn" else H * dk) + H * dv
    w = {"in": normal(D, width, scale=D ** -0.5), "out": normal(H * dv, D, scale=(H * dv) ** -0.5),
         "norm": 1 + normal(D, scale=0.1), "norm2": 1 + normal(D, scale=0.1), "gain": 1 + normal(dv, scale=0.1),
         "scale": 0.5 + normal(D, scale=0.1), "read": normal(T, D)}
    x, u, s0 = normal(T, D), normal(H, dk, scale=0.3) if op == "rwkv6" else None, normal(3, H, dk, dv, scale=0.2)
    leaves = {**w, "x": x, "s0": s0}
    if u is not None:
        leaves["u"] = u
    a = {n: t.cuda().requires_grad_(True) for n, t in leaves.items()}
    b = {n: f64(t) for n, t in leaves.items()}
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    loss = layer(op, H, dk, dv, lambda op, q, k, v, beta, ld, u, s0, cu: rsu.scan(op, q, k, v, beta, ld, u, s0, cu),
                 rsu.gated_norm, lambda x, y, s, n: rsu.residual_norm(x, y, s, n, dtype=torch.float32),
                 a["x"], a, cut, a.get("u"), a["s0"])
    ref = layer(op, H, dk, dv, scan_ref, lambda o, g, w: gated_norm_ref(o, g, w, EPS),
                lambda x, y, s, n: residual_norm_ref(x, y, s, n, EPS), b["x"], b, cu, b.get("u"), b["s0"])
    assert abs(float(loss) - float(ref)) <= 1e-5 * abs(float(ref))
    got = torch.autograd.grad(loss, list(a.values()))
    want = torch.autograd.grad(ref, list(b.values()))
    errs = {n: far(x, y) for n, x, y in zip(a, got, want)}
    print(f"[training step {op}] " + " ".join(f"{n}={e:.1e}" for n, e in errs.items()), flush=True)
    assert all(e <= 1e-4 for e in errs.values()), errs
