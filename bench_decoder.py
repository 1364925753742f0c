"""Synthetic multi-layer decode harness around the recurrent-state step.

    python bench_decoder.py [--op gdn] [--layers 8] [--B 64] [--H 32] [--d 128]
                            [--M 8] [--hidden 2048] [--ffn 4096] [--cycles 8]
                            [--gated] [--fused] [--prompt T]

The pages find that the state-update kernel's speedup shrinks end to end,
since the rest of a decode step is unchanged ([sum] "Results" and
"Significance"; [abs]).  This harness shows that effect without trained
weights.  It stacks L layers with seeded random weights; per layer and token:

    h  = rms(x)                                 RMS normalisation, no gain
    [q | k | v | zb | zd] = h @ W_in            one input projection
    q, k <- q / sqrt(|q|^2 + d_k 1e-6)          per head (GDN, KDA only)
    beta = sigmoid(zb);  ld = -softplus(zd - 3) per head (GDN) or per key
    o  = state step                             DeltaLog or eager, libdeltalog
    x += o @ W_o
    [g | u] = rms(x) @ W_gu;   x += (silu(g) * u) @ W_dn

and the next token's input is rms of the last layer's output.  There is no
attention layer, expert routing, embedding or sampling: the stand-ins put a
realistic amount of weight streaming between the state steps (which also
keeps the states out of the Infinity Cache) and the small elementwise work of
a decode step.  The projections are plain library GEMMs (torch, hipBLASLt)
and the glue is torch elementwise work; neither belongs to the decode step,
which runs in libdeltalog.

--gated puts a per-head norm with an output gate behind the step, as GDN and
KDA layers have it: o <- rms(o) g silu(h @ W_g).  --fused runs the residual
adds and norms (and that gated norm) as the library's fused operators instead
of torch's elementwise ones.  --prompt T first runs a prompt of T tokens per
request through all layers as whole sequences (the library's scan, from the
initial states), times it, and decodes from the states it leaves.

Each path is captured as a HIP graph of one merge cycle (M tokens through all
layers) and replayed.  One JSON line reports tokens/s for both paths, the
end-to-end speedup, the state steps alone (same layers and shapes, also graph
replayed), and the end-to-end speedup Amdahl's law predicts from the eager
path's state-step share.
"""
from __future__ import annotations

import argparse
import json
import os
import sys
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import synth  # noqa: E402

EPS = 1e-6
DECAY_SHIFT = 3.0


def log(*a):
    print(*a, file=sys.stderr, flush=True)


class SyntheticDecoder:
    """L layers of the stand-in model above on cuda:0.  `path` is "deltalog"
    (dl_decode_step on a DeltaLog state per layer) or "eager" (dl_eager_step
    on a dense state per layer).  `wdtype` is the weight and activation
    dtype of the GEMMs and of q, k, v (torch.bfloat16 or torch.float32).
    Layers can share weight tensors with another decoder (`weights_from`).
    `fused`: residual adds and norms as the library's operators."""

    def __init__(self, ds: synth.DecoderShape, path: str, wdtype, weights_from=None, fused=False):
        import torch
        import recurrent_state_update_amd as rsu
        assert path in ("deltalog", "eager")
        self.ds, self.path, self.wd, self.fused = ds, path, wdtype, fused
        self.rsu = rsu
        self.layers = []
        for l in range(ds.L):
            if weights_from is None:
                p = synth.decoder_layer(ds, l)
                # kept as [out, in] (the nn.Linear layout, for which the
                # library GEMM picks a better kernel at decode batch sizes)
                lay = {k: torch.from_numpy(p[k]).cuda().to(wdtype).t().contiguous()
                       for k in ("W_in", "W_o", "W_gu", "W_dn", "W_g") if k in p}
                lay["g"] = torch.from_numpy(p["g"]).cuda() if ds.gated else None
                lay["u"] = None if p["u"] is None else torch.from_numpy(p["u"]).cuda()
                lay["X0"] = p["X0"]
            else:
                src = weights_from.layers[l]
                lay = {k: src[k] for k in ("W_in", "W_o", "W_gu", "W_dn", "W_g", "g", "u", "X0") if k in src}
            lay["base"] = torch.from_numpy(lay["X0"]).cuda()
            if path == "deltalog":
                lay["st"] = rsu.DeltaLogState(ds.op, ds.B, ds.H, ds.dk, ds.dv, ds.M, dtype=wdtype,
                                              base=lay["base"], u=lay["u"])
            self.layers.append(lay)

    def _norm_heads(self, t, d):
        import torch.nn.functional as F
        # t / sqrt(|t|^2 + d*EPS) == rms_norm(t, eps=EPS) / sqrt(d)
        return F.rms_norm(t, (d,), eps=EPS) * (1.0 / d ** 0.5)

    def layer_inputs(self, x, lay):
        """Norm, projection and per-head prep of one layer (project)."""
        import torch.nn.functional as F
        return self.project(F.rms_norm(x, (self.ds.hidden,), eps=EPS).to(self.wd), lay)

    def project(self, h, lay):
        """Projection and per-head prep of one layer: q, k, v in the input
        dtype, beta and ld in fp32, shaped as the decode step takes them, for
        rows h [n, hidden] (a request's tokens, or one of each request)."""
        import torch
        import torch.nn.functional as F
        ds = self.ds
        n, H = h.shape[0], ds.H
        p = F.linear(h, lay["W_in"]).float()
        q, k, v, zb, zd = torch.split(p, ds.proj_split, dim=1)
        q = q.reshape(n, H, ds.dk)
        k = k.reshape(n, H, ds.dk)
        if ds.op != "rwkv6":
            q, k = self._norm_heads(q, ds.dk), self._norm_heads(k, ds.dk)
            beta = torch.sigmoid(zb).contiguous()
        else:
            beta = None
        ld = -F.softplus(zd - DECAY_SHIFT)
        ld = ld.reshape(n, H) if ds.op == "gdn" else ld.reshape(n, H, ds.dk)
        return (q.to(self.wd).contiguous(), k.to(self.wd).contiguous(),
                v.reshape(n, H, ds.dv).to(self.wd).contiguous(), beta, ld.contiguous())

    def state_step(self, lay, q, k, v, beta, ld):
        if self.path == "deltalog":
            return lay["st"].step(q, k, v, beta, ld)
        return self.rsu.eager_step(self.ds.op, lay["base"], q, k, v, beta, ld, lay["u"])

    def sequence_step(self, lay, q, k, v, beta, ld, B, T):
        """The recurrence over T tokens of each of B requests (rows request by
        request), from the layer's states, which it leaves at the end ones."""
        import torch
        args = [None if t is None else t.unflatten(0, (B, T)) for t in (q, k, v, beta, ld)]
        if self.path == "deltalog":
            return lay["st"].prefill(*args).flatten(0, 1)
        with torch.no_grad():
            o, s = self.rsu.scan(self.ds.op, *args, u=lay["u"], initial_state=lay["base"])
            lay["base"].copy_(s)
        return o.flatten(0, 1)

    def add_norm(self, x, y=None, dtype=None):
        """x + y, and its norm (without y: of x) in the GEMMs' dtype."""
        import torch.nn.functional as F
        dtype = self.wd if dtype is None else dtype
        if self.fused:
            return self.rsu.residual_norm(x, y, eps=EPS, dtype=dtype)
        x = x if y is None else x + y.float()
        return x, F.rms_norm(x, (self.ds.hidden,), eps=EPS).to(dtype)

    def output(self, o, h, lay):
        """o [n,H,dv] of the recurrence as rows for the output projection."""
        import torch.nn.functional as F
        ds = self.ds
        if ds.gated:
            gate = F.linear(h, lay["W_g"]).unflatten(1, (ds.H, ds.dv))
            if self.fused:
                o = self.rsu.gated_norm(o, gate, lay["g"], eps=EPS)
            else:
                o = F.rms_norm(o.float(), (ds.dv,), eps=EPS) * lay["g"] * F.silu(gate.float())
        return o.reshape(-1, ds.H * ds.dv).to(self.wd)

    def rows(self, x, recurrence):
        """Rows x [n, hidden] fp32 through all layers; recurrence(lay, q, k, v,
        beta, ld) gives their o.  Returns the last layer's output and its rms
        (both fp32)."""
        import torch
        import torch.nn.functional as F
        ds = self.ds
        x, h = self.add_norm(x)
        for i, lay in enumerate(self.layers):
            o = recurrence(lay, *self.project(h, lay))
            x, h = self.add_norm(x, F.linear(self.output(o, h, lay), lay["W_o"]))
            g, u = F.linear(h, lay["W_gu"]).float().split(ds.ffn, dim=1)
            last = i + 1 == len(self.layers)
            y = F.linear((F.silu(g) * u).to(self.wd), lay["W_dn"])
            if last and self.wd != torch.float32:
                x = x + y.float()
                h = self.add_norm(x, dtype=torch.float32)[1]
            else:
                x, h = self.add_norm(x, y)
        return x, h

    def prompt(self, X):
        """A prompt's hidden inputs X [B, T, hidden] fp32 through all layers,
        leaving every layer's states.  Returns what `token` returns for each
        request's last token."""
        B, T, hidden = X.shape
        out, h = self.rows(X.reshape(B * T, hidden), lambda lay, *a: self.sequence_step(lay, *a, B, T))
        return out.unflatten(0, (B, T))[:, -1], h.unflatten(0, (B, T))[:, -1]

    def token(self, x):
        """One token through all layers.  x [B, hidden] fp32.  Returns the
        last layer's output (fp32) and the next token's input rms(output)."""
        import torch.nn.functional as F
        ds = self.ds
        if self.fused or ds.gated:
            return self.rows(x, self.state_step)
        for lay in self.layers:
            o = self.state_step(lay, *self.layer_inputs(x, lay))
            x = x + F.linear(o.reshape(ds.B, ds.H * ds.dv).to(self.wd), lay["W_o"]).float()
            gu = F.linear(F.rms_norm(x, (ds.hidden,), eps=EPS).to(self.wd), lay["W_gu"]).float()
            g, u = gu.split(ds.ffn, dim=1)
            x = x + F.linear((F.silu(g) * u).to(self.wd), lay["W_dn"]).float()
        return x, F.rms_norm(x, (ds.hidden,), eps=EPS)

    def capture_cycle(self, x_static):
        """A HIP graph of M tokens (one merge cycle, so the host-side log
        schedule ends where it began) that reads its input from x_static,
        writes every token's output into the returned [M, B, hidden] buffer
        and leaves the next input in x_static."""
        import torch
        ds = self.ds
        outs = torch.empty(ds.M, ds.B, ds.hidden, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x = x_static
            for t in range(ds.M):
                out, x = self.token(x)
                outs[t].copy_(out)
            x_static.copy_(x)
        return g, outs

    def close(self):
        for lay in self.layers:
            if "st" in lay:
                lay["st"].close()


def warm_up(dec, x, tokens: int):
    """Run `tokens` tokens directly on a side stream (library handles and
    workspaces are created outside any capture), then rejoin."""
    import torch
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(tokens):
            _, x = dec.token(x)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    return x


def time_prompt(dec, X, passes: int = 4):
    """Run a prompt `passes` times from the initial states, the first untimed;
    the next token's input, and the mean time of a pass in ms."""
    import torch
    t = []
    for _ in range(passes):
        for lay in dec.layers:
            lay["base"].copy_(torch.from_numpy(lay["X0"]))
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        _, x = dec.prompt(X)
        e[1].record()
        torch.cuda.synchronize()
        t.append(e[0].elapsed_time(e[1]))
    return x.contiguous(), sum(t[1:]) / (passes - 1)


def time_graph(g, replays: int) -> float:
    import torch
    g.replay()
    torch.cuda.synchronize()
    t0 = torch.cuda.Event(enable_timing=True)
    t1 = torch.cuda.Event(enable_timing=True)
    t0.record()
    for _ in range(replays):
        g.replay()
    t1.record()
    torch.cuda.synchronize()
    return t0.elapsed_time(t1) / replays


def state_only_graph(dec, inputs):
    """A graph of the same state steps as one merge cycle of the model (M
    tokens x L layers) on fixed, pre-staged inputs."""
    import torch
    ds = dec.ds
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for t in range(ds.M):
            for lay in dec.layers:
                dec.state_step(lay, *inputs)
    return g


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--op", default="gdn", choices=["gdn", "kda", "rwkv6"])
    ap.add_argument("--layers", type=int, default=8)
    ap.add_argument("--B", type=int, default=64)
    ap.add_argument("--H", type=int, default=32)
    ap.add_argument("--d", type=int, default=128)
    ap.add_argument("--M", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--ffn", type=int, default=4096)
    ap.add_argument("--cycles", type=int, default=8, help="timed graph replays (M tokens each)")
    ap.add_argument("--gated", action="store_true", help="a gated per-head norm behind the step")
    ap.add_argument("--fused", action="store_true", help="residual adds and norms as the library's operators")
    ap.add_argument("--prompt", type=int, default=0, help="tokens per request run as whole sequences first")
    args = ap.parse_args()

    import torch
    assert torch.cuda.is_available(), "bench_decoder.py needs a GPU"
    torch.cuda.set_device(0)
    ds = synth.DecoderShape(args.op, args.layers, args.B, args.H, args.d, args.d, args.M,
                            args.hidden, args.ffn, gated=args.gated)
    wd = torch.bfloat16
    t0 = time.time()
    dl = SyntheticDecoder(ds, "deltalog", wd, fused=args.fused)
    eg = SyntheticDecoder(ds, "eager", wd, weights_from=dl, fused=args.fused)
    log(f"built {ds.describe()} in {time.time() - t0:.1f}s")
    x0 = torch.from_numpy(synth.decoder_input(ds)).cuda()

    res, prompt = {}, None
    for name, dec in (("deltalog", dl), ("eager", eg)):
        x = x0.clone()
        if args.prompt:
            X = torch.from_numpy(synth.decoder_prompt(ds, args.prompt)).cuda()
            x, ms = time_prompt(dec, X)
            if name == "deltalog":
                prompt = dict(tokens_per_request=args.prompt, ms=round(ms, 4),
                              tokens_per_s=round(ds.B * args.prompt / (ms * 1e-3), 1))
                log(f"prompt: {ms:.3f} ms for {ds.B} x {args.prompt} tokens")
        x = warm_up(dec, x, ds.M)
        g, _ = dec.capture_cycle(x)
        ms = time_graph(g, args.cycles) / ds.M
        res[name] = dict(tokens_per_s=round(ds.B / (ms * 1e-3), 1), ms_per_token=round(ms, 5))
        log(f"{name}: {ms * 1e3:.1f} us per token step ({ds.L} layers)")
        del g

    w = synth.Workload(11, ds.op, ds.B, ds.H, ds.dk, ds.dv, ds.M, 1, "bf16")
    s = synth.step(w, 0)
    inputs = tuple(None if s[k] is None else
                   torch.from_numpy(s[k]).cuda().to(wd if k in ("q", "k", "v") else torch.float32)
                   for k in ("q", "k", "v", "beta", "ld"))
    st_ms = {}
    for name, dec in (("deltalog", dl), ("eager", eg)):
        g = state_only_graph(dec, inputs)
        st_ms[name] = time_graph(g, args.cycles) / ds.M
        del g
    kernel_speedup = st_ms["eager"] / st_ms["deltalog"]
    share = st_ms["eager"] / res["eager"]["ms_per_token"]
    e2e = res["eager"]["ms_per_token"] / res["deltalog"]["ms_per_token"]
    out = {
        "metric": "synthetic decoder tokens/s, DeltaLog vs eager state step",
        "unit": "tokens/s",
        "config": {"workload": f"synthetic {ds.op.upper()} decoder: {ds.L} recurrent layers, B={ds.B} "
                               f"H={ds.H} d_k=d_v={ds.dk} M={ds.M}, hidden {ds.hidden}, gated MLP "
                               f"{ds.ffn}, bf16 weights, random init",
                   "op": ds.op, "layers": ds.L, "B": ds.B, "H": ds.H, "d": ds.dk, "M": ds.M,
                   "hidden": ds.hidden, "ffn": ds.ffn},
        "deltalog": res["deltalog"],
        "eager": res["eager"],
        "e2e_speedup": round(e2e, 3),
        "state_step_only": {"deltalog_ms_per_token": round(st_ms["deltalog"], 5),
                            "eager_ms_per_token": round(st_ms["eager"], 5),
                            "kernel_speedup": round(kernel_speedup, 3)},
        "eager_state_share": round(share, 3),
        "amdahl_predicted_e2e": round(1.0 / ((1.0 - share) + share / kernel_speedup), 3),
        "data": "synthetic (seeded PCG64 weights, states and first input)",
    }
    if args.gated or args.fused:
        out["config"].update(gated=args.gated, fused=args.fused)
    if prompt:
        out["prompt"] = prompt
    dl.close()
    print(json.dumps(out), flush=True)


if __name__ == "__main__":
    main()
