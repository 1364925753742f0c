"""What the operators of a state space layer compute, and cases to measure them on.

  short_conv         the short causal convolution of every channel in front of
                     a recurrence, with its SiLU: prompts, training, and
  short_conv_step    one token of each of many requests
  ssm_scan           the selective state space recurrence, a diagonal state per
                     channel: prompts, training, and
  ssm_step           one token of each of many requests
  residual_norm_fp8  residual add and RMS norm, the result in 8 bits (e4m3) with
                     a scale for each row, or for every 128 columns of one

`own` false: the plain forms below, in elementary torch operations.  `own`
true: the framework's calls."""
import math

import torch

if __name__ == "__main__":
    raise SystemExit("a module of cases, not a program")

own = False

EPS = 1e-6
E4M3_MOST = 448.0  # the largest e4m3 value


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # several prompts packed, q, k and v of 32 heads of 128 being one slice
        # of a wider projection, some of them going on from a cached state
        dict(name="conv packed prompts", kind="conv", lens="731,64,1,1537,333,90", channels=12288, taps=4, dtype="bf16",
             bias=False, sliced=True, init=True, train=False),
        # a training step's documents
        dict(name="conv training", kind="conv", lens="4096,1000,3096", channels=4096, taps=4, dtype="bf16", bias=True,
             sliced=False, init=False, train=True),
        # an odd width with three taps in fp32
        dict(name="conv training odd fp32", kind="conv", lens="301,2,474", channels=1531, taps=3, dtype="f32", bias=True,
             sliced=False, init=True, train=True),
        # a decode step of 64 requests, their states anywhere in a cache
        dict(name="conv decode", kind="conv step", rows=64, slots=96, channels=12288, taps=4, dtype="bf16", bias=True),
        # a few tokens through a toy layer: latency only
        dict(name="ssm tiny fp32", kind="ssm", lens="5", channels=32, states=16, groups=1, dtype="f32", gate=True,
             sliced=False, init=True, train=False),
        # a long prompt on its own
        dict(name="ssm prompt", kind="ssm", lens="4096", channels=4096, states=16, groups=1, dtype="bf16", gate=True,
             sliced=True, init=False, train=False),
        # prompts of several requests packed, a narrower layer
        dict(name="ssm packed prompts", kind="ssm", lens="731,64,1,1537,333,90", channels=2048, states=16, groups=1,
             dtype="bf16", gate=True, sliced=True, init=True, train=False),
        # a training step
        dict(name="ssm training", kind="ssm", lens="2048,2048", channels=2048, states=16, groups=1, dtype="bf16",
             gate=True, sliced=True, init=False, train=True),
        # wide states in two groups, no gate, fp32
        dict(name="ssm training wide fp32", kind="ssm", lens="301,17,300", channels=512, states=64, groups=2, dtype="f32",
             gate=False, sliced=False, init=True, train=True),
        # a decode step of 64 requests
        dict(name="ssm decode", kind="ssm step", rows=64, slots=96, channels=4096, states=16, groups=1, dtype="bf16",
             gate=True),
        # the residual stream of a decode step, and of a long prompt
        dict(name="norm fp8 decode", kind="norm", rows=64, D=2048, dtype="bf16", scaled=False, group=0),
        dict(name="norm fp8 prompt", kind="norm", rows=16384, D=2048, dtype="bf16", scaled=True, group=128),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cut(rng, total, n):
    cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    kind = rng.choice(["conv", "conv", "conv step", "ssm", "ssm", "ssm", "ssm step", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "norm":
        group = rng.choice([0, 0, 128])
        D = 128 * _log_uniform(rng, 1, 64) if group else _log_uniform(rng, 48, 8192)
        return dict(kind=kind, rows=_log_uniform(rng, 1, 16384 * 2048 // D), D=D, dtype=dtype, scaled=rng.random() < 0.5,
                    group=group)
    train = rng.random() < 0.5
    if kind in ("conv step", "ssm step"):
        rows = _log_uniform(rng, 1, 256)
        case = dict(kind=kind, rows=rows, slots=rows + rng.randrange(64), dtype=dtype)
        if kind == "conv step":
            return dict(case, channels=_log_uniform(rng, 16, 12288), taps=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.5)
        groups = rng.choice([1, 1, 1, 2, 4])
        return dict(case, channels=groups * _log_uniform(rng, 8, 4096 // groups), states=rng.choice([16, 16, 16, 8, 24, 64]),
                    groups=groups, gate=rng.random() < 0.7)
    n = _log_uniform(rng, 1, 12)
    if kind == "conv":
        C = _log_uniform(rng, 16, 12288)
        total = _log_uniform(rng, n, max(n, min(16384, 8192 * 4096 // C)))
        return dict(kind=kind, lens=_cut(rng, total, n), channels=C, taps=rng.choice([2, 3, 4, 4]), dtype=dtype,
                    bias=rng.random() < 0.5, sliced=rng.random() < 0.5, init=rng.random() < 0.5, train=train)
    groups = rng.choice([1, 1, 1, 2, 4])
    N = rng.choice([16, 16, 16, 16, 8, 24, 32, 64])
    C = groups * _log_uniform(rng, 8, 4096 // groups)
    total = _log_uniform(rng, n, max(n, min(8192, (2048 if train else 4096) * 4096 * 16 // (C * N))))
    return dict(kind=kind, lens=_cut(rng, total, n), channels=C, states=N, groups=groups, dtype=dtype,
                gate=rng.random() < 0.7, sliced=rng.random() < 0.5, init=rng.random() < 0.5, train=train)


def _type(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "norm":
        n = case["rows"] * case["D"]
        # x, y in; x, h and its scales out
        scales = case["rows"] * (case["D"] // case["group"] if case["group"] else 1)
        return {"bytes": n * (4 + e + 4 + 1) + 4 * scales, "flops": 10 * n}
    step, C = case["kind"].endswith("step"), case["channels"]
    T, n = (case["rows"], case["rows"]) if step else (sum(_lens(case)), len(_lens(case)))
    train = not step and case["train"]
    if case["kind"].startswith("conv"):
        W = case["taps"]
        state = n * (W - 1) * C * e
        fwd = 2 * T * C * e + state * (2 if step or case["init"] else 1)
        flops = T * C * (2 * W + 5)
        if not train:
            return {"bytes": fwd, "flops": flops}
        # x and the cotangents in; a gradient for each input out
        return {"bytes": fwd + 3 * T * C * e + state * (2 if case["init"] else 1), "flops": flops + T * C * (6 * W + 10)}
    N, G, gate = case["states"], case["groups"], case["gate"]
    inputs = T * e * (C * (3 if gate else 2) + 2 * G * N)
    state = n * C * N * 4
    fwd = inputs + T * C * e + state * (2 if step or case["init"] else 1)
    flops = T * C * (7 * N + 15)
    if not train:
        return {"bytes": fwd, "flops": flops}
    return {"bytes": fwd + 2 * inputs + T * C * e + state * (2 if case["init"] else 1), "flops": flops + T * C * (20 * N + 40)}


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale + shift

    def rows_of(T, C, sliced):  # [T, C], or such a slice of a wider projection
        return normal(T, 2 * C).to(dt)[:, C:] if sliced else normal(T, C).to(dt)

    dt = _type(case["dtype"])
    st = dict(case)
    if case["kind"] == "norm":
        rows, D = case["rows"], case["D"]
        st["x"] = normal(rows, D, scale=2.0)
        st["y"] = normal(rows, D).to(dt)
        st["weight"] = normal(D, scale=0.2, shift=1.0) if case["scaled"] else None
        st["scale"] = normal(D, scale=0.1, shift=0.5) if case["scaled"] else None
        return st
    step, C = case["kind"].endswith("step"), case["channels"]
    if step:
        T = case["rows"]
        st["rows"] = torch.randperm(case["slots"], generator=g, device="cuda")[:T].int()
        n = case["slots"]
    else:
        st["lens"] = _lens(case)
        T, n = sum(st["lens"]), len(st["lens"])
        st["cu"] = torch.tensor([sum(st["lens"][:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    train, sliced = not step and case["train"], not step and case["sliced"]
    if case["kind"].startswith("conv"):
        W = case["taps"]
        x = rows_of(T, C, sliced)
        weight = normal(C, W, scale=W ** -0.5)
        bias = normal(C, scale=0.2) if case["bias"] else None
        state = normal(n, W - 1, C).to(dt) if step or case["init"] else None
        st["in"] = dict(x=x, weight=weight, bias=bias, state=state)
        if train:
            st["dy"], st["ds"] = normal(T, C).to(dt), normal(n, W - 1, C).to(dt)
        return st
    N, G = case["states"], case["groups"]
    # channels remember for 10 to 1000 tokens, their states for up to N times less
    rate = torch.rand(C, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3)
    bc = normal(T, 2 * G * N + 8).to(dt)  # the projection of x that gives B and C, and what dt comes from
    B, Cs = (bc[:, 8 + i * G * N: 8 + (i + 1) * G * N].unflatten(1, (G, N)) for i in (0, 1))
    if not sliced:
        B, Cs = B.contiguous(), Cs.contiguous()
    st["in"] = dict(x=normal(T, C).to(dt), dt=normal(T, C, scale=0.7).to(dt),
                    A=-torch.arange(1, N + 1, device="cuda") * (normal(C, N, scale=0.1).exp()), B=B, C=Cs,
                    D=normal(C, scale=0.3, shift=1.0), z=rows_of(T, C, sliced) if case["gate"] else None,
                    dt_bias=rate.exp().expm1().log(),
                    state=normal(n, C, N, scale=0.3) if step or case["init"] else None)
    if train:
        st["dy"], st["ds"] = normal(T, C).to(dt), normal(n, C, N, scale=0.3)
    return st


# ------------------------------------------------------------- plain forms --

def _silu(x):
    return x / (1 + (-x).exp())


def _softplus(x):
    return x.clamp(min=0) + (-x.abs()).exp().log1p()


def _tokens(cu, T):
    """Every token's sequence, and its place in it."""
    cu, token = cu.long(), torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu[1:], token, right=True)
    return seq, token - cu[seq], cu


def _plain_conv(cu, x, weight, bias, state):
    T, C = x.shape
    W = weight.shape[1]
    seq, pos, cu = _tokens(cu, T)
    x32 = x.float()
    old = torch.zeros(cu.numel() - 1, W - 1, C, device=x.device) if state is None else state.float()
    token = torch.arange(T, device=x.device)
    s = 0 if bias is None else bias
    for k in range(W):  # k tokens back
        before = old[seq, (W - 1 - k + pos).clamp(max=W - 2)]
        s = s + weight[:, W - 1 - k] * torch.where((pos >= k)[:, None], x32[(token - k).clamp(min=0)], before)
    at = (cu[1:] - cu[:-1])[:, None] - (W - 1) + torch.arange(W - 1, device=x.device)  # of each sequence's last inputs
    seqs = torch.arange(cu.numel() - 1, device=x.device)[:, None]
    end = torch.where((at >= 0)[..., None], x32[(cu[:-1, None] + at).clamp(0, max(T - 1, 0))],
                      old[seqs, (at + W - 1).clamp(max=W - 2)])
    return _silu(s).to(x.dtype), end.to(x.dtype)


def _plain_conv_step(rows, x, weight, bias, state):
    rows = rows.long()
    seen = torch.cat([state[rows], x[:, None]], 1)
    s = (seen.float() * weight.t()).sum(1)
    state[rows] = seen[:, 1:]
    return _silu(s if bias is None else s + bias).to(x.dtype), state


def _per_channel(x, C):
    """[T, G, N] as [T, C, N], every group's row for each of its channels."""
    T, G, N = x.shape
    return x.float()[:, :, None].expand(T, G, C // G, N).reshape(T, C, N)


def _plain_ssm(cu, x, dt, A, B, C, D, z, dt_bias, state):
    """All prefixes by doubling: after the step of stride s, (a, h) take every
    token back 2s tokens."""
    T, ch = x.shape
    seq, pos, cu = _tokens(cu, T)
    delta = _softplus(dt.float() + dt_bias)
    x32 = x.float()
    a = (delta[..., None] * A).exp()
    h = (delta * x32)[..., None] * _per_channel(B, ch)
    first = (pos == 0)[:, None, None]
    if state is not None:
        h = torch.where(first, h + a * state[seq], h)
    a = a.masked_fill(first, 0)
    s = 1
    while s < T:
        h = torch.cat([h[:s], h[s:] + a[s:] * h[:-s]])
        a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    y = (h * _per_channel(C, ch)).sum(-1) + D * x32
    if z is not None:
        y = y * _silu(z.float())
    old = torch.zeros(cu.numel() - 1, *A.shape, device=x.device) if state is None else state
    end = torch.where((cu[1:] > cu[:-1])[:, None, None], h[(cu[1:] - 1).clamp(min=0)], old)
    return y.to(x.dtype), end


def _plain_ssm_step(rows, x, dt, A, B, C, D, z, dt_bias, state):
    rows = rows.long()
    ch = x.shape[1]
    delta, x32 = _softplus(dt.float() + dt_bias), x.float()
    h = (delta[..., None] * A).exp() * state[rows] + (delta * x32)[..., None] * _per_channel(B, ch)
    y = (h * _per_channel(C, ch)).sum(-1) + D * x32
    if z is not None:
        y = y * _silu(z.float())
    state[rows] = h
    return y.to(x.dtype), state


def _plain_norm(x, y, scale, weight, group):
    y32 = y.float()
    x = x + (y32 if scale is None else y32 * scale)
    h = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    if weight is not None:
        h = h * weight
    h = h.unflatten(1, (-1, group or h.shape[1]))
    s = h.abs().amax(-1) / E4M3_MOST
    h = (h / s[..., None]).flatten(1)
    return x, h.to(torch.float8_e4m3fn), s if group else s[:, 0]


# ----------------------------------------------------------------- one pass --

def run(state):
    if own:
        import recurrent_state_update_amd as rsu
    kind = state["kind"]
    if kind == "norm":
        args = [state[n] for n in ("x", "y", "scale", "weight")]
        x, h, s = (rsu.residual_norm_fp8(*args, eps=EPS, group=state["group"] or None) if own
                   else _plain_norm(*args, state["group"]))
        return dict(x=x, h=h, scale=s)
    if kind == "conv step":
        i = state["in"]
        if own:
            y, s = rsu.short_conv_step(i["x"], i["state"], i["weight"], i["bias"], rows=state["rows"]), i["state"]
        else:
            y, s = _plain_conv_step(state["rows"], **i)
        return dict(y=y, state=s)
    if kind == "ssm step":
        i = state["in"]
        if own:
            y, s = rsu.ssm_step(i["x"], i["dt"], i["state"], i["A"], i["B"], i["C"], i["D"], i["z"], i["dt_bias"],
                                rows=state["rows"]), i["state"]
        else:
            y, s = _plain_ssm_step(state["rows"], **i)
        return dict(y=y, state=s)
    train = state["train"]
    x = {n: t.detach().requires_grad_(True) if train and t is not None else t for n, t in state["in"].items()}
    if kind == "conv":
        if own:
            y, s = rsu.short_conv(x["x"], x["weight"], x["bias"], initial_state=x["state"], cu_seqlens=state["cu"])
        else:
            y, s = _plain_conv(state["cu"], **x)
    elif own:
        y, s = rsu.ssm_scan(x["x"], x["dt"], x["A"], x["B"], x["C"], x["D"], x["z"], x["dt_bias"],
                            initial_state=x["state"], cu_seqlens=state["cu"])
    else:
        y, s = _plain_ssm(state["cu"], **x)
    out = dict(y=y, state=s)
    if train:
        wrt = {n: t for n, t in x.items() if t is not None}
        grads = torch.autograd.grad([y, s], list(wrt.values()), [state["dy"], state["ds"]])
        out.update(("d" + n, t) for n, t in zip(wrt, grads))
    return {n: t.detach() for n, t in out.items()}


# -------------------------------------------------------------- in 64 bits --

def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "norm":
        x, y, s, w = (1.0 if st[n] is None else st[n].double() for n in ("x", "y", "scale", "weight"))
        x = x + y * s
        h = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        most = h.reshape(h.shape[0], -1, case["group"] or case["D"]).abs().max(-1).values
        scale = most / E4M3_MOST
        h = (h.reshape(*scale.shape, -1) / scale.unsqueeze(-1)).reshape(h.shape)
        return dict(x=x, h=h, scale=scale if case["group"] else scale.squeeze(1))
    x = {n: None if t is None else t.double() for n, t in st["in"].items()}
    exact_of = _exact_conv if case["kind"].startswith("conv") else _exact_ssm
    if not case["kind"].endswith("step"):
        return exact_of(x, st["lens"], st if case["train"] else None)
    # one token each, as sequences of length one
    rows = st["rows"].tolist()
    out = exact_of(dict(x, state=x["state"][rows]), [1] * len(rows), None)
    state = x["state"].clone()
    for i, r in enumerate(rows):
        state[r] = out["state"][i]
    return dict(y=out["y"], state=state)


def _exact_conv(x, lens, train):
    """Each sequence by itself, behind the W - 1 inputs before it."""
    w, b = x["weight"], x["bias"]
    C, W = w.shape
    out = {n: [] for n in ("y", "state", "dx", "dstate")}
    dw, db, at = torch.zeros_like(w), torch.zeros_like(w[:, 0]), 0
    for n, L in enumerate(lens):
        old = torch.zeros(W - 1, C, dtype=w.dtype, device=w.device) if x["state"] is None else x["state"][n]
        seen = torch.cat([old, x["x"][at:at + L]])
        s = torch.zeros(L, C, dtype=w.dtype, device=w.device) if b is None else b.expand(L, C)
        for j in range(W):
            s = s + seen[j:j + L] * w[:, j]
        sig = torch.sigmoid(s)
        out["y"].append(s * sig)
        out["state"].append(seen[L:])
        if train:
            ds = train["dy"][at:at + L].double() * sig * (1 + s * (1 - sig))
            dseen = torch.zeros_like(seen)
            dseen[L:] += train["ds"][n].double()
            for j in range(W):
                dseen[j:j + L] += ds * w[:, j]
                dw[:, j] += (ds * seen[j:j + L]).sum(0)
            db += ds.sum(0)
            out["dx"].append(dseen[W - 1:])
            out["dstate"].append(dseen[:W - 1])
        at += L
    got = dict(y=torch.cat(out["y"]), state=torch.stack(out["state"]))
    if train:
        got.update(dx=torch.cat(out["dx"]), dweight=dw)
        if b is not None:
            got["dbias"] = db
        if x["state"] is not None:
            got["dstate"] = torch.stack(out["dstate"])
    return got


def _exact_ssm(x, lens, train):
    """Token by token; the adjoint token by token too."""
    A, dev = x["A"], x["A"].device
    ch, N = A.shape
    T, G = sum(lens), x["B"].shape[1]
    if train and T * ch * N * 8 > 60e9:
        return None  # its states would not fit
    raw = x["dt"] + x["dt_bias"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    z = x["z"]
    sig = None if z is None else torch.sigmoid(z)
    y = torch.zeros_like(x["x"])
    before, ends = [], []

    def wide(v):  # [G, N] -> [G, C / G, N], broadcast
        return v[:, None].expand(G, ch // G, N).reshape(ch, N)

    t = 0
    for n, L in enumerate(lens):
        h = torch.zeros(ch, N, dtype=A.dtype, device=dev) if x["state"] is None else x["state"][n]
        for _ in range(L):
            if train:
                before.append(h)
            h = torch.exp(delta[t, :, None] * A) * h + (delta[t] * x["x"][t])[:, None] * wide(x["B"][t])
            y[t] = (h * wide(x["C"][t])).sum(1)
            t += 1
        ends.append(h)
    y = y + x["D"] * x["x"]
    out = dict(y=y if z is None else y * z * sig, state=torch.stack(ends))
    if not train:
        return out
    dy = train["dy"].double()
    if z is not None:
        out["dz"] = dy * y * sig * (1 + z * (1 - sig))
        dy = dy * z * sig
    dx, dd, dB, dC = dy * x["D"], torch.zeros_like(delta), torch.zeros_like(x["B"]), torch.zeros_like(x["C"])
    dA, dstate = torch.zeros_like(A), []
    t = T
    for n in reversed(range(len(lens))):
        g = train["ds"][n].double()
        for _ in range(lens[n]):
            t -= 1
            a, b = torch.exp(delta[t, :, None] * A), wide(x["B"][t])
            h = a * before[t] + (delta[t] * x["x"][t])[:, None] * b
            g = g + dy[t, :, None] * wide(x["C"][t])
            dC[t] = (dy[t, :, None] * h).reshape(G, -1, N).sum(1)
            dB[t] = ((delta[t] * x["x"][t])[:, None] * g).reshape(G, -1, N).sum(1)
            gb, gah = (g * b).sum(1), g * a * before[t]
            dx[t] += gb * delta[t]
            dd[t] = gb * x["x"][t] + (gah * A).sum(1)
            dA += delta[t, :, None] * gah
            g = a * g
        dstate.append(g)
    ddt = dd * torch.sigmoid(raw)
    out.update(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(dy * x["x"]).sum(0), ddt_bias=ddt.sum(0))
    if x["state"] is not None:
        out["dstate"] = torch.stack(dstate[::-1])
    return out
