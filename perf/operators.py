"""What the sequence operators compute, and cases to measure them on.

Three operators next to the decode step, each forward and (training) backward:

  scan           the GDN / KDA / RWKV6 recurrence of the decode step over whole
                 (packed) sequences: a prompt's prefill, or a training step
  gated_norm     RMS norm of the recurrence's output per head, times its gain
                 and the SiLU of the output gate
  residual_norm  residual add with a per-channel residual scale, then the RMS
                 norm that opens the next block

`own` false: the plain forms below, in elementary torch operations.  `own`
true: the framework's calls."""
import math

import torch

if __name__ == "__main__":
    raise SystemExit("a module of cases, not a program")

own = False

EPS = 1e-6


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a few tokens through a toy model in fp32: latency only
        dict(name="scan gdn tiny fp32", kind="scan", op="gdn", lens="5", H=2, dk=16, dv=16, dtype="f32",
             batched=False, fused=False, init=True, train=False),
        # a long prompt on its own, the head shape of the headline workload
        dict(name="scan gdn prompt", kind="scan", op="gdn", lens="4096", H=32, dk=128, dv=128, dtype="bf16",
             batched=False, fused=False, init=False, train=False),
        # prompts of several requests packed, continuing from cached states,
        # q, k, v being slices of one projection
        dict(name="scan kda packed prompts", kind="scan", op="kda", lens="731,64,1,1537,333,90", H=32, dk=128,
             dv=128, dtype="bf16", batched=False, fused=True, init=True, train=False),
        # a batch of equal prompts, many narrow heads
        dict(name="scan rwkv6 batch", kind="scan", op="rwkv6", lens="512,512,512,512", H=64, dk=64, dv=64,
             dtype="bf16", batched=True, fused=False, init=False, train=False),
        # training steps: one long sequence; packed documents; a batch in fp32
        dict(name="scan gdn training", kind="scan", op="gdn", lens="4096", H=32, dk=128, dv=128, dtype="bf16",
             batched=False, fused=False, init=False, train=True),
        dict(name="scan kda training packed", kind="scan", op="kda", lens="1000,17,911", H=16, dk=128, dv=128,
             dtype="bf16", batched=False, fused=True, init=False, train=True),
        dict(name="scan rwkv6 training fp32", kind="scan", op="rwkv6", lens="301,301", H=16, dk=64, dv=64,
             dtype="f32", batched=True, fused=False, init=True, train=True),
        # the decode step's output (fp32) of a batch of 64 requests
        dict(name="gated_norm decode", kind="gated", rows=64, H=32, d=128, odtype="f32", dtype="bf16", train=False),
        # a training step's tokens
        dict(name="gated_norm training", kind="gated", rows=8192, H=32, d=128, odtype="bf16", dtype="bf16",
             train=True),
        # one decode step's residual stream; a training step's; an odd width
        dict(name="residual_norm decode", kind="residual", rows=64, D=2048, dtype="bf16", scaled=False, train=False),
        dict(name="residual_norm training", kind="residual", rows=16384, D=2048, dtype="bf16", scaled=True,
             train=True),
        dict(name="residual_norm odd fp32", kind="residual", rows=777, D=1531, dtype="f32", scaled=True, train=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["scan", "scan", "scan", "gated", "residual"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    train = rng.random() < 0.5
    if kind == "gated":
        return dict(kind=kind, rows=_log_uniform(rng, 1, 8192), H=_log_uniform(rng, 1, 32),
                    d=rng.choice([16, 32, 64, 128]), odtype=rng.choice(["f32", "bf16"]), dtype=dtype, train=train)
    if kind == "residual":
        return dict(kind=kind, rows=_log_uniform(rng, 1, 8192), D=_log_uniform(rng, 48, 4096), dtype=dtype,
                    scaled=rng.random() < 0.5, train=train)
    op = rng.choice(["gdn", "kda", "rwkv6"])
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (32, 32), (16, 16), (128, 64)])
    H = _log_uniform(rng, 1, 32)
    batched = rng.random() < 0.3
    n = _log_uniform(rng, 1, 8)
    # tokens so that a case costs no more than the largest listed ones
    most = min(8192, (4096 if op == "gdn" else 2048) * 32 * 128 // (H * dk))
    total = max(n, _log_uniform(rng, n, most))
    if batched:
        lens = [max(1, total // n)] * n
    else:
        cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    return dict(kind=kind, op=op, lens=",".join(map(str, lens)), H=H, dk=dk, dv=dv, dtype=dtype, batched=batched,
                fused=not batched and rng.random() < 0.5, init=rng.random() < 0.5, train=train)


def _type(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "scan":
        lens, H, dk, dv = _lens(case), case["H"], case["dk"], case["dv"]
        th, delta = sum(lens) * H, case["op"] != "rwkv6"
        small = 4 * (delta + (1 if case["op"] == "gdn" else dk))  # beta and log-decay
        states = 4 * len(lens) * H * dk * dv
        inputs = th * (e * (2 * dk + dv) + small)
        # per token and head: the state read by q, the rank-1 update, and for
        # the delta rule the state read by k
        flops = th * dk * dv * (6 if delta else 4)
        if not case["train"]:
            return {"bytes": inputs + th * e * dv + states * (1 + case["init"]), "flops": flops}
        # forward: inputs in, o and the state out; backward: inputs and the
        # two cotangents in, a gradient for each input out
        return {"bytes": 3 * inputs + 2 * th * e * dv + states * (2 + 2 * case["init"]), "flops": 3 * flops}
    if case["kind"] == "gated":
        n = case["rows"] * case["H"] * case["d"]
        eo = 2 if case["odtype"] == "bf16" else 4
        fwd = n * (eo + 2 * e)
        return {"bytes": fwd + (n * (2 * eo + 3 * e) if case["train"] else 0), "flops": n * (30 if case["train"] else 10)}
    n = case["rows"] * case["D"]
    fwd = n * (4 + e + 4 + e)  # x, y in; x, h out
    # backward: x_new and the cotangents of x_new and h in; dx, dy out
    # (and y in again for the scale's gradient)
    bwd = n * (4 + 4 + e + 4 + e + (e if case["scaled"] else 0))
    return {"bytes": fwd + (bwd if case["train"] else 0), "flops": n * (25 if case["train"] else 8)}


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale + shift

    dt = _type(case["dtype"])
    st = dict(case)
    if case["kind"] == "gated":
        rows, H, d = case["rows"], case["H"], case["d"]
        st["o"] = normal(rows, H, d, scale=0.7).to(_type(case["odtype"]))
        st["gate"] = normal(rows, H, d).to(dt)
        st["weight"] = normal(d, scale=0.2, shift=1.0)
        if case["train"]:
            st["dy"] = normal(rows, H, d).to(dt)
    elif case["kind"] == "residual":
        rows, D = case["rows"], case["D"]
        st["x"] = normal(rows, D, scale=2.0)
        st["y"] = normal(rows, D).to(dt)
        st["weight"] = normal(D, scale=0.2, shift=1.0) if case["scaled"] else None
        st["scale"] = normal(D, scale=0.1, shift=0.5) if case["scaled"] else None
        if case["train"]:
            st["dx"] = normal(rows, D)
            st["dh"] = normal(rows, D).to(dt)
    else:
        lens, H, dk, dv, op = _lens(case), case["H"], case["dk"], case["dv"], case["op"]
        T, N = sum(lens), len(lens)
        q, k, v = normal(T, H, dk), normal(T, H, dk), normal(T, H, dv)
        if op != "rwkv6":
            q = q / q.square().sum(-1, keepdim=True).sqrt()
            k = k / k.square().sum(-1, keepdim=True).sqrt()
            beta = torch.sigmoid(normal(T, H))
            ld = -torch.nn.functional.softplus(normal(*((T, H) if op == "gdn" else (T, H, dk)), scale=0.5, shift=-3.0))
        else:
            beta = None
            ld = -torch.exp(normal(T, H, dk, scale=0.5, shift=-0.5))
        q, k, v = (x.to(dt) for x in (q, k, v))
        if case["fused"]:
            p = torch.cat([x.reshape(T, -1) for x in (q, k, v)], dim=1)  # the projection's output
            q, k, v = (x.unflatten(1, (H, -1)) for x in p.split([H * dk, H * dk, H * dv], dim=1))
        do = normal(T, H, dv).to(dt) if case["train"] else None
        if case["batched"]:
            q, k, v, beta, ld, do = (None if x is None else x.unflatten(0, (N, T // N)) for x in (q, k, v, beta, ld, do))
            st["cu"] = None
        else:
            st["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32, device="cuda")
        st["lens"] = lens
        st["in"] = dict(q=q, k=k, v=v, beta=beta, log_decay=ld,
                        u=normal(H, dk, scale=0.1) if op == "rwkv6" else None,
                        initial_state=normal(N, H, dk, dv, scale=0.1) if case["init"] else None)
        if case["train"]:
            st["do"], st["ds"] = do, normal(N, H, dk, dv, scale=0.1)
    return st


# ------------------------------------------------------------- plain forms --

CHUNK = 32


def _plain_scan(op, lens, cu, q, k, v, beta, log_decay, u, initial_state):
    """The recurrence in chunks of CHUNK tokens, in fp32: within a chunk the
    products of all pairs of tokens (and, for the delta rule, the inverse of
    I + A diag(beta) from products alone); from chunk to chunk the state."""
    N, H, dk, dv = len(lens), q.shape[-2], q.shape[-1], v.shape[-1]
    dev, dtype, shape = q.device, q.dtype, v.shape
    L = -(-max(max(lens), 1) // CHUNK) * CHUNK
    nc = L // CHUNK
    T = sum(lens)
    if cu is None:
        cu = torch.arange(N + 1, device=dev) * lens[0]
    cu = cu.long()
    pos = torch.arange(L, device=dev)
    valid = pos[None, :] < (cu[1:] - cu[:-1])[:, None]
    at = (cu[:-1, None] + pos[None, :]).clamp(max=max(T - 1, 0))

    def chunks(x):  # [tokens, H, w] -> [N, H, chunk, CHUNK, w], zeros behind the end
        x = x.reshape(T, H, -1).float()[at] * valid[:, :, None, None]
        return x.permute(0, 2, 1, 3).reshape(N, H, nc, CHUNK, -1)

    Q, K, V, E = chunks(q), chunks(k), chunks(v), chunks(log_decay)
    G = E.cumsum(3)
    read = G if op != "rwkv6" else G - E  # the decay up to the state that a token reads
    strict = torch.ones(CHUNK, CHUNK, device=dev).tril(-1).bool()
    lower = strict if op == "rwkv6" else torch.ones(CHUNK, CHUNK, device=dev).tril().bool()

    def pairs(row, col, R, mask):  # sum_d row_i col_j e^(R_i - G_j)
        P = (R[:, :, :, :, None] - G[:, :, :, None, :]).masked_fill(~mask[:, :, None], -math.inf).exp()
        if op == "gdn":
            return row @ col.transpose(-1, -2) * P[..., 0]
        return (row[:, :, :, :, None] * P * col[:, :, :, None, :]).sum(-1)

    B = pairs(Q, K, read, lower)
    end = G[:, :, :, -1:]
    Qs, Ke, gend = Q * read.exp(), K * (end - G).exp(), end[:, :, :, 0].exp()
    if op == "rwkv6":
        B = B + torch.diag_embed((Q * K * u[:, None, None]).sum(-1))
    else:
        b = chunks(beta)
        Ks = K * G.exp()
        M = -pairs(K, K, G, strict) * b.transpose(-1, -2)
        inv = torch.eye(CHUNK, device=dev) + M
        for _ in range(CHUNK.bit_length() - 2):
            M = M @ M
            inv = inv + M @ inv
    S = torch.zeros(N, H, dk, dv, device=dev) if initial_state is None else initial_state
    out = []
    for c in range(nc):
        X = V[:, :, c]
        if op != "rwkv6":
            X = b[:, :, c] * (inv[:, :, c] @ (X - Ks[:, :, c] @ S))
        out.append(Qs[:, :, c] @ S + B[:, :, c] @ X)
        S = gend[:, :, c, :, None] * S + Ke[:, :, c].transpose(-1, -2) @ X
    o = torch.stack(out, 2).reshape(N, H, L, dv).transpose(1, 2).reshape(N * L, H, dv)
    token = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu[1:], token, right=True)
    return o[seq * L + token - cu[seq]].to(dtype).reshape(shape), S


def _plain_gated_norm(o, gate, weight):
    o32, g32 = o.float(), gate.float()
    y = o32 * (o32.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight
    return (y * g32 / (1 + (-g32).exp())).to(gate.dtype)


def _plain_residual_norm(x, y, scale, weight):
    y32 = y.float()
    x = x + (y32 if scale is None else y32 * scale)
    h = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x, (h if weight is None else h * weight).to(y.dtype)


# ----------------------------------------------------------------- one pass --

def run(state):
    if own:
        import recurrent_state_update_amd as rsu
    kind, train = state["kind"], state["train"]

    def leaf(x):
        return x.detach().requires_grad_(True) if train and x is not None else x

    if kind == "scan":
        x = {n: leaf(t) for n, t in state["in"].items()}
        if own:
            o, s = rsu.scan(state["op"], x["q"], x["k"], x["v"], x["beta"], x["log_decay"], u=x["u"],
                            initial_state=x["initial_state"], cu_seqlens=state["cu"])
        else:
            o, s = _plain_scan(state["op"], state["lens"], state["cu"], **x)
        out, cot = dict(o=o, state=s), None if not train else [state["do"], state["ds"]]
    elif kind == "gated":
        x = {n: leaf(state[n]) for n in ("o", "gate", "weight")}
        y = rsu.gated_norm(x["o"], x["gate"], x["weight"], eps=EPS) if own else _plain_gated_norm(**x)
        out, cot = dict(y=y), None if not train else [state["dy"]]
    else:
        x = {n: leaf(state[n]) for n in ("x", "y", "scale", "weight")}
        xn, h = (rsu.residual_norm(x["x"], x["y"], x["scale"], x["weight"], eps=EPS) if own
                 else _plain_residual_norm(**x))
        out, cot = dict(x=xn, h=h), None if not train else [state["dx"], state["dh"]]
    if train:
        wrt = {n: t for n, t in x.items() if t is not None}
        grads = torch.autograd.grad(list(out.values()), list(wrt.values()), cot)
        out.update(("d" + n, g) for n, g in zip(wrt, grads))
    return {n: t.detach() for n, t in out.items()}


# -------------------------------------------------------------- in 64 bits --

def exact(case, seed):
    st = prepare(case, seed)

    def f64(x):
        return None if x is None else x.double()

    if case["kind"] == "gated":
        o, g, w = f64(st["o"]), f64(st["gate"]), f64(st["weight"])
        r = 1 / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS)
        sig = torch.sigmoid(g)
        out = dict(y=o * r * w * g * sig)
        if case["train"]:
            dy = f64(st["dy"])
            dn = dy * g * sig * w  # cotangent of the normalised o
            out["do"] = r * (dn - o * r * (dn * o * r).mean(-1, keepdim=True))
            out["dgate"] = dy * o * r * w * sig * (1 + g * (1 - sig))
            out["dweight"] = (dy * o * r * g * sig).sum((0, 1))
        return out
    if case["kind"] == "residual":
        x, y, s, w = f64(st["x"]), f64(st["y"]), f64(st["scale"]), f64(st["weight"])
        s1, w1 = (1.0 if t is None else t for t in (s, w))
        x = x + y * s1
        r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        out = dict(x=x, h=x * r * w1)
        if case["train"]:
            dh = f64(st["dh"])
            dn = dh * w1
            d = f64(st["dx"]) + r * (dn - x * r * (dn * x * r).mean(-1, keepdim=True))
            out.update(dx=d, dy=d * s1)
            if s is not None:
                out["dscale"] = (d * y).sum(0)
            if w is not None:
                out["dweight"] = (dh * x * r).sum(0)
        return out
    return _exact_scan(case, st)


def _exact_scan(case, st):
    """Token by token, all sequences abreast; the adjoint token by token too."""
    lens, H, dk, dv = st["lens"], case["H"], case["dk"], case["dv"]
    N, L, delta = len(lens), max(lens), case["op"] != "rwkv6"
    if L * N * H * dk * dv * 8 > 60e9:
        return None  # its states would not fit
    start = [sum(lens[:i]) for i in range(N)]
    T, x = sum(lens), st["in"]

    def spread(t, w):  # [.., H, w] -> [L, N, H, w]
        z = torch.zeros(L, N, H, w, dtype=torch.float64, device=x["q"].device)
        if t is not None:
            t = t.reshape(T, H, w).double()
            for n in range(N):
                z[:lens[n], n] = t[start[n]:start[n] + lens[n]]
        return z

    def gather(z, like):
        z = torch.cat([z[:lens[n], n] for n in range(N)])
        return z.reshape(like.shape)

    q, k, v, beta = spread(x["q"], dk), spread(x["k"], dk), spread(x["v"], dv), spread(x["beta"], 1)
    D = spread(x["log_decay"], 1 if case["op"] == "gdn" else dk).exp().unsqueeze(-1)  # 1 behind the end
    u = x["u"].double() if x["u"] is not None else 0.0
    X = torch.zeros(N, H, dk, dv, dtype=torch.float64, device=q.device)
    if x["initial_state"] is not None:
        X = x["initial_state"].double()
    states, o = [X], torch.empty(L, N, H, dv, dtype=torch.float64, device=q.device)
    qc, kc = q.unsqueeze(-1), k.unsqueeze(-1)

    def read(S, c):  # S^T c
        return (S * c).sum(-2)

    for t in range(L):
        if delta:
            X = D[t] * X
            X = X + kc[t] * (beta[t] * (v[t] - read(X, kc[t]))).unsqueeze(-2)
            o[t] = read(X, qc[t])
        else:
            o[t] = read(X, qc[t]) + (q[t] * u * k[t]).sum(-1, keepdim=True) * v[t]
            X = D[t] * X + kc[t] * v[t].unsqueeze(-2)
        if case["train"]:
            states.append(X)
    out = dict(o=gather(o, x["v"]), state=X)
    if not case["train"]:
        return out
    do = spread(st["do"], dv)
    Y = st["ds"].double()
    dq, dk_, dv_, dbeta = (torch.zeros_like(t) for t in (q, k, v, beta))
    dld = torch.zeros_like(D[..., 0])
    du = torch.zeros(N, H, dk, dtype=torch.float64, device=q.device)
    for t in reversed(range(L)):
        g, before, after = do[t].unsqueeze(-2), states[t], states[t + 1]
        if delta:
            Xd = D[t] * before
            e = v[t] - read(Xd, kc[t])
            dq[t] = (after * g).sum(-1)
            Y = Y + qc[t] * g
            db = read(Y, kc[t])
            de = beta[t] * db
            dbeta[t] = (db * e).sum(-1, keepdim=True)
            dv_[t] = de
            dk_[t] = (Y * (beta[t] * e).unsqueeze(-2)).sum(-1) - (Xd * de.unsqueeze(-2)).sum(-1)
            Y = Y - kc[t] * de.unsqueeze(-2)
            moved = (Y * Xd).sum(-1)
            Y = D[t] * Y
        else:
            s, gv = (q[t] * u * k[t]).sum(-1, keepdim=True), (do[t] * v[t]).sum(-1, keepdim=True)
            dq[t] = (before * g).sum(-1) + gv * u * k[t]
            dk_[t] = (Y * v[t].unsqueeze(-2)).sum(-1) + gv * u * q[t]
            dv_[t] = read(Y, kc[t]) + s * do[t]
            du += gv * q[t] * k[t]
            moved = (Y * D[t] * before).sum(-1)
            Y = D[t] * Y + qc[t] * g
        dld[t] = moved if dld.shape[-1] == dk and case["op"] != "gdn" else moved.sum(-1, keepdim=True)
    out.update(dq=gather(dq, x["q"]), dk=gather(dk_, x["k"]), dv=gather(dv_, x["v"]),
               dlog_decay=gather(dld, x["log_decay"]))
    if delta:
        out["dbeta"] = gather(dbeta, x["beta"])
    else:
        out["du"] = du.sum(0)
    if x["initial_state"] is not None:
        out["dinitial_state"] = Y
    return out
