"""GPU checks of the sequence scan (dl_scan, dl_scan_backward) against the
recurrence in 64 bits, token by token, and its autograd gradients.

Tolerances, as |x - ref| / |ref| in the 2-norm per output.  All sums are in
fp32 (a rounding is at most 2^-24 of its value) over at most d_k + 64 + d_v <=
320 products in a chunk; independent roundings of a sum of n terms leave about
sqrt(n) 2^-24 of it, 18 x 6e-8 = 1.1e-6, and an output passes through at most
six such sums in a row (K~S, N, b, the state, its adjoint, the gradient), sqrt(6)
of that: 2.6e-6.  FP32 is four times this, for outputs whose terms partly
cancel.  The log-decay's gradient is a difference of sums that mostly cancel:
ten times FP32.  A bf16 output adds its own rounding, at most 2^-8 of each
value."""
import pytest
import torch

from sequence_ref import f64, far, scan_ref

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")

FP32 = 1.1e-5
LD = 10 * FP32
BF16 = 2.0 ** -8


def tol(name, dtype):
    if name in ("o", "dq", "dk", "dv") and dtype == torch.bfloat16:
        return BF16 + FP32
    return LD if name == "dlog_decay" else FP32


def inputs(op, lens, H, dk, dv, dtype, seed=0, tail=0, init=True, decay=None, unit=True):
    """Packed inputs (with `tail` rows behind the last sequence) and cotangents."""
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens) + tail, len(lens)

    def normal(*s):
        return torch.randn(*s, generator=g)
    q, k, v = normal(T, H, dk), normal(T, H, dk), normal(T, H, dv)
    if unit and op != "rwkv6":
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    ld = -torch.nn.functional.softplus(normal(*((T, H) if op == "gdn" else (T, H, dk))) * 0.5 - 3)
    if op == "rwkv6":
        ld = -torch.exp(normal(T, H, dk) * 0.5 - 0.5)
    x = dict(q=q.to(dtype), k=k.to(dtype), v=v.to(dtype),
             beta=None if op == "rwkv6" else torch.sigmoid(normal(T, H)), log_decay=ld,
             u=normal(H, dk) * 0.5 if op == "rwkv6" else None,
             initial_state=normal(N, H, dk, dv) * 0.3 if init else None)
    if decay is not None:
        x["log_decay"] = decay(ld, g)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    do, ds = normal(T, H, dv).to(dtype), normal(N, H, dk, dv)
    do[cu[-1]:] = 0 if not tail else 7  # rows of no sequence take no part
    return x, cu, do, ds


def gpu_run(op, x, cu, do, ds, grad=True):
    import recurrent_state_update_amd as rsu
    x = {n: None if t is None else t.cuda().requires_grad_(grad) for n, t in x.items()}
    cu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, s = rsu.scan(op, x["q"], x["k"], x["v"], x["beta"], x["log_decay"], u=x["u"],
                    initial_state=x["initial_state"], cu_seqlens=cu)
    out = dict(o=o, state=s)
    if grad:
        wrt = {n: t for n, t in x.items() if t is not None}
        got = torch.autograd.grad([o, s], list(wrt.values()), [do.cuda(), ds.cuda()])
        out.update(("d" + n, t) for n, t in zip(wrt, got))
    return out


def ref_run(op, x, cu, do, ds):
    x = {n: f64(t) for n, t in x.items()}
    o, s = scan_ref(op, x["q"], x["k"], x["v"], x["beta"], x["log_decay"], x["u"], x["initial_state"], cu)
    out = dict(o=o, state=s)
    wrt = {n: t for n, t in x.items() if t is not None}
    keep = torch.zeros_like(o)
    keep[cu[0]:cu[-1]] = 1
    cot = [(y, c) for y, c in ((o, f64(do, False) * keep), (s, f64(ds, False))) if y.requires_grad]
    got = torch.autograd.grad([y for y, _ in cot], list(wrt.values()), [c for _, c in cot],
                              allow_unused=True) if cot else [None] * len(wrt)
    out.update(("d" + n, torch.zeros_like(wrt[n]) if t is None else t) for n, t in zip(wrt, got))
    return out


def compare(op, x, cu, do, ds, dtype):
    got, want = gpu_run(op, x, cu, do, ds), ref_run(op, x, cu, do, ds)
    assert set(got) == set(want)
    errs = {n: far(got[n], want[n]) for n in want}
    print(f"[scan {op}] " + " ".join(f"{n}={e:.1e}" for n, e in errs.items()), flush=True)
    bad = {n: e for n, e in errs.items() if not e <= tol(n, dtype)}
    assert not bad, bad
    return got


OPS = ["gdn", "kda", "rwkv6"]


@needs_gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 64), (64, 32), (128, 128), (128, 16), (16, 128)])
def test_dims(op, dtype, dk, dv):
    x, cu, do, ds = inputs(op, [100], 2, dk, dv, dtype, seed=dk + dv)
    compare(op, x, cu, do, ds, dtype)


@needs_gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63], [64], [65], [128], [129], [200],
                                  [0], [0, 0], [1, 1, 1], [0, 64, 0, 1, 63, 65, 0], [130, 3, 0, 77]],
                         ids=lambda v: "-".join(map(str, v)))
def test_lengths(op, lens):
    x, cu, do, ds = inputs(op, lens, 3, 32, 32, torch.float32, seed=sum(lens) + len(lens))
    compare(op, x, cu, do, ds, torch.float32)


@needs_gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dk,dv,n", [(16, 32, 20), (128, 32, 20), (64, 64, 10), (32, 128, 5)])
def test_many_sequences_and_heads(op, dtype, dk, dv, n):
    """More 16-column tiles than the GPU has CUs twice over (n 13 dv / 16 =
    520): tiles of 32."""
    lens = [65, 0, 1, 130, 64, 17, 3, 70, 0, 90][:n] * (n // 10 or 1)
    x, cu, do, ds = inputs(op, lens, 13, dk, dv, dtype, seed=n, tail=3)
    compare(op, x, cu, do, ds, dtype)


@needs_gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lens,H,dk,dv,tail,weak", [
    ([2700], 1, 128, 128, 0, True),  # segments of 5 chunks, the last one of 3 with 12 tokens at its end
    ([2700], 3, 16, 32, 0, False),
    ([2562, 0, 130, 5100, 1], 2, 64, 16, 5200, True),  # several, one and no segment; rows behind
], ids=["one", "heads", "packed"])
def test_long_sequences_with_few_heads(op, dtype, lens, H, dk, dv, tail, weak):
    """Sequences cut into segments and joined; weakly decaying, the state of
    the first tokens reaches the last."""
    x, cu, do, ds = inputs(op, lens, H, dk, dv, dtype, seed=H, tail=tail, decay=(lambda ld, g: ld * 0.004) if weak else None)
    if weak and op == "rwkv6":
        x["v"] = x["v"] / 8  # its state is a plain sum
    compare(op, x, cu, do, ds, dtype)


@needs_gpu
@pytest.mark.parametrize("op", OPS)
def test_long_prompt_in_place(op):
    """The end state of a cut sequence over the initial one (prefill), against
    tensors of their own, twice on."""
    import recurrent_state_update_amd as rsu
    x = {n: None if t is None else t.cuda() for n, t in inputs(op, [3000, 2700], 2, 32, 32, torch.bfloat16, seed=9)[0].items()}
    cu = torch.tensor([0, 3000, 5700], dtype=torch.int32, device="cuda")
    a = tuple(x[n] for n in ("q", "k", "v", "beta", "log_decay"))
    st = rsu.DeltaLogState(op, 2, 2, 32, 32, 4, dtype=torch.bfloat16, base=x["initial_state"].clone(), u=x["u"])
    s = x["initial_state"]
    for _ in range(3):
        o = st.prefill(*a, cu_seqlens=cu)
        want, s = rsu.scan(op, *a, u=x["u"], initial_state=s, cu_seqlens=cu)
        assert torch.equal(o, want) and torch.equal(st.base, s)
    st.close()


@needs_gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("lens,tail", [([5, 70], 3), ([64], 64), ([0], 130), ([33, 31], 200)])
def test_rows_behind_the_last_sequence(op, lens, tail):
    x, cu, do, ds = inputs(op, lens, 2, 16, 32, torch.float32, tail=tail)
    got = compare(op, x, cu, do, ds, torch.float32)
    for n in ("o", "dq", "dk", "dv", "dlog_decay") + (("dbeta",) if op != "rwkv6" else ()):
        assert not got[n][cu[-1]:].any(), n


@needs_gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("kind", ["erase", "erase often", "none", "strong", "very strong", "mixed"])
def test_decays(op, kind):
    """-inf (full forgetting), 0, and decays whose products underflow within a
    few rows: nothing overflows and nothing is lost."""
    def decay(ld, g):
        r = torch.rand(ld.shape, generator=g)
        if kind == "erase":
            return torch.where(r < 0.02, -torch.inf, ld)
        if kind == "erase often":
            return torch.where(r < 0.5, -torch.inf, ld)
        if kind == "none":
            return torch.zeros_like(ld)
        if kind == "strong":
            return -5 * r
        if kind == "very strong":
            return -60 * r
        return torch.where(r < 0.3, -40 * r, torch.where(r < 0.6, torch.zeros_like(ld), ld))
    x, cu, do, ds = inputs(op, [150, 20], 2, 32, 32, torch.float32, seed=5, decay=decay)
    compare(op, x, cu, do, ds, torch.float32)


@needs_gpu
@pytest.mark.parametrize("op", ["gdn", "kda"])
@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0, "zero or one"])
def test_beta(op, beta):
    x, cu, do, ds = inputs(op, [140], 2, 64, 32, torch.float32, seed=8)
    g = torch.Generator().manual_seed(1)
    x["beta"] = (torch.rand(x["beta"].shape, generator=g) < 0.5).float() if isinstance(beta, str) \
        else torch.full_like(x["beta"], beta)
    compare(op, x, cu, do, ds, torch.float32)


@needs_gpu
@pytest.mark.parametrize("op", ["gdn", "kda"])
def test_repeated_key(op):
    """The same key over and over: the strongest coupling within a chunk."""
    x, cu, do, ds = inputs(op, [130], 2, 32, 32, torch.float32, seed=9)
    x["k"] = x["k"][:1].expand_as(x["k"]).contiguous()
    compare(op, x, cu, do, ds, torch.float32)


@needs_gpu
@pytest.mark.parametrize("op", OPS)
def test_scales(op):
    """Values far from one: q, v and the cotangents large and small."""
    x, cu, do, ds = inputs(op, [90], 2, 32, 32, torch.float32, seed=10)
    x["q"] = x["q"] * 1e6
    x["v"] = x["v"] * 1e-9
    x["initial_state"] = x["initial_state"] * 1e-9
    compare(op, x, cu, do * 1e-12, ds * 1e-6, torch.float32)


@needs_gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_slices_of_a_projection_and_batches(op, dtype):
    """q, k, v as slices of one projection, off any vector alignment, packed
    or [N,T,H,d]: the same results as from contiguous copies, bit for bit."""
    import recurrent_state_update_amd as rsu
    N, T, H, dk, dv = 3, 70, 2, 16, 32
    x, cu, do, ds = inputs(op, [T] * N, H, dk, dv, dtype, seed=3)
    want = gpu_run(op, x, cu, do, ds)
    p = torch.full((N * T, 1 + H * (2 * dk + dv) + 2), 9.0, dtype=dtype, device="cuda")
    w = [H * dk, H * dk, H * dv]
    views = p[:, 1:-2].split(w, dim=1)
    for view, n in zip(views, "qkv"):
        view.copy_(x[n].reshape(N * T, -1))
    def small(n):
        return None if x[n] is None else x[n].cuda()
    q, k, v = (view.unflatten(1, (H, -1)) for view in views)
    a = (small("beta"), small("log_decay"))
    for batched in (False, True):
        if batched:
            q, k, v = (t.unflatten(0, (N, T)) for t in (q, k, v))
            a = tuple(None if t is None else t.unflatten(0, (N, T)) for t in a)
        assert not q.is_contiguous()
        o, s = rsu.scan(op, q, k, v, *a, u=small("u"), initial_state=small("initial_state"),
                        cu_seqlens=None if batched else torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert torch.equal(o.reshape(N * T, H, dv), want["o"]) and torch.equal(s, want["state"])


@needs_gpu
@pytest.mark.parametrize("op", OPS)
def test_long_and_repeatable(op):
    """A longer run in bf16, twice: within tolerance and bit-identical (no
    result depends on timing)."""
    x, cu, do, ds = inputs(op, [700, 333], 4, 64, 64, torch.bfloat16, seed=4)
    a = compare(op, x, cu, do, ds, torch.bfloat16)
    b = gpu_run(op, x, cu, do, ds)
    for n in a:
        assert torch.equal(a[n], b[n]), n


@needs_gpu
@pytest.mark.parametrize("op", OPS)
def test_gradients_against_differences(op):
    """<gradient, direction> against a central difference of the kernel's own
    forward pass in fp32.  Step 1e-2: its cubic term is below 1e-3 of the
    slope for these inputs of order one, and the rounding of the two losses
    (1e-6 of their parts) over the step below 1e-3: 1e-2 in all."""
    import recurrent_state_update_amd as rsu
    x, cu, do, ds = inputs(op, [90, 40], 2, 16, 16, torch.float32, seed=6)
    got = gpu_run(op, x, cu, do, ds)
    g = torch.Generator().manual_seed(2)
    cuda = {n: None if t is None else t.cuda() for n, t in x.items()}
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def loss(y):
        o, s = rsu.scan(op, y["q"], y["k"], y["v"], y["beta"], y["log_decay"], u=y["u"],
                        initial_state=y["initial_state"], cu_seqlens=cut)
        return float((o.double() * do.cuda()).sum() + (s.double() * ds.cuda()).sum())
    for n, t in x.items():
        if t is None:
            continue
        slope = got["d" + n].double().cpu()
        way = slope / slope.norm() + 0.3 * torch.randn(t.shape, generator=g).double() / t.numel() ** 0.5
        h = 1e-2
        ways = [loss({**cuda, n: (cuda[n].double() + f * h * way.cuda()).float()}) for f in (1, -1)]
        num, ana = (ways[0] - ways[1]) / (2 * h), float((slope * way).sum())
        print(f"[scan {op}] d{n}: difference {num:.6g} gradient {ana:.6g}", flush=True)
        assert abs(num - ana) <= 1e-2 * abs(ana), n


@needs_gpu
@pytest.mark.parametrize("op", OPS)
def test_parts_of_the_gradient(op):
    """One cotangent only, or inputs that need none."""
    import recurrent_state_update_amd as rsu
    x, cu, do, ds = inputs(op, [80], 2, 16, 16, torch.float32, seed=7, init=False)
    both = gpu_run(op, x, cu, do, ds)
    c = {n: None if t is None else t.cuda() for n, t in x.items()}
    sums = []
    for first in (True, False):
        k = c["k"].clone().requires_grad_(True)
        o, s = rsu.scan(op, c["q"], k, c["v"], c["beta"], c["log_decay"], u=c["u"])
        (g,) = torch.autograd.grad(o if first else s, k, (do if first else ds).cuda())
        sums.append(g)
    assert far(sums[0] + sums[1], both["dk"].double().cpu()) <= 2 * FP32


@needs_gpu
@pytest.mark.parametrize("op", OPS)
def test_against_the_decode_step(op):
    """prefill, then decode steps, against one scan over all tokens; named
    slots of a per-slot state; a second prompt behind the first."""
    import recurrent_state_update_amd as rsu
    B, H, d, L, more = 3, 2, 32, 77, 6
    x, cu, _, _ = inputs(op, [L + more] * B, H, d, d, torch.float32, seed=12)
    c = {n: None if t is None else t.cuda() for n, t in x.items()}

    def at(n, lo, hi):
        return None if c[n] is None else c[n].unflatten(0, (B, L + more))[:, lo:hi].contiguous()
    names = ("q", "k", "v", "beta", "log_decay")
    whole, end = rsu.scan(op, *(at(n, 0, L + more) for n in names), u=c["u"], initial_state=c["initial_state"])
    for per_slot in (False, True):
        st = rsu.DeltaLogState(op, B, H, d, d, 4, dtype=torch.float32, base=c["initial_state"].clone(), u=c["u"])
        if per_slot:
            st.enable_slots()
            order = [2, 0, 1]
            parts = [at(n, 0, 40) for n in names]
            o1 = st.prefill(*(None if p is None else p[order].contiguous() for p in parts), slots=order)
            o1 = o1[[1, 2, 0]]
            o = torch.cat([o1, st.prefill(*(at(n, 40, L) for n in names))], dim=1)
        else:
            o = st.prefill(*(at(n, 0, L) for n in names))
        assert far(o, whole[:, :L].double().cpu()) <= FP32
        for t in range(L, L + more):
            step = st.step(*(None if c[n] is None else at(n, t, t + 1).squeeze(1) for n in names))
            assert far(step, whole[:, t].double().cpu()) <= 2 * FP32
        with pytest.raises(ValueError):
            st.prefill(*(at(n, 0, L) for n in names))  # entries pending (6 steps at M = 4)
        st.merge()
        assert far(st.base, end.double().cpu()) <= 2 * FP32
        st.close()


@needs_gpu
@pytest.mark.parametrize("op", OPS)
def test_graph_replays(op):
    """Forward and backward captured in a graph, replayed on new inputs with
    other work in between, against eager calls: bit for bit."""
    import recurrent_state_update_amd as rsu
    sets = [inputs(op, [70, 30], 2, 16, 32, torch.float32, seed=s) for s in range(4)]
    cu = torch.tensor(sets[0][1], dtype=torch.int32, device="cuda")
    x = {n: None if t is None else t.cuda().requires_grad_(True) for n, t in sets[0][0].items()}
    do, ds = sets[0][2].cuda(), sets[0][3].cuda()
    wrt = [t for t in x.values() if t is not None]

    def step():
        o, s = rsu.scan(op, x["q"], x["k"], x["v"], x["beta"], x["log_decay"], u=x["u"],
                        initial_state=x["initial_state"], cu_seqlens=cu)
        return [o, s, *torch.autograd.grad([o, s], wrt, [do, ds])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [t.detach() for t in step()]
    junk = torch.randn(256, 256, device="cuda")
    for new, _, ndo, nds in sets[1:] + sets[:1]:
        with torch.no_grad():
            for n, t in new.items():
                if t is not None:
                    x[n].copy_(t)
            do.copy_(ndo)
            ds.copy_(nds)
        g.replay()
        got = [t.clone() for t in outs]
        junk = (junk @ junk).tanh_()
        torch.cuda.synchronize()
        want = gpu_run(op, new, sets[0][1], ndo, nds)
        assert all(torch.equal(a, b) for a, b in zip(got, want.values()))


@needs_gpu
def test_long_sequence_in_a_graph():
    """Segments in a captured training step, replayed on new inputs among other
    work, against eager calls: bit for bit."""
    import recurrent_state_update_amd as rsu
    sets = [inputs("gdn", [2700], 2, 32, 32, torch.bfloat16, seed=s) for s in range(3)]
    x = {n: t.cuda().requires_grad_(True) for n, t in sets[0][0].items() if t is not None}
    do, ds = sets[0][2].cuda(), sets[0][3].cuda()

    def step():
        o, s = rsu.scan("gdn", x["q"], x["k"], x["v"], x["beta"], x["log_decay"], initial_state=x["initial_state"])
        return [o, s, *torch.autograd.grad([o, s], list(x.values()), [do, ds])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [t.detach() for t in step()]
    for new, cu, ndo, nds in sets[1:] + sets[:1]:
        with torch.no_grad():
            for n, t in x.items():
                t.copy_(new[n])
            do.copy_(ndo)
            ds.copy_(nds)
        g.replay()
        got = [t.clone() for t in outs]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, gpu_run("gdn", new, cu, ndo, nds).values()))


@needs_gpu
def test_prefill_in_a_graph():
    """Prompts continued by replays, against eager calls; a list of slots is
    refused there, and the capture goes on."""
    import recurrent_state_update_amd as rsu
    x = {n: None if t is None else t.cuda() for n, t in inputs("kda", [70, 30], 2, 16, 32, torch.float32)[0].items()}
    a = tuple(x[n] for n in ("q", "k", "v", "beta", "log_decay"))
    cu = torch.tensor([0, 70, 100], dtype=torch.int32, device="cuda")
    st, other = (rsu.DeltaLogState("kda", 2, 2, 16, 32, 4, dtype=torch.float32) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        st.prefill(*a, cu_seqlens=cu)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(ValueError):
            st.prefill(*a, cu_seqlens=cu, slots=[1, 0])
        o = st.prefill(*a, cu_seqlens=cu)
    other.prefill(*a, cu_seqlens=cu)
    for _ in range(3):
        g.replay()
        want = other.prefill(*a, cu_seqlens=cu)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(st.base, other.base)
    st.close()
    other.close()


@needs_gpu
def test_another_stream_and_two_at_once():
    """Calls on streams of their own, at the same time, each with a workspace
    of its own: as alone."""
    import recurrent_state_update_amd as rsu
    runs = [inputs(op, [300], 4, 64, 64, torch.bfloat16, seed=20 + i) for i, op in enumerate(OPS)]
    alone = [gpu_run(op, *r, grad=False) for op, r in zip(OPS, runs)]
    cuda = [{n: None if t is None else t.cuda() for n, t in r[0].items()} for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in OPS]
    outs = []
    for op, x, s in zip(OPS, cuda, streams):
        outs.append(rsu.scan(op, x["q"], x["k"], x["v"], x["beta"], x["log_decay"], u=x["u"],
                             initial_state=x["initial_state"], stream=s))
    torch.cuda.synchronize()
    for (o, s), a in zip(outs, alone):
        assert torch.equal(o, a["o"]) and torch.equal(s, a["state"])


@needs_gpu
def test_refusals():
    """Shapes, types, devices and layouts that the entry point names."""
    import recurrent_state_update_amd as rsu
    c = {n: None if t is None else t.cuda() for n, t in inputs("gdn", [20, 12], 2, 16, 32, torch.float32)[0].items()}
    cu = torch.tensor([0, 20, 32], dtype=torch.int32, device="cuda")

    def call(op="gdn", cu_seqlens=cu, **kw):
        x = {**c, **kw}
        return rsu.scan(op, x["q"], x["k"], x["v"], x["beta"], x["log_decay"], u=x["u"],
                        initial_state=x["initial_state"], cu_seqlens=cu_seqlens)
    call()
    bad = [dict(op="gla"), dict(op="rwkv6"), dict(op="kda"), dict(q=c["q"].half()), dict(k=c["k"][:, :1]),
           dict(k=c["k"].bfloat16()), dict(v=c["v"][:31]), dict(v=c["v"][..., :24]), dict(beta=None),
           dict(beta=c["beta"].double()), dict(log_decay=c["log_decay"][:, :1]), dict(u=c["q"][0]),
           dict(initial_state=c["initial_state"][:1]), dict(initial_state=c["initial_state"].bfloat16()),
           dict(beta=c["beta"].cpu()), dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu.cpu()), dict(cu_seqlens=cu[:1]),
           dict(cu_seqlens=None), dict(q=c["q"][0]), dict(q=c["q"][..., :8].repeat(1, 1, 3), k=c["k"][..., :8].repeat(1, 1, 3))]
    for kw in bad:
        with pytest.raises(ValueError):
            call(**kw)
    st = rsu.DeltaLogState("gdn", 3, 2, 16, 32, 4, dtype=torch.float32)
    a = tuple(c[n] for n in ("q", "k", "v", "beta", "log_decay"))
    for slots in (None, [0], [0, 0], [0, 3], [-1, 0]):
        with pytest.raises(ValueError):
            st.prefill(*a, cu_seqlens=cu, slots=slots)
    with pytest.raises(ValueError):
        st.prefill(a[0].bfloat16(), a[1].bfloat16(), a[2].bfloat16(), *a[3:], cu_seqlens=cu, slots=[0, 1])
    st.prefill(*a, cu_seqlens=cu, slots=[2, 0])
    assert not st.base[1].any() and st.base[0].any() and st.base[2].any()
    st.close()


@needs_gpu
@pytest.mark.parametrize("op", OPS)
def test_bad_offsets_stay_in_range(op):
    """Offsets out of order or out of range: meaningless results, no access
    outside the tensors (guard rows around every output keep their values)."""
    import recurrent_state_update_amd as rsu
    T, H, d = 100, 2, 32
    x = {n: None if t is None else t.cuda() for n, t in inputs(op, [T], H, d, d, torch.float32, init=False)[0].items()}
    for cu in ([0, 70, 30, 100], [0, 200, 300, 400], [-50, -20, 40, 1 << 30], [100, 0, 0, 0], [0, 0, 0, 0]):
        cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o = torch.full((T + 2, H, d), 5.0, device="cuda")
        fin = torch.full((3 + 2, H, d, d), 5.0, device="cuda")
        p = {n: None if t is None else t.data_ptr() for n, t in x.items()}
        desc = rsu.dl_scan_desc(rsu.OPS[op], 0, T, 3, H, d, d, 0, 0, 0, cut.data_ptr(), p["q"], p["k"], p["v"], p["beta"],
                                p["log_decay"], p["u"])
        n = rsu.dl_scan_workspace_bytes(desc)
        ws = torch.full((n + 512,), 7, dtype=torch.uint8, device="cuda")
        assert rsu.dl_scan(desc, None, fin[1], None, 0, o[1], None, ws) == 0
        torch.cuda.synchronize()
        assert (o[0] == 5).all() and (o[-1] == 5).all() and (fin[0] == 5).all() and (fin[-1] == 5).all()
        assert (ws[n:] == 7).all()


@needs_gpu
@pytest.mark.parametrize("op", OPS)
def test_state_rows_and_null_outputs(op):
    """State rows by index, some out of range; no end state; no initial one."""
    import recurrent_state_update_amd as rsu
    H, d = 2, 32
    x, cu, _, _ = inputs(op, [40, 30, 20], H, d, d, torch.float32, init=False)
    c = {n: None if t is None else t.cuda() for n, t in x.items()}
    want = gpu_run(op, x, cu, None, None, grad=False)
    p = {n: None if t is None else t.data_ptr() for n, t in c.items()}
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    desc = rsu.dl_scan_desc(rsu.OPS[op], 0, 90, 3, H, d, d, 0, 0, 0, cut.data_ptr(), p["q"], p["k"], p["v"], p["beta"],
                            p["log_decay"], p["u"])
    ws = torch.empty(rsu.dl_scan_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    o = torch.empty(90, H, d, device="cuda")
    base = torch.zeros(4, H, d, d, device="cuda")
    rows = torch.tensor([3, 9, 0], dtype=torch.int32, device="cuda")
    assert rsu.dl_scan(desc, base, base, rows, 4, o, None, ws) == 0
    assert torch.equal(o, want["o"])
    assert torch.equal(base[3], want["state"][0]) and torch.equal(base[0], want["state"][2])
    assert not base[1:3].any()
    o.zero_()
    assert rsu.dl_scan(desc, None, None, None, 0, o, None, ws) == 0
    assert torch.equal(o, want["o"])


@needs_gpu
@pytest.mark.parametrize("op", OPS)
def test_nan_stays_in_its_sequence_and_head(op):
    x, cu, _, _ = inputs(op, [70, 50], 3, 16, 16, torch.float32)
    want = gpu_run(op, x, cu, None, None, grad=False)
    for n in ("q", "k", "v", "log_decay"):
        y = {m: None if t is None else t.clone() for m, t in x.items()}
        y[n][80, 1] = float("nan")
        got = gpu_run(op, y, cu, None, None, grad=False)
        assert torch.equal(got["o"][:70], want["o"][:70]) and torch.equal(got["o"][:, [0, 2]], want["o"][:, [0, 2]])
        assert torch.equal(got["state"][0], want["state"][0]) and torch.equal(got["state"][1][[0, 2]], want["state"][1][[0, 2]])
        # RWKV6 reads the state before the token's own decay
        row = 81 if (op, n) == ("rwkv6", "log_decay") else 80
        assert not torch.isfinite(got["o"][row, 1]).all()
