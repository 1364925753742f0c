"""GPU checks of short_conv and short_conv_step against the convolution in 64 bits
and its gradients, element by element.

Tolerances, in roundings of 32 bits (2^-24) of the sum of the absolute values of an
output's terms (layer_ref.within): a sum of up to five terms, an exponential good to
2, a quotient, and what follows them: 20; ds, which the gradients are sums of, takes
two more products: 30; sums over a run of up to 128 tokens in fp32, in 64 bits
beyond: 160.  (A bf16 output adds its own rounding.)"""
import pytest
import torch

from layer_ref import check, conv_ref, offsets

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
UNITS = dict(y=20, end=0, dx=30, dinitial=30, dweight=160, dbias=160)
NAMES = ("x", "weight", "bias", "initial")


def inputs(lens, C, W, dtype="f32", bias=True, init=True, first=0, tail=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    t, cu = DT[dtype], offsets(lens, first)
    T, N = cu[-1] + tail, len(lens)

    def normal(*s):
        return torch.randn(*s, generator=g)
    x = dict(x=normal(T, C).to(t), weight=normal(C, W), bias=normal(C) if bias else None,
             initial=normal(N, W - 1, C).to(t) if init else None)
    return x, cu, normal(T, C).to(t), normal(N, W - 1, C).to(t)


def run(x, cu, dy=None, dend=None, act=True, batch=None):
    import recurrent_state_update_amd as rsu
    v = {n: None if t is None else t.cuda() for n, t in x.items()}
    if batch:
        v["x"] = v["x"].unflatten(0, batch)
    if dy is not None:
        v = {n: None if t is None else t.requires_grad_(True) for n, t in v.items()}
    off = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, end = rsu.short_conv(v["x"], v["weight"], v["bias"], initial_state=v["initial"], cu_seqlens=off, silu=act)
    out = dict(y=y, end=end)
    if dy is not None:
        wrt = [n for n in NAMES if v[n] is not None]
        out.update(("d" + n, t) for n, t in zip(wrt, torch.autograd.grad(
            [y, end], [v[n] for n in wrt], [dy.cuda().reshape(y.shape), dend.cuda()])))
    return {n: t.flatten(0, 1) if batch and n in ("y", "dx") else t for n, t in out.items()}


def compare(x, cu, dy, dend, got, act=True):
    refs = [conv_ref(*x.values(), cu, act, dy, dend, size=s) for s in (False, True)]
    live = torch.zeros(x["x"].shape[0], 1, dtype=torch.float64)
    live[cu[0]:cu[-1]] = 1
    want = {n: t for n, t in refs[0].items() if n in got}
    assert set(want) == set(got)
    check(got, want, refs[1], UNITS)


def poison(n=1 << 26):
    torch.full((n,), float("nan"), device="cuda")


SHAPES = [
    # lens, channels, taps, first, tail
    ([1], 1, 2, 0, 0),
    ([5], 32, 4, 0, 0),
    ([0, 1, 0, 2, 3, 4, 0], 20, 4, 0, 0),
    ([0, 1, 0, 2, 3, 4, 0], 21, 3, 2, 1),
    ([33, 0, 7], 36, 2, 3, 5),
    ([300], 64, 4, 0, 0),
    ([1, 1, 1, 1, 1, 90], 130, 4, 1, 70),
    ([9] * 30, 12, 3, 0, 0),
    ([0], 16, 4, 0, 0),
    ([0, 0], 8, 4, 0, 3),
    ([2600, 1], 4, 4, 0, 0),
    ([700], 1000, 4, 0, 2),
]


@needs_gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)).replace(" ", "")[:40])
def test_against_64_bits(shape, dtype):
    lens, C, W, first, tail = shape
    x, cu, dy, dend = inputs(lens, C, W, dtype, first=first, tail=tail, seed=C + W)
    poison()
    compare(x, cu, dy, dend, run(x, cu, dy, dend))


@needs_gpu
@pytest.mark.parametrize("without", [("bias",), ("initial",), ("silu",), ("bias", "initial", "silu")], ids="+".join)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_options(without, dtype):
    act = "silu" not in without
    x, cu, dy, dend = inputs([21, 2, 40], 24, 4, dtype, bias="bias" not in without, init="initial" not in without)
    compare(x, cu, dy, dend, run(x, cu, dy, dend, act), act)


@needs_gpu
def test_batch_and_packed_agree():
    x, cu, dy, dend = inputs([37, 37, 37], 20, 4, "bf16")
    a, b = run(x, cu, dy, dend), run(x, None, dy, dend, batch=(3, 37))
    for n in a:
        assert torch.equal(a[n], b[n]), n


@needs_gpu
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_slices(shift):
    """x as a slice of a projection at any alignment, other tensors off a vector's
    boundary: the same results."""
    import recurrent_state_update_amd as rsu
    x, cu, dy, dend = inputs([40, 9], 32, 4, "bf16")
    want = run(x, cu, dy, dend)
    wide = torch.zeros(49, 32 + shift + 3, dtype=torch.bfloat16, device="cuda").requires_grad_(True)
    with torch.no_grad():
        wide[:, shift:shift + 32] = x["x"].cuda()

    def off(t):
        return torch.cat([torch.zeros(shift, dtype=t.dtype), t.reshape(-1)]).cuda()[shift:].view(t.shape)
    init = off(x["initial"]).requires_grad_(True)
    y, end = rsu.short_conv(wide[:, shift:shift + 32], x["weight"].cuda(), x["bias"].cuda(), initial_state=init,
                            cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, want["y"]) and torch.equal(end, want["end"])
    dw, d0 = torch.autograd.grad([y, end], [wide, init], [off(dy), off(dend)])
    assert torch.equal(dw[:, shift:shift + 32], want["dx"]) and torch.equal(d0, want["dinitial"])


@needs_gpu
def test_some_gradients():
    import recurrent_state_update_amd as rsu
    x, cu, dy, dend = inputs([40], 16, 4)
    want = run(x, None, dy, dend)
    for n in NAMES:
        v = {m: t.cuda().requires_grad_(m == n) for m, t in x.items()}
        out = rsu.short_conv(v["x"], v["weight"], v["bias"], initial_state=v["initial"])
        assert torch.equal(torch.autograd.grad(out, v[n], [dy.cuda(), dend.cuda()])[0], want["d" + n]), n
    v = {m: t.cuda().requires_grad_(True) for m, t in x.items()}
    y, end = rsu.short_conv(v["x"], v["weight"], v["bias"], initial_state=v["initial"])
    for out, cot, a, b in ((y, dy, dy, 0 * dend), (end, dend, 0 * dy, dend)):
        got = dict(zip(NAMES, torch.autograd.grad(out, list(v.values()), cot.cuda(), retain_graph=True)))
        alone = run(x, None, a, b)
        for n in NAMES:
            assert torch.equal(got[n], alone["d" + n]), n


@needs_gpu
def test_gradient_against_differences():
    """fp32: as the scan's test of this name."""
    x, cu, dy, dend = inputs([30], 8, 4)
    g = torch.Generator().manual_seed(3)
    grads = run(x, None, dy, dend)

    def loss(v):
        o = run(v, None)
        return float((o["y"].cpu().double() * dy).sum() + (o["end"].cpu().double() * dend).sum())
    for n in NAMES:
        d = torch.randn(x[n].shape, generator=g)
        d /= d.norm()
        h = 2.0 ** -6
        slope = (loss({**x, n: x[n] + h * d}) - loss({**x, n: x[n] - h * d})) / (2 * h)
        want = float((grads["d" + n].cpu().double() * d).sum())
        assert abs(slope - want) <= 0.02 * float(grads["d" + n].norm()) + 1e-3, (n, slope, want)


@needs_gpu
def test_repeatable():
    x, cu, dy, dend = inputs([900, 77], 200, 4, "bf16")
    a, b = run(x, cu, dy, dend), run(x, cu, dy, dend)
    for n in a:
        assert torch.equal(a[n], b[n]), n


@needs_gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_continues_where_it_ended(W, dtype):
    """A sequence in parts of 40, 1 and 2 tokens and then token by token: bit for bit."""
    import recurrent_state_update_amd as rsu
    x, _, _, _ = inputs([60], 20, W, dtype)
    v = {n: t.cuda() for n, t in x.items()}
    args = v["weight"], v["bias"]
    y, end = rsu.short_conv(v["x"], *args, initial_state=v["initial"])
    parts, state, at = [], v["initial"], 0
    for n in (40, 1, 2):
        row, state = rsu.short_conv(v["x"][at:at + n], *args, initial_state=state)
        parts.append(row)
        at += n
    state = state.clone()
    for t in range(at, 60):
        parts.append(rsu.short_conv_step(v["x"][t:t + 1], state, *args))
    assert torch.equal(torch.cat(parts), y) and torch.equal(state, end)


@needs_gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 20, 23])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_step(W, C, dtype):
    """Rows anywhere in the cache, rows outside it, and rows that no token names."""
    import recurrent_state_update_amd as rsu
    rows, S = [3, -1, 10, 0, 11, 7, 1], 11
    known = [0 <= r < S for r in rows]
    x, cu, _, _ = inputs([1] * 7, C, W, dtype, init=False, seed=C)
    g = torch.Generator().manual_seed(W)
    cache = torch.randn(S, W - 1, C, generator=g).to(DT[dtype])
    x["initial"] = torch.stack([cache[r] if k else 0 * cache[0] for r, k in zip(rows, known)])
    refs = [conv_ref(*x.values(), cu, size=s) for s in (False, True)]
    state = cache.cuda()
    y = rsu.short_conv_step(x["x"].cuda(), state, x["weight"].cuda(), x["bias"].cuda(),
                            rows=torch.tensor(rows, dtype=torch.int32, device="cuda"))
    check(dict(y=y), dict(y=refs[0]["y"]), refs[1], UNITS)
    want = cache.clone()
    for i, r in enumerate(rows):
        if known[i]:
            want[r] = refs[0]["end"][i].to(cache.dtype)
    assert torch.equal(state.cpu(), want)
    state = cache.cuda()
    y = rsu.short_conv_step(x["x"].cuda(), state, x["weight"].cuda(), silu=False)
    x.update(initial=cache[:7], bias=None)
    refs = [conv_ref(*x.values(), cu, False, size=s) for s in (False, True)]
    check(dict(y=y, end=state[:7]), refs[0], refs[1], UNITS)
    assert torch.equal(state[7:].cpu(), cache[7:])


@needs_gpu
def test_nan_stays_in_its_sequence_and_channel():
    x, cu, dy, dend = inputs([33, 2, 40], 20, 4, first=3, tail=9)
    clean = run(x, cu, dy, dend)
    x["x"][:3] = x["x"][-9:] = float("nan")  # rows of no sequence take no part
    dy[:3] = dy[-9:] = float("inf")
    dirty = run(x, cu, dy, dend)
    for n in clean:
        assert torch.equal(dirty[n], clean[n]), n
    x["x"][36, 5] = float("nan")  # the second sequence's first token
    dirty = run(x, cu, dy, dend)
    ok = torch.ones(87, 20, dtype=torch.bool)
    ok[36:38, 5] = False
    assert torch.equal(dirty["y"].cpu()[ok], clean["y"].cpu()[ok]) and torch.isnan(dirty["y"][36:38, 5]).all()
    assert torch.equal(dirty["dx"].cpu()[ok], clean["dx"].cpu()[ok])


@needs_gpu
@pytest.mark.parametrize("cu", [[0, 50, 20, 60], [-5, 30, 90, 60], [60, 40, 20, 0], [0, 2 ** 31 - 1, 10, 60],
                                [-2 ** 31, 5, 5, 70]])
def test_bad_offsets_stay_in_range(cu):
    x, _, dy, dend = inputs([20] * 3, 16, 4)
    out = run(x, cu, dy, dend)
    torch.cuda.synchronize()
    assert out["y"].shape == (60, 16)


@needs_gpu
def test_graph_replays():
    """Forward, backward and steps captured in a graph, replayed on new inputs and
    offsets, with eager work between."""
    import recurrent_state_update_amd as rsu
    sets = [inputs([40, 0, 33], 20, 4, "bf16", seed=s) for s in range(4)]
    v = [t.cuda() for t in sets[0][0].values()]
    dy, dend = sets[0][2].cuda(), sets[0][3].cuda()
    cu = torch.tensor(sets[0][1], dtype=torch.int32, device="cuda")

    def step():
        a = [t.detach().requires_grad_(True) for t in v]
        y, end = rsu.short_conv(*a[:3], initial_state=a[3], cu_seqlens=cu)
        state = v[3].clone()
        one = rsu.short_conv_step(v[0][:3], state, v[1], v[2])
        return [y.detach(), end.detach(), one, state, *torch.autograd.grad([y, end], a, [dy, dend])]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for k in range(3):
        x, off, a, b = sets[k + 1]
        for t, new in zip([*v, dy, dend, cu], [*x.values(), a, b, torch.tensor([0, 40 - k, 41 + k, 73], dtype=torch.int32)]):
            t.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for p, q in zip(got, step()):
            assert torch.equal(p, q)


@needs_gpu
def test_streams():
    import recurrent_state_update_amd as rsu
    x, cu, dy, dend = inputs([300], 64, 4)
    want = run(x, cu, dy, dend)
    v = {n: t.cuda().requires_grad_(True) for n, t in x.items()}
    dy, dend = dy.cuda(), dend.cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y, end = rsu.short_conv(v["x"], v["weight"], v["bias"], initial_state=v["initial"], stream=s)
    with torch.cuda.stream(s):
        grads = torch.autograd.grad([y, end], list(v.values()), [dy, dend])
    torch.cuda.synchronize()
    assert torch.equal(y, want["y"]) and torch.equal(end, want["end"])
    for n, t in zip(NAMES, grads):
        assert torch.equal(t, want["d" + n]), n


@needs_gpu
def test_offsets_beyond_32_bits():
    """Rows more than 2^31 elements from the first, both ways and in a step's cache: as
    a call on those rows alone."""
    import recurrent_state_update_amd as rsu
    C, T, L = 16384, 131200, 60
    x, _, dy, dend = inputs([L], C, 4, "bf16", seed=9)
    want = run(x, None, dy, dend)
    v = {n: t.cuda() for n, t in x.items()}
    big = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    big[-L:] = v["x"]
    bdy = torch.zeros_like(big)
    bdy[-L:] = dy.cuda()
    big.requires_grad_(True)
    init = torch.cat([0 * v["initial"], v["initial"]]).requires_grad_(True)
    cu = torch.tensor([0, T - L, T], dtype=torch.int32, device="cuda")
    y, end = rsu.short_conv(big, v["weight"], v["bias"], initial_state=init, cu_seqlens=cu)
    assert torch.equal(y[-L:], want["y"]) and torch.equal(end[1:], want["end"])
    dx, d0 = torch.autograd.grad([y, end], [big, init], [bdy, torch.cat([0 * dend, dend]).cuda()])
    assert torch.equal(dx[-L:], want["dx"]) and torch.equal(d0[1:], want["dinitial"])
    del y, dx, bdy, big
    S = 45000
    assert (S - 1) * 3 * C > 2 ** 31
    cache = torch.zeros(S, 3, C, dtype=torch.bfloat16, device="cuda")
    cache[S - 1] = v["initial"][0]
    one = v["initial"].clone()
    y = rsu.short_conv_step(v["x"][:1], cache, v["weight"], v["bias"],
                            rows=torch.tensor([S - 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(y, rsu.short_conv_step(v["x"][:1], one, v["weight"], v["bias"]))
    assert torch.equal(cache[S - 1], one[0]) and not cache[:S - 1].any()
