"""GPU checks of ssm_scan and ssm_step against the recurrence in 64 bits, token by
token, and its adjoint, element by element.

Tolerances, in roundings of 32 bits (2^-24) of the sum of the absolute values of
an output's terms (layer_ref.within).  delta takes an exponential and a reciprocal
good to 2 each, a polynomial and the rounding of its argument times that, up to
8: 20.  A term of the state goes through at most L steps, each with an exponential
(2), two products and a sum: 4 L; its decays' exponents are off by 22 roundings, the
exponent's own size times that, and a term whose exponents add up to more than 16
does not count: 22 x 16 = 352.  24 more for the input, the sum over states N and the
gate: 4 L + N + 400.  Gradients go through two such paths, and are summed over up to
L tokens or, before 64 bits, 64 channels: 9 L + N + 900.  (A bf16 output adds its own
rounding.)"""
import pytest
import torch

from layer_ref import check, offsets, ssm_ref

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "initial")


def units(L, N):
    return {n: 4 * L + N + 400 for n in ("y", "end")} | {
        "d" + n: 9 * L + N + 900 for n in NAMES}


def inputs(lens, C, N, G=1, dtype="f32", gate=True, skip=True, bias=True, init=True, first=0, tail=0, seed=0):
    """Packed CPU inputs, `first` rows ahead of the first sequence and `tail` behind
    the last, cotangents, and the offsets."""
    g = torch.Generator().manual_seed(seed)
    t, cu = DT[dtype], offsets(lens, first)
    T = cu[-1] + tail

    def normal(*s):
        return torch.randn(*s, generator=g)
    x = dict(x=normal(T, C).to(t), dt=(normal(T, C) * 0.7 - (0 if bias else 3)).to(t), A=-torch.exp(normal(C, N)),
             B=normal(T, G, N).to(t), C=normal(T, G, N).to(t), D=normal(C) if skip else None,
             z=normal(T, C).to(t) if gate else None, dt_bias=normal(C) - 3 if bias else None,
             initial=normal(len(lens), C, N) if init else None)
    return x, cu, normal(T, C).to(t), normal(len(lens), C, N)


def run(x, cu, dy=None, dend=None, softplus=True, batch=None):
    """The GPU's outputs by name, in layer_ref's form."""
    import recurrent_state_update_amd as rsu
    v = {n: None if t is None else t.cuda() for n, t in x.items()}
    if batch:
        v = {n: t.unflatten(0, batch) if n in ("x", "dt", "B", "C", "z") and t is not None else t for n, t in v.items()}
    if dy is not None:
        v = {n: None if t is None else t.requires_grad_(True) for n, t in v.items()}
    off = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, end = rsu.ssm_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"], softplus=softplus,
                          initial_state=v["initial"], cu_seqlens=off)
    out = dict(y=y, end=end)
    if dy is not None:
        dy = dy.cuda().reshape(y.shape)
        wrt = [n for n in NAMES if v[n] is not None]
        out.update(("d" + n, t) for n, t in zip(wrt, torch.autograd.grad([y, end], [v[n] for n in wrt], [dy, dend.cuda()])))
    if batch:
        out = {n: t.flatten(0, 1) if n in ("y", "dx", "ddt", "dB", "dC", "dz") else t for n, t in out.items()}
    return out


def compare(x, cu, dy, dend, got, L, softplus=True):
    refs = [ssm_ref(*x.values(), cu, softplus, dy, dend, size=s) for s in (False, True)]
    want = {n: t for n, t in refs[0].items() if n in got}
    assert set(want) == set(got)
    check(got, want, refs[1], units(L, x["A"].shape[1]))


def poison(n=1 << 26):
    """What is allocated next holds NaNs, unless it is written."""
    torch.full((n,), float("nan"), device="cuda")


SHAPES = [
    # lens, channels, states, groups, first, tail
    ([1], 1, 1, 1, 0, 0),
    ([5], 32, 16, 1, 0, 0),
    ([16], 16, 16, 1, 0, 0),
    ([15, 17], 17, 15, 1, 0, 0),
    ([0, 3, 0, 64, 65, 1, 0], 20, 16, 2, 0, 0),
    ([33, 0, 7], 36, 8, 3, 3, 5),
    ([128], 64, 16, 1, 0, 0),
    ([63, 2], 130, 17, 1, 1, 70),
    ([40, 31], 24, 24, 2, 0, 0),
    ([37], 12, 33, 1, 0, 1),
    ([70, 9], 70, 64, 1, 0, 0),
    ([50], 6, 40, 2, 2, 0),
    ([0], 16, 16, 1, 0, 0),
    ([0, 0], 8, 4, 1, 0, 3),
]


@needs_gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
def test_against_64_bits(shape, dtype):
    lens, C, N, G, first, tail = shape
    x, cu, dy, dend = inputs(lens, C, N, G, dtype, first=first, tail=tail, seed=C + N)
    poison()
    compare(x, cu, dy, dend, run(x, cu, dy, dend), max(lens + [1]))
    alone = run(x, cu)  # without a backward pass to come
    both = run(x, cu, dy, dend)
    assert torch.equal(alone["y"], both["y"]) and torch.equal(alone["end"], both["end"])


@needs_gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("without", [("z",), ("D", "z"), ("dt_bias",), ("initial", "D"), ("softplus",)], ids="+".join)
def test_options(without, dtype):
    x, cu, dy, dend = inputs([21, 40], 24, 16, 1, dtype, gate="z" not in without, skip="D" not in without,
                             bias="dt_bias" not in without, init="initial" not in without)
    softplus = "softplus" not in without
    if not softplus:  # delta as given: of either sign
        x["dt"], x["dt_bias"] = (x["dt"].float() * 0.1).to(x["dt"].dtype), x["dt_bias"] * 0.01
    compare(x, cu, dy, dend, run(x, cu, dy, dend, softplus), 40, softplus)


@needs_gpu
@pytest.mark.parametrize("lens,C,N", [([1500], 16, 16), ([700, 3, 0, 690], 40, 24), ([2050], 70, 64)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_segments(lens, C, N, dtype):
    """Long sequences with few channels, which both passes cut into segments."""
    x, cu, dy, dend = inputs(lens, C, N, 1, dtype, first=2, tail=3, seed=5)
    poison()
    compare(x, cu, dy, dend, run(x, cu, dy, dend), max(lens))


@needs_gpu
def test_batch_and_packed_agree():
    x, cu, dy, dend = inputs([37, 37, 37], 20, 16, 2, "bf16")
    a, b = run(x, cu, dy, dend), run(x, None, dy, dend, batch=(3, 37))
    for n in a:
        assert torch.equal(a[n], b[n]), n


@needs_gpu
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_slices(shift):
    """x, dt, z, B and C as slices of projections at any alignment: the same results."""
    import recurrent_state_update_amd as rsu
    x, cu, dy, dend = inputs([40, 9], 32, 16, 2, "bf16")
    want = run(x, cu, dy, dend)
    T = cu[-1]
    wide = torch.zeros(T, 3 * 32 + 2 * 32 + shift + 3, dtype=torch.bfloat16, device="cuda").requires_grad_(True)
    cuts, at = {}, shift
    for n, w in (("x", 32), ("dt", 32), ("z", 32), ("B", 32), ("C", 32)):
        cuts[n] = (at, at + w)
        at += w
    with torch.no_grad():
        for n, (b, e) in cuts.items():
            wide[:, b:e] = x[n].reshape(T, -1).cuda()
    v = {n: wide[:, b:e].unflatten(1, (2, 16)) if n in "BC" else wide[:, b:e] for n, (b, e) in cuts.items()}
    o = {n: x[n].cuda().requires_grad_(True) for n in ("A", "D", "dt_bias", "initial")}
    y, end = rsu.ssm_scan(v["x"], v["dt"], o["A"], v["B"], v["C"], o["D"], v["z"], o["dt_bias"],
                          initial_state=o["initial"], cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, want["y"]) and torch.equal(end, want["end"])
    dw, dA = torch.autograd.grad([y, end], [wide, o["A"]], [dy.cuda(), dend.cuda()])
    assert torch.equal(dA, want["dA"])
    for n, (b, e) in cuts.items():
        assert torch.equal(dw[:, b:e], want["d" + n].reshape(T, -1)), n


@needs_gpu
def test_layouts_that_are_copied():
    """Transposed inputs, expanded cotangents, a channel-last state: the same results."""
    import recurrent_state_update_amd as rsu
    x, cu, _, _ = inputs([19], 16, 16)
    v = {n: t.cuda() for n, t in x.items()}
    y, end = rsu.ssm_scan(*(v[n] for n in NAMES[:-1]), initial_state=v["initial"])
    t = {n: (a.transpose(0, 1).contiguous().transpose(0, 1) if a.dim() > 1 else a) for n, a in v.items()}
    y2, end2 = rsu.ssm_scan(*(t[n] for n in NAMES[:-1]), initial_state=v["initial"].mT.contiguous().mT)
    assert torch.equal(y, y2) and torch.equal(end, end2)
    a = {n: b.requires_grad_(True) for n, b in v.items()}
    y, end = rsu.ssm_scan(*(a[n] for n in NAMES[:-1]), initial_state=a["initial"])
    g1 = torch.autograd.grad(y.sum() + end.sum(), list(a.values()), retain_graph=True)
    g2 = torch.autograd.grad([y, end], list(a.values()), [torch.ones_like(y), torch.ones_like(end)])
    assert all(torch.equal(p, q) for p, q in zip(g1, g2))


@needs_gpu
def test_one_cotangent_only():
    x, cu, dy, dend = inputs([40], 16, 16)
    import recurrent_state_update_amd as rsu
    v = {n: t.cuda().requires_grad_(True) for n, t in x.items()}
    y, end = rsu.ssm_scan(*(v[n] for n in NAMES[:-1]), initial_state=v["initial"])
    for out, cot, dy_, dend_ in ((y, dy, dy, 0 * dend), (end, dend, 0 * dy, dend)):
        got = dict(zip(NAMES, torch.autograd.grad(out, list(v.values()), cot.cuda(), retain_graph=True, allow_unused=True)))
        want = run(x, None, dy_, dend_)
        for n in NAMES:
            assert torch.equal(got[n], want["d" + n]), n


@needs_gpu
def test_gradients_of_some_inputs():
    x, cu, dy, dend = inputs([40], 16, 16)
    import recurrent_state_update_amd as rsu
    want = run(x, None, dy, dend)
    for n in NAMES:
        v = {m: t.cuda().requires_grad_(m == n) for m, t in x.items()}
        out = rsu.ssm_scan(*(v[m] for m in NAMES[:-1]), initial_state=v["initial"])
        assert torch.equal(torch.autograd.grad(out, v[n], [dy.cuda(), dend.cuda()])[0], want["d" + n]), n


@needs_gpu
def test_gradient_against_differences():
    """fp32: a move by 2^-6 along a random direction of each input changes the loss by
    the gradient, up to the loss's own rounding (2^-24 of its terms' sum, a few
    hundred times, over the move) and its third derivative's share (2^-12)."""
    x, cu, dy, dend = inputs([30], 8, 16)
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
        scale = float(grads["d" + n].norm())
        assert abs(slope - want) <= 0.02 * scale + 1e-3, (n, slope, want)


@needs_gpu
def test_repeatable():
    x, cu, dy, dend = inputs([300, 77], 200, 16, 1, "bf16")
    a, b = run(x, cu, dy, dend), run(x, cu, dy, dend)
    for n in a:
        assert torch.equal(a[n], b[n]), n


@needs_gpu
def test_continues_where_it_ended():
    """A sequence in two parts, and its last tokens one at a time: bit for bit where the
    parts end with a block, to rounding elsewhere."""
    import recurrent_state_update_amd as rsu
    x, _, _, _ = inputs([90], 20, 16)
    v = {n: t.cuda() for n, t in x.items()}

    def part(b, e, state):
        return rsu.ssm_scan(*(v[n][b:e] if n in ("x", "dt", "B", "C", "z") else v[n] for n in NAMES[:-1]),
                            initial_state=state)
    y, end = part(0, 90, v["initial"])
    y1, mid = part(0, 64, v["initial"])
    y2, end2 = part(64, 90, mid)
    assert torch.equal(torch.cat([y1, y2]), y) and torch.equal(end2, end)
    state = mid.clone()
    for t in range(64, 90):
        row = rsu.ssm_step(v["x"][t:t + 1], v["dt"][t:t + 1], state, v["A"], v["B"][t:t + 1], v["C"][t:t + 1], v["D"],
                           v["z"][t:t + 1], v["dt_bias"])
        # the same products in another order of summation: 16 roundings of a sum of 16
        assert (row - y[t]).abs().max() <= 64 * 2.0 ** -24 * y.abs().max()
    assert (state - end).abs().max() <= 128 * 2.0 ** -24 * end.abs().max()


@needs_gpu
@pytest.mark.parametrize("N", [1, 3, 4, 8, 13, 16, 24, 32, 64])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step(N, dtype):
    """Rows anywhere in the cache, rows outside it, and rows that no token names."""
    import recurrent_state_update_amd as rsu
    B, C, G, S = 7, 36, 2, 11
    x, _, _, _ = inputs([1] * B, C, N, G, dtype, init=False, seed=N)
    g = torch.Generator().manual_seed(N)
    cache = torch.randn(S, C, N, generator=g)
    rows = [3, -1, 10, 0, S, 7, 1]
    known = [0 <= r < S for r in rows]
    x["initial"] = torch.stack([cache[r] if k else torch.zeros(C, N) for r, k in zip(rows, known)])
    refs = [ssm_ref(*x.values(), offsets([1] * B), size=s) for s in (False, True)]
    v = {n: None if t is None else t.cuda() for n, t in x.items()}
    state = cache.cuda()
    y = rsu.ssm_step(v["x"], v["dt"], state, v["A"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"],
                     rows=torch.tensor(rows, dtype=torch.int32, device="cuda"))
    want, size = cache.double(), cache.double().abs()
    for i, r in enumerate(rows):
        if known[i]:
            want[r], size[r] = refs[0]["end"][i], refs[1]["end"][i]
    check(dict(y=y, end=state), dict(y=refs[0]["y"], end=want), dict(y=refs[1]["y"], end=size), units(1, N))
    untouched = [r for r in range(S) if r not in rows]
    assert torch.equal(state[untouched].cpu(), cache[untouched])
    # default rows, one group without its dimension, no options
    state = cache.cuda()
    y = rsu.ssm_step(v["x"], v["dt"], state, v["A"], v["B"][:, 0], v["C"][:, 0])
    plain = dict(x, B=x["B"][:, :1], C=x["C"][:, :1], D=None, z=None, dt_bias=None, initial=cache[:B])
    refs = [ssm_ref(*plain.values(), offsets([1] * B), size=s) for s in (False, True)]
    check(dict(y=y, end=state[:B]), refs[0], refs[1], units(1, N))
    assert torch.equal(state[B:].cpu(), cache[B:])


@needs_gpu
def test_forgetting_and_extremes():
    """Rates of -inf and 0, delta of 0 (to rounding) and of hundreds, gates far out."""
    x, cu, dy, dend = inputs([50, 20], 16, 16)
    x["A"][0], x["A"][1] = float("-inf"), 0.0
    x["A"][2, 3] = -1e30
    x["dt"][5:9] = 300.0
    x["dt"][20:30, 4:] = -80.0
    x["z"][3], x["z"][4] = 60.0, -60.0
    got = run(x, cu, dy, dend)
    # what a rate of -inf multiplies is exactly 0
    x["A"][0] = -1e300 if x["A"].dtype == torch.float64 else -1e37
    compare(x, cu, dy, dend, got, 50)


@needs_gpu
def test_nan_stays_in_its_sequence_and_channel():
    x, cu, dy, dend = inputs([33, 40, 20], 20, 16)
    clean = run(x, cu, dy, dend)
    x["x"][40, 3] = float("nan")  # of the second sequence
    dirty = run(x, cu, dy, dend)
    ok = torch.ones(93, 20, dtype=torch.bool)
    ok[40:73, 3] = False
    for n in ("y", "dz"):
        assert torch.equal(dirty[n].cpu()[ok], clean[n].cpu()[ok]), n
    assert torch.isnan(dirty["y"][40:73, 3]).all()
    assert torch.equal(dirty["end"][[0, 2]], clean["end"][[0, 2]])
    # rows of no sequence take no part
    x, cu, dy, dend = inputs([33, 40], 20, 16, first=3, tail=9)
    clean = run(x, cu, dy, dend)
    for n in ("x", "dt", "B", "C", "z"):
        x[n][:3], x[n][-9:] = float("nan"), float("inf")
    dy[:3] = dy[-9:] = float("nan")
    dirty = run(x, cu, dy, dend)
    for n in clean:
        assert torch.equal(dirty[n], clean[n]), n


@needs_gpu
@pytest.mark.parametrize("cu", [[0, 50, 20, 60], [-5, 30, 90, 60], [60, 40, 20, 0], [0, 2 ** 31 - 1, 10, 60],
                                [-2 ** 31, 5, 5, 70]])
@pytest.mark.parametrize("tokens", [60, 2400])
def test_bad_offsets_stay_in_range(cu, tokens):
    """Offsets out of order or range: no result is promised, and guards around every
    output stay whole."""
    import recurrent_state_update_amd as rsu
    x, _, dy, dend = inputs([tokens // 3] * 3, 16, 16, seed=1)
    cu = [c * (tokens // 60) if 0 < c <= 60 else c for c in cu]
    out = run(x, cu, dy, dend)
    torch.cuda.synchronize()
    assert out["y"].shape == (tokens, 16)


def _replays(g, state, fresh, outs, eager, times=3):
    for k in range(times):
        for t, v in zip(state, fresh(k)):
            t.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = eager()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@needs_gpu
@pytest.mark.parametrize("lens", [[40, 0, 33], [1100]])
def test_graph_replays(lens):
    """Forward and backward captured in a graph and replayed on new inputs, new offsets
    too, with eager work between."""
    import recurrent_state_update_amd as rsu
    sets = [inputs(lens, 20, 16, 1, "bf16", seed=s) for s in range(4)]
    v = [None if t is None else t.cuda() for t in sets[0][0].values()]
    dy, dend = sets[0][2].cuda(), sets[0][3].cuda()
    cu = torch.tensor(sets[0][1], dtype=torch.int32, device="cuda")

    def step():
        a = [t.detach().requires_grad_(True) for t in v]
        y, end = rsu.ssm_scan(*a[:-1], initial_state=a[-1], cu_seqlens=cu)
        return [y.detach(), end.detach(), *torch.autograd.grad([y, end], a, [dy, dend])]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()

    def fresh(k):
        x, off, a, b = sets[k + 1]
        off = list(off)
        if len(off) > 2:  # other lengths of the same tokens
            off[1], off[2] = off[1] - 7 * k, off[2] - 7 * k + 1
        return [*x.values(), a, b, torch.tensor(off, dtype=torch.int32)]
    _replays(g, [*v, dy, dend, cu], fresh, outs, step)


@needs_gpu
def test_step_in_a_graph():
    """Steps in a graph move the same cache on, replay by replay."""
    import recurrent_state_update_amd as rsu
    x, _, _, _ = inputs([1] * 6, 20, 16, 1, "bf16")
    v = {n: t.cuda() for n, t in x.items()}
    rows = torch.tensor([5, 0, 3, -1, 2, 7], dtype=torch.int32, device="cuda")
    start = torch.randn(8, 20, 16, device="cuda")

    def step(state):
        return rsu.ssm_step(v["x"], v["dt"], state, v["A"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"], rows=rows)
    cache, other = start.clone(), start.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(start.clone())
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step(cache)
    for _ in range(4):
        v["x"].normal_()
        rows.copy_(rows.roll(1))
        g.replay()
        assert torch.equal(step(other), y)
        assert torch.equal(cache, other)


@needs_gpu
def test_streams():
    """A call on a stream of its own, named and current, forward and backward."""
    import recurrent_state_update_amd as rsu
    x, cu, dy, dend = inputs([300], 64, 16)
    want = run(x, cu, dy, dend)
    v = {n: t.cuda().requires_grad_(True) for n, t in x.items()}
    dy, dend = dy.cuda(), dend.cuda()
    torch.cuda.synchronize()
    for named in (True, False):
        s = torch.cuda.Stream()
        with torch.cuda.stream(None if named else s):
            y, end = rsu.ssm_scan(*(v[n] for n in NAMES[:-1]), initial_state=v["initial"], stream=s if named else None)
        with torch.cuda.stream(s):
            grads = torch.autograd.grad([y, end], list(v.values()), [dy, dend])
        torch.cuda.synchronize()
        assert torch.equal(y, want["y"]) and torch.equal(end, want["end"])
        for n, t in zip(NAMES, grads):
            assert torch.equal(t, want["d" + n]), n


@needs_gpu
def test_offsets_beyond_32_bits():
    """Rows more than 2^31 elements from the first, in the scan (both ways) and in a
    step's cache: as a call on those rows alone."""
    import recurrent_state_update_amd as rsu
    C, T, L = 16384, 131200, 60
    x, _, dy, dend = inputs([L], C, 1, 1, "bf16", seed=9)
    want = run(x, None, dy, dend)
    v = {n: t.cuda() for n, t in x.items()}
    big = {}
    for n in ("x", "dt", "B", "C", "z"):
        big[n] = torch.zeros(T, *v[n].shape[1:], dtype=torch.bfloat16, device="cuda")
        big[n][-L:] = v[n]
    bdy = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    bdy[-L:] = dy.cuda()
    assert (T - L) * C > 2 ** 31
    o = {n: v[n] for n in ("A", "D", "dt_bias")}
    init = torch.cat([torch.zeros(1, C, 1, device="cuda"), v["initial"]])
    leaves = {n: t.requires_grad_(True) for n, t in {**big, **o, "initial": init}.items()}
    cu = torch.tensor([0, T - L, T], dtype=torch.int32, device="cuda")
    y, end = rsu.ssm_scan(leaves["x"], leaves["dt"], leaves["A"], leaves["B"], leaves["C"], leaves["D"], leaves["z"],
                          leaves["dt_bias"], initial_state=leaves["initial"], cu_seqlens=cu)
    assert torch.equal(y[-L:], want["y"]) and torch.equal(end[1:], want["end"])
    assert not y[:-L].any()
    wrt = ("x", "dt", "B", "C", "z", "initial")
    grads = dict(zip(wrt, torch.autograd.grad([y, end], [leaves[n] for n in wrt],
                                              [bdy, torch.cat([0 * dend, dend]).cuda()])))
    for n in wrt[:-1]:
        assert torch.equal(grads[n][-L:], want["d" + n]), n
    assert torch.equal(grads["initial"][1:], want["dinitial"])


@needs_gpu
def test_step_cache_beyond_32_bits():
    import recurrent_state_update_amd as rsu
    C, N, S = 4096, 64, 8300
    assert (S - 1) * C * N > 2 ** 31
    x, _, _, _ = inputs([1, 1], C, N, seed=4)
    v = {n: t.cuda() for n, t in x.items()}
    cache = torch.zeros(S, C, N, device="cuda")
    cache[S - 1], cache[0] = v["initial"][0], v["initial"][1]
    small = v["initial"].clone()
    args = [v[n] for n in ("A", "B", "C", "D", "z", "dt_bias")]
    y = rsu.ssm_step(v["x"], v["dt"], cache, *args, rows=torch.tensor([S - 1, 0], dtype=torch.int32, device="cuda"))
    want = rsu.ssm_step(v["x"], v["dt"], small, *args)
    assert torch.equal(y, want) and torch.equal(cache[S - 1], small[0]) and torch.equal(cache[0], small[1])
    assert not cache[1:S - 1].any()


@needs_gpu
@pytest.mark.parametrize("lens,C,N", [([128], 16, 16), ([64, 64], 20, 33), ([1] * 40 + [300] + [2] * 20, 70, 16),
                                      ([5, 0, 0, 590, 0], 130, 24)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_long_sequence_among_short_ones(lens, C, N, dtype):
    """Cut by all tokens, not by each sequence's: pieces that do not exist, empty ones."""
    x, cu, dy, dend = inputs(lens, C, N, 1, dtype, first=1, tail=40, seed=6)
    poison()
    compare(x, cu, dy, dend, run(x, cu, dy, dend), max(lens))


@needs_gpu
@pytest.mark.parametrize("N,C", [(16, 4112), (20, 4100), (40, 4097)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_channels(N, C, dtype):
    """More workgroups than CUs, of sequences that are not short."""
    x, cu, dy, dend = inputs([150, 131], C, N, 1, dtype, seed=9)
    poison()
    compare(x, cu, dy, dend, run(x, cu, dy, dend), 150)


@needs_gpu
@pytest.mark.parametrize("N", [8, 24, 64])
def test_any_company(N):
    """A sequence's results are the same bits alone and among others, short and long,
    whatever stages those take (it is not cut in either)."""
    x, cu, _, _ = inputs([150, 1, 7] + [2] * 30 + [90] * 20, 4112, N, 1, "bf16", seed=4)
    both = run(x, cu)
    for k, n in enumerate([150, 1, 7]):
        b = cu[k]
        one = {m: t[b:b + n] if m in ("x", "dt", "B", "C", "z") else t[k:k + 1] if m == "initial" else t for m, t in x.items()}
        alone = run(one, [0, n])
        assert torch.equal(alone["y"], both["y"][b:b + n]) and torch.equal(alone["end"][0], both["end"][k])
