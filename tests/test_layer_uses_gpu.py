"""Uses of a state space layer's operators that the other files do not make: saved
tensors kept elsewhere, two calls at once, graphs that share memory, broadcast inputs,
no token at all, states that grow through many segments, parts of larger caches."""
import pytest
import torch
import torch.utils.checkpoint

from layer_ref import check, ssm_ref
from test_ssm_gpu import NAMES, inputs, poison, run

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")


def block(p, conv, bias, A, D, dt_bias, cu):
    """Slices of a projection through convolution and scan."""
    import recurrent_state_update_amd as rsu
    C, N = A.shape
    u, seen = rsu.short_conv(p[:, :C], conv, bias, cu_seqlens=cu)
    y, end = rsu.ssm_scan(u, p[:, C:2 * C], A, p[:, 3 * C:3 * C + N], p[:, 3 * C + N:], D, p[:, 2 * C:3 * C], dt_bias,
                          cu_seqlens=cu)
    return y, end, seen


def block_leaves(T=150, C=40, N=16, dtype=torch.float32, seed=1):
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = [normal(T, 3 * C + 2 * N).to(dtype), normal(C, 4) / 2, normal(C) / 5, -torch.exp(normal(C, N)), normal(C),
         normal(C) - 3]
    cu = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device="cuda")
    return [t.cuda().requires_grad_() for t in a], cu


def gradients(outs, leaves):
    """With cotangents 1, 2, 3 of the outputs."""
    return torch.autograd.grad(outs, leaves, [torch.full_like(t, k + 1) for k, t in enumerate(outs)])


@needs_gpu
@pytest.mark.parametrize("T", [150, 1400])
@pytest.mark.parametrize("kept", ["checkpoint", "offload"])
def test_saved_elsewhere(kept, T):
    leaves, cu = block_leaves(T)

    def grads(how):
        if how == "checkpoint":
            outs = torch.utils.checkpoint.checkpoint(block, *leaves, cu, use_reentrant=False)
        elif how == "offload":
            with torch.autograd.graph.save_on_cpu():
                outs = block(*leaves, cu)
        else:
            outs = block(*leaves, cu)
        poison()  # over what was freed
        return gradients(outs, leaves)
    want = grads(None)
    assert all(w.isfinite().all() and w.abs().max() > 0 for w in want)
    for got, w in zip(grads(kept), want):
        assert torch.equal(got, w)


@needs_gpu
def test_no_second_derivative():
    leaves, cu = block_leaves(40)
    first = torch.autograd.grad(block(*leaves, cu)[0].sum(), leaves, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(first[-1].sum(), leaves)


@needs_gpu
def test_inputs_changed_before_the_backward_pass():
    import recurrent_state_update_amd as rsu
    x, _, _, _ = inputs([20], 16, 16)
    v = {n: t.cuda().requires_grad_() for n, t in x.items()}
    y, _ = rsu.ssm_scan(*(v[n] for n in NAMES[:-1]), initial_state=v["initial"])
    with torch.no_grad():
        v["A"].mul_(2)
    with pytest.raises(RuntimeError):
        y.sum().backward()


@needs_gpu
@pytest.mark.parametrize("T", [400, 1600])
def test_two_calls_at_once(T):
    """Forward and backward passes of two layers on two streams, side by side."""
    sets = [block_leaves(T, C=c, dtype=torch.bfloat16, seed=c) for c in (40, 96)]
    want = [gradients(block(*leaves, cu), leaves) for leaves, cu in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got, outs = [], []
        for s, (leaves, cu) in zip(streams, sets):
            with torch.cuda.stream(s):
                outs.append(block(*leaves, cu))
        for s, out, (leaves, _) in zip(streams, outs, sets):
            with torch.cuda.stream(s):
                got.append(gradients(out, leaves))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@needs_gpu
def test_graphs_that_share_a_pool():
    """Two captured training steps in one memory pool, whose workspaces are then the same
    memory, replayed in turn."""
    sets = [block_leaves(1400, C=c, dtype=torch.bfloat16, seed=c) for c in (40, 24)]

    def step(leaves, cu):
        a = [t.detach().requires_grad_() for t in leaves]
        return gradients(block(*a, cu), a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = [step(*x) for x in sets]
    torch.cuda.current_stream().wait_stream(s)
    pool, graphs, outs = torch.cuda.graph_pool_handle(), [], []
    for x in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], pool=pool):
            outs.append(step(*x))
    for k in (0, 1, 1, 0, 1, 0):
        graphs[k].replay()
        assert all(torch.equal(a, b) for a, b in zip(outs[k], want[k]))
        eager = step(*sets[k])
        assert all(torch.equal(a, b) for a, b in zip(eager, want[k]))


@needs_gpu
def test_decode_steps_at_once():
    """The same cache's halves moved on from two streams, and the norm beside them."""
    import recurrent_state_update_amd as rsu
    x, _, _, _ = inputs([1] * 64, 48, 16, 1, "bf16")
    v = {n: t.cuda() for n, t in x.items()}
    cache = torch.randn(3, 80, 48, 16, device="cuda")  # of three layers
    rows = torch.randperm(80, device="cuda", dtype=torch.int32)[:64].contiguous()
    res = torch.randn(64, 256, device="cuda")

    def step(state, b, e):
        return rsu.ssm_step(v["x"][b:e], v["dt"][b:e], state, v["A"], v["B"][b:e], v["C"][b:e], v["D"], v["z"][b:e],
                            v["dt_bias"], rows=rows[b:e])
    with torch.no_grad():
        other = cache[1].clone()
        want = [step(other, 0, 64) for _ in range(3)]
        _, h, scale = rsu.residual_norm_fp8(res)
        before = cache[[0, 2]].clone()
        torch.cuda.synchronize()
        streams, got = [torch.cuda.Stream() for _ in range(3)], []
        for _ in range(3):
            ys = []
            for k in (0, 1):
                with torch.cuda.stream(streams[k]):
                    ys.append(step(cache[1], 32 * k, 32 * k + 32))
            got.append(ys)
            with torch.cuda.stream(streams[2]):
                again = rsu.residual_norm_fp8(res)
        torch.cuda.synchronize()
    assert all(torch.equal(torch.cat(ys), w) for ys, w in zip(got, want))
    assert torch.equal(cache[1], other) and torch.equal(cache[[0, 2]], before)
    assert torch.equal(again[1].view(torch.uint8), h.view(torch.uint8)) and torch.equal(again[2], scale)


@needs_gpu
def test_broadcast_inputs():
    """Inputs that are broadcast views, and one tensor as several inputs: their gradients
    are those of the inputs written out, summed."""
    import recurrent_state_update_amd as rsu
    g = torch.Generator().manual_seed(2)
    T, C, N, G = 40, 24, 16, 3
    normal = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    small = dict(x=normal(T, 1), dt=normal(1, C), A=-normal(1, N).exp(), BC=normal(T, 1, N), D=normal(1), w=normal(1, 4),
                 dy=normal(T, C))

    def go(written):
        v = {n: t.clone().requires_grad_() for n, t in small.items()}
        e = (lambda t, *s: t.expand(*s).contiguous()) if written else (lambda t, *s: t.expand(*s))
        x, bc = e(v["x"], T, C), e(v["BC"], T, G, N)
        u, _ = rsu.short_conv(x, e(v["w"], C, 4))
        y, _ = rsu.ssm_scan(u, e(v["dt"], T, C), e(v["A"], C, N), bc, bc, e(v["D"], C), x)
        return y.detach(), torch.autograd.grad(y, [v[n] for n in ("x", "dt", "A", "BC", "D", "w")], small["dy"])
    (y, got), (y2, want) = go(False), go(True)
    assert torch.equal(y, y2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@needs_gpu
def test_no_tokens():
    """Nothing to do: states pass through, weights' gradients are zero."""
    import recurrent_state_update_amd as rsu
    leaves, _ = block_leaves(0)
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    p, conv, bias, A, D, dt_bias = leaves
    seen = torch.randn(3, 3, 40, device="cuda", requires_grad=True)
    state = torch.randn(3, 40, 16, device="cuda", requires_grad=True)
    poison()
    u, s1 = rsu.short_conv(p[:, :40], conv, bias, seen, cu)
    y, s2 = rsu.ssm_scan(u, p[:, 40:80], A, p[:, 120:136], p[:, 136:], D, p[:, 80:120], dt_bias, initial_state=state,
                         cu_seqlens=cu)
    assert y.shape == (0, 40) and torch.equal(s1, seen) and torch.equal(s2, state)
    grads = torch.autograd.grad(y.sum() + s1.sum() + s2.sum(), [conv, bias, A, D, dt_bias, seen, state])
    assert all((t == (1 if k > 4 else 0)).all() for k, t in enumerate(grads))
    with torch.no_grad():
        y = rsu.ssm_step(p[:, :40], p[:, :40], state.detach(), A, p[:, :16], p[:, :16])
        assert y.shape == (0, 40)
        assert rsu.short_conv_step(p[:, :40], seen.detach(), conv).shape == (0, 40)


@needs_gpu
def test_states_that_grow():
    """A > 0, in sequences that are cut: a state of zero stays zero behind segments whose
    decay, e^128, is no number of 32 bits, and so does a gradient of zero ahead of them."""
    x, cu, dy, dend = inputs([1500], 16, 4, gate=False, init=False)
    x["A"], x["dt"], x["dt_bias"] = torch.ones(16, 4), torch.ones_like(x["dt"]), None
    x["x"][:1440] = 0  # e^60 of them at the end
    dy[60:] = 0        # and of those at the front
    dend.zero_()
    poison()
    got = run(x, cu, dy, dend, softplus=False)
    refs = [ssm_ref(*x.values(), cu, False, dy, dend, size=s) for s in (False, True)]
    # 60 steps of e at 4 roundings, their exponents' 60 at 22, the sums of 60 and 64
    check(got, {n: refs[0][n] for n in got}, refs[1], 4 * 60 + 22 * 60 + 124)
    assert (got["y"][:1440] == 0).all() and (got["dx"][60:1440] == 0).all()


@needs_gpu
def test_small_states_that_grow():
    """A state of 1e-30 through a segment whose decay is e^128: 1e25, a number."""
    x, cu, _, _ = inputs([1500], 16, 4, gate=False, init=True)
    x["A"], x["dt_bias"] = torch.ones(16, 4), None
    x["dt"].zero_()
    x["dt"][:128] = 1
    x["x"][:128] = 0
    x["initial"] *= 1e-30
    got = run(x, cu, softplus=False)
    refs = [ssm_ref(*x.values(), cu, False, size=s) for s in (False, True)]
    # 128 steps at 4 roundings, their exponents' 128 at 22, the sum of 4 and D's
    check(got, {n: refs[0][n] for n in got}, refs[1], 4 * 128 + 22 * 128 + 8)


@needs_gpu
def test_copies_are_made_on_the_stream_named():
    """Offsets and rows that have to be copied, on a stream other than the current one,
    which is busy: the copies wait for nothing there."""
    import recurrent_state_update_amd as rsu
    x, _, _, _ = inputs([30, 34], 20, 16, dtype="bf16")
    v = {n: t.cuda() for n, t in x.items()}
    off = torch.tensor([[0, 9], [30, 9], [64, 9]], dtype=torch.int32, device="cuda")[:, 0]
    rows = torch.tensor([[k, 9] for k in range(64)], dtype=torch.int32, device="cuda").flip(0)[:, 0]
    w = torch.randn(20, 4, device="cuda")
    cache = torch.randn(64, 3, 20, device="cuda").bfloat16(), torch.randn(64, 20, 16, device="cuda")

    def go(stream, off, rows):
        with torch.no_grad():
            a, b = (t.clone() for t in cache)
            torch.cuda.synchronize()
            if stream:
                torch.cuda._sleep(50_000_000)
            outs = [*rsu.short_conv(v["x"], w, cu_seqlens=off, stream=stream),
                    *rsu.ssm_scan(*(v[n] for n in NAMES[:-1]), cu_seqlens=off, stream=stream),
                    rsu.short_conv_step(v["x"], a, w, rows=rows, stream=stream),
                    rsu.ssm_step(v["x"], v["dt"], b, *(v[n] for n in NAMES[2:-1]), rows=rows, stream=stream), a, b]
            torch.cuda.synchronize()
        return outs
    want = go(None, off.contiguous(), rows.contiguous())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert all(torch.equal(p, q) for p, q in zip(go(s, off, rows), want))
