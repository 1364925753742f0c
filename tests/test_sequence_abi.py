"""Host-side checks of the sequence operators (no GPU needed): bad arguments
are reported by the documented status before any HIP call, sizes of buffers,
and the torch entry points' refusals.  No call here reaches a kernel launch:
addresses are fake and every call is invalid, or returns before launching."""
import pytest
import torch

import recurrent_state_update_amd as rsu

OK, INVALID, SHAPE, ALIGN = range(4)
GDN, KDA, RWKV6 = 0, 1, 2
F32, BF16 = 0, 1
A = [0x7f0000000000 + 0x10000000 * i for i in range(24)]  # aligned, far apart, never dereferenced


def desc(op=GDN, dt=BF16, T=128, N=2, H=3, dk=32, dv=64, qs=0, ks=0, vs=0, cu=A[0], q=A[1], k=A[2], v=A[3],
         beta=A[4], ld=A[5], u=None):
    if op == RWKV6:
        beta, u = None, A[6] if u is None else u
    return rsu.dl_scan_desc(op, dt, T, N, H, dk, dv, qs, ks, vs, cu, q, k, v, beta, ld, u)


def scan(d, initial=A[7], final=A[8], rows=None, n_rows=0, o=A[9], saved=None, ws=A[10]):
    return rsu.dl_scan(d, initial, final, rows, n_rows, o, saved, ws, stream=0)


def test_scan_sizes():
    slots = 128 // 64 + 2 + 1
    d = desc()
    assert rsu.dl_scan_workspace_bytes(d) % 256 == 0
    assert rsu.dl_scan_workspace_bytes(desc(op=KDA)) > rsu.dl_scan_workspace_bytes(d) > 0
    states, e = slots * 3 * 32 * 64 * 4, slots * 3 * 64 * 64 * 4
    assert states + e <= rsu.dl_scan_saved_bytes(d) < states + e + 512
    assert states <= rsu.dl_scan_saved_bytes(desc(op=RWKV6)) < states + 256
    assert rsu.dl_scan_backward_workspace_bytes(d) > rsu.dl_scan_saved_bytes(d)
    # large shapes do not wrap around
    big = desc(T=1 << 23, N=1, H=16, dk=128, dv=128)
    assert rsu.dl_scan_saved_bytes(big) > (1 << 23) // 64 * 16 * 128 * 128 * 4


BAD_SIZES = [dict(dk=24), dict(dv=256), dict(dk=0), dict(T=-1), dict(N=0), dict(H=0), dict(op=3), dict(dt=2), dict(op=-1),
             dict(N=1 << 19, H=2), dict(T=1 << 30, H=32)]


@pytest.mark.parametrize("bad", BAD_SIZES, ids=str)
def test_scan_refuses_sizes(bad):
    d = desc(**bad)
    assert rsu.dl_scan_workspace_bytes(d) == rsu.dl_scan_saved_bytes(d) == 0
    assert rsu.dl_scan_backward_workspace_bytes(d) == 0
    assert scan(d) in (INVALID, SHAPE)
    assert rsu.dl_scan_backward(d, *([A[11]] * 11), stream=0) in (INVALID, SHAPE)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(beta=None), INVALID),
    (dict(ld=None), INVALID), (dict(q=A[1] + 1), ALIGN), (dict(ld=A[5] + 2), ALIGN), (dict(cu=A[0] + 2), ALIGN),
    (dict(qs=95), INVALID), (dict(vs=191), INVALID), (dict(ks=1 << 23), SHAPE), (dict(cu=None, T=127), INVALID)])
def test_scan_refuses_inputs(kw, status):
    assert scan(desc(**kw)) == status


def test_scan_refuses_outputs():
    d = desc()
    assert scan(d, o=None) == INVALID and scan(d, ws=None) == INVALID
    assert scan(d, ws=A[10] + 16) == ALIGN and scan(d, final=A[8] + 4) == ALIGN and scan(d, o=A[9] + 1) == ALIGN
    assert scan(d, saved=A[12] + 128) == ALIGN and scan(d, rows=A[13], n_rows=0) == INVALID
    r = desc(op=RWKV6)
    r.u = None
    assert scan(r) == INVALID
    # what a call writes overlaps nothing else of it
    assert scan(d, o=A[3]) == INVALID and scan(d, o=A[3] + 128 * 3 * 64 * 2 - 2) == INVALID
    assert scan(d, initial=A[8] + 16) == INVALID and scan(d, final=A[9]) == INVALID
    assert scan(d, saved=A[10]) == INVALID and scan(d, ws=A[0]) == INVALID
    assert scan(desc(vs=1000), o=A[3] + 2 * 1000 * 100) == INVALID  # inside v's strided span


def test_scan_backward_refuses():
    names = ["saved", "d_o", "d_final", "dq", "dk", "dv", "dbeta", "dld", "du", "d_initial", "ws"]
    good = dict(zip(names, A[11:22]))

    def call(op=GDN, **kw):
        x = {**good, **kw}
        if op != RWKV6:
            x["du"] = None
        return rsu.dl_scan_backward(desc(op=op), *(x[n] for n in names), stream=0)
    for n in ("saved", "dq", "dk", "dv", "dbeta", "dld", "ws"):
        assert call(**{n: None}) == INVALID, n
    assert call(op=RWKV6, du=None) == INVALID
    for n in ("saved", "ws", "d_final", "d_initial"):
        assert call(**{n: good[n] + 8}) == ALIGN, n
    assert call(dq=A[1]) == INVALID and call(dk=good["dq"]) == INVALID and call(dv=good["d_o"]) == INVALID
    assert call(ws=good["saved"]) == INVALID and call(d_initial=good["d_final"]) == INVALID


def test_gated_norm_refuses():
    def call(rows=4, H=2, d=64, ot=F32, t=BF16, o=A[0], g=A[1], gs=0, w=A[2], eps=1e-6, y=A[3]):
        return rsu.dl_gated_norm(rows, H, d, ot, t, o, g, gs, w, eps, y, stream=0)
    assert call(d=48) == SHAPE and call(rows=-1) == INVALID and call(H=0) == INVALID
    assert call(ot=2) == INVALID and call(t=-1) == INVALID
    assert call(eps=0.0) == INVALID and call(eps=float("nan")) == INVALID and call(eps=float("inf")) == INVALID
    assert call(o=None) == INVALID and call(g=None) == INVALID and call(y=None) == INVALID
    assert call(gs=127) == INVALID and call(o=A[0] + 2) == ALIGN and call(y=A[3] + 1) == ALIGN
    assert call(y=A[0]) == INVALID  # o and y differ in type
    assert call(ot=BF16, y=A[0] + 2) == INVALID and call(gs=200, y=A[1]) == INVALID
    assert call(rows=0, o=None, g=None, y=None) == OK
    assert rsu.dl_gated_norm_workspace_bytes(4, 2, 48) == 0 and rsu.dl_gated_norm_workspace_bytes(4, 2, 64) > 0

    def back(dy=A[4], do=A[5], dg=A[6], dw=A[7], ws=A[8]):
        return rsu.dl_gated_norm_backward(4, 2, 64, F32, BF16, A[0], A[1], 0, A[2], 1e-6, dy, do, dg, dw, ws, stream=0)
    for kw in (dict(dy=None), dict(do=None), dict(dg=None), dict(ws=None), dict(do=A[0]), dict(dg=A[4]), dict(ws=A[5])):
        assert back(**kw) == INVALID, kw
    assert back(ws=A[8] + 4) == ALIGN


def test_residual_norm_refuses():
    def call(rows=4, D=100, t=BF16, x=A[0], y=A[1], s=A[2], w=A[3], eps=1e-6, xo=A[4], h=A[5]):
        return rsu.dl_residual_norm(rows, D, t, x, y, s, w, eps, xo, h, stream=0)
    assert call(D=0) == SHAPE and call(D=16385) == SHAPE and call(rows=-1) == INVALID and call(t=2) == INVALID
    assert call(eps=-1.0) == INVALID and call(x=None) == INVALID and call(h=None) == INVALID
    assert call(xo=None) == INVALID and call(y=None) == INVALID  # x_out and scale go with y
    assert call(x=A[0] + 2) == ALIGN and call(h=A[5] + 1) == ALIGN
    assert call(h=A[1]) == INVALID and call(xo=A[0] + 4) == INVALID and call(h=A[4]) == INVALID
    assert call(rows=0) == OK and rsu.dl_residual_norm_workspace_bytes(1, 0) == 0

    def back(y=A[1], s=A[2], dxo=A[4], dh=A[5], dx=A[6], dy=A[7], ds=A[8], dw=A[9], ws=A[10]):
        return rsu.dl_residual_norm_backward(4, 100, BF16, A[0], y, s, A[3], 1e-6, dxo, dh, dx, dy, ds, dw, ws, stream=0)
    for kw in (dict(dx=None), dict(y=None), dict(s=None), dict(ws=None), dict(dy=None), dict(dy=A[5]), dict(dx=A[0]),
               dict(ds=A[9])):
        assert back(**kw) == INVALID, kw
    assert back(dw=A[9] + 1) == ALIGN


def test_torch_entry_points_refuse_cpu_tensors():
    q = torch.zeros(5, 2, 16)
    with pytest.raises(ValueError, match="q: want a GPU tensor"):
        rsu.scan("gdn", q, q, q, torch.zeros(5, 2), torch.zeros(5, 2))
    with pytest.raises(ValueError, match="o: want a GPU tensor"):
        rsu.gated_norm(q, q)
    with pytest.raises(ValueError, match="x: want a GPU tensor"):
        rsu.residual_norm(q)
    with pytest.raises(ValueError):
        rsu.scan("gdn", None, None, None, None, None)
