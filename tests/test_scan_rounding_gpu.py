"""The scan's outputs are sums in 32 bits of factors in 32 bits, rounded once:
outputs whose terms cancel to `SMALL` of them, against 64 bits.

Tolerances, |x - ref| / |ref| in the 2-norm over heads and columns: a factor
or sum that is rounded to fp32 is off by at most 2^-24 of itself, 2^-9 of the
output, and n such roundings by the root of n times that.  Each test counts its
roundings; a bf16 output adds its own, 2^-8.  (Two bf16 values in place of a
factor would be off by 2^-17, 2^-2 of the output.)"""
import pytest
import torch

from sequence_ref import f64, far, scan_ref

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")

OPS = ["gdn", "kda", "rwkv6"]
SMALL = 2.0 ** -15
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
both = pytest.mark.parametrize("dtype", ["f32", "bf16"])


def zeros(op, T, H, dk, dv):
    return dict(q=torch.zeros(T, H, dk), k=torch.zeros(T, H, dk), v=torch.zeros(T, H, dv),
                beta=None if op == "rwkv6" else torch.ones(T, H),
                log_decay=torch.zeros(*((T, H) if op == "gdn" else (T, H, dk))),
                u=torch.zeros(H, dk) if op == "rwkv6" else None, initial_state=None)


def both_ways(op, x, dtype, do=None):
    """o and (with do) dq, from the library and in 64 bits."""
    import recurrent_state_update_amd as rsu
    x = {n: t.to(dtype) if n in "qkv" else t for n, t in x.items()}
    out = []
    for ref in (False, True):
        y = {n: None if t is None else (f64(t) if ref else t.cuda().requires_grad_(n == "q")) for n, t in x.items()}
        a = (y["q"], y["k"], y["v"], y["beta"], y["log_decay"], y["u"], y["initial_state"])
        o = scan_ref(op, *a)[0] if ref else rsu.scan(op, *a)[0]
        out.append(o if do is None else torch.autograd.grad(o, y["q"], do.to(dtype).double() if ref else do.to(dtype).cuda())[0])
    return out


def close(got, want, roundings, dtype):
    tol = roundings ** 0.5 * 2.0 ** -24 / SMALL + (2.0 ** -8 if dtype == "bf16" else 0.0)
    err = far(got, want)
    print(f"off by {err:.1e} of {tol:.1e}", flush=True)
    assert err <= tol


@needs_gpu
@both
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dk,dv", [(16, 32), (128, 128)])
def test_reads_of_the_state(op, dtype, dk, dv):
    """o = S[0] - S[1] with S[1] = (1 + SMALL) S[0].  Roundings: two factors,
    two sums."""
    g = torch.Generator().manual_seed(1)
    x = zeros(op, 5, 3, dk, dv)
    x["q"][:, :, 0], x["q"][:, :, 1] = 1, -1
    s = torch.randn(1, 3, dk, dv, generator=g)
    s[:, :, 1] = s[:, :, 0] * (1 + SMALL)
    x["initial_state"] = s
    close(*both_ways(op, x, DT[dtype]), 4, dtype)


@needs_gpu
@both
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dk", [16, 128])
def test_reads_of_earlier_rows(op, dtype, dk):
    """o_4 = (P_41 - P_42) v, the decay between rows 1 and 2 being 1 - SMALL or
    so (those behind are common to both).  Roundings: two units (four squared)
    of an exponential, two products and a factor in either term, two sums."""
    g = torch.Generator().manual_seed(2)
    H = 8
    x = zeros(op, 4, H, dk, 32)
    x["k"][0, :, 0], x["k"][1, :, 1] = 1, 1
    x["q"][3, :, 0], x["q"][3, :, 1] = 1, -1
    x["v"][:2] = torch.randn(1, H, 32, generator=g)
    ld = -torch.rand(4, H, generator=g)
    ld[1] *= 2 * SMALL
    x["log_decay"] += ld if op == "gdn" else ld.unsqueeze(-1)
    got, want = both_ways(op, x, DT[dtype])
    close(got[3], want[3], 4 + 6 + 2, dtype)


@needs_gpu
@both
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dk", [16, 128])
def test_gradient_of_a_query(op, dtype, dk):
    """dq_4 = (P_41 dO.b_1 - P_42 dO.b_2) e_0 with k_2 = -k_1 = -e_0; the delta
    rule's b_2 = v_2 + P_21 b_1 with v_2 of SMALL.  Roundings: two units
    (four squared) of an exponential, two products in either term and two in
    b_2, two sums of sixteen terms and one of two."""
    g = torch.Generator().manual_seed(3)
    H = 8
    x = zeros(op, 4, H, dk, 16)
    x["k"][0, :, 0], x["k"][1, :, 0] = 1, -1
    x["v"][0] = 0.5 + torch.rand(H, 16, generator=g)
    x["v"][1] = x["v"][0] if op == "rwkv6" else SMALL * (0.5 + torch.rand(H, 16, generator=g))
    ld = -torch.rand(4, H, generator=g)
    if op == "rwkv6":
        ld[1] *= 2 * SMALL
    x["log_decay"] += ld if op == "gdn" else ld.unsqueeze(-1)
    do = torch.zeros(4, H, 16)
    do[3] = 0.5 + torch.rand(H, 16, generator=g)
    got, want = both_ways(op, x, DT[dtype], do)
    close(got[3], want[3], 4 + 6 + 32 + 1, dtype)


@needs_gpu
@both
def test_gradient_of_u_over_many_chunks(dtype):
    """A large chunk and 69 others of 2^-24 of it each, behind it and before:
    du = sum_t q k (dO.v), which no decay enters.  One rounding to fp32."""
    import recurrent_state_update_amd as rsu
    T, H, d = 70 * 64, 2, 16
    x = zeros("rwkv6", T, H, d, d)
    x["q"] += 1
    x["k"] += 1
    x["v"][:, :, 0] = 1
    do = torch.zeros(T, H, d)
    do[5::64, :, 0] = 1
    do[5, 0, 0] = do[-59, 1, 0] = 2.0 ** 24
    x = {n: None if t is None else (t.to(DT[dtype]) if n in "qkv" else t).cuda() for n, t in x.items()}
    u = x["u"].requires_grad_()
    o, _ = rsu.scan("rwkv6", x["q"], x["k"], x["v"], None, x["log_decay"], u)
    (du,) = torch.autograd.grad(o, u, do.to(DT[dtype]).cuda())
    want = do.double().sum((0, 2)).view(H, 1).expand(H, d)
    assert far(du, want) <= 2.0 ** -24
