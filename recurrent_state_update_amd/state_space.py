"""The operators of a state space layer, on torch tensors: `short_conv` (the
short causal convolution in front of a recurrence; GDN and KDA layers have it on
q, k and v), `ssm_scan` (the selective state space scan), and `short_conv_step`
and `ssm_step`, the same for one token of each of many requests.

Argument checks, output and workspace allocation and autograd nodes only, as in
sequence.py, and with its rules for streams, graphs, derivatives and devices: the
arithmetic is in libdeltalog (dl_short_conv, dl_ssm_scan, their backward passes
and steps).
"""
from __future__ import annotations

import torch

from . import (_check, _dtype_id, _lib, dl_conv_desc, dl_short_conv_workspace_bytes, dl_ssm_backward_workspace_bytes,
               dl_ssm_desc, dl_ssm_saved_bytes, dl_ssm_workspace_bytes)
from .sequence import _MOST_STRIDE, _count, _current, _gpu, _no_grad, _on, _p, _plain, _rows, _tensor, _wants_grad

_MOST_STATES = 64


def _shape(x):
    """The leading dimensions of x [T,C] or [N,T,C], its channels and rows."""
    if x.dim() not in (2, 3):
        raise ValueError(f"x: want [T,C] or [N,T,C], got {tuple(x.shape)}")
    *lead, C = x.shape
    if C < 1:
        raise ValueError("x: want at least one channel")
    return tuple(lead), _count(C, "channels"), _count(x.numel() // C)


def _sequences(lead, cu_seqlens, device):
    """How many sequences there are."""
    if cu_seqlens is None:
        N = lead[0] if len(lead) == 2 else 1
    else:
        if len(lead) != 1:
            raise ValueError("cu_seqlens goes with packed tensors [T,C]")
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens: want a 1-D int32 GPU tensor of at least two offsets")
        _tensor(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, device)
        N = cu_seqlens.numel() - 1
    if N < 1:
        raise ValueError("want at least one sequence")
    return _count(N, "sequences")


def _channel_rows(t, lead):
    """t [*lead,C] as rows a fixed distance apart (copied if it is not laid out
    so), and that distance."""
    if t is None:
        return None, 0
    if t.is_contiguous():
        return t, t.shape[-1]
    wide, stride = _rows(t.unsqueeze(-2), lead, _MOST_STRIDE)
    return wide.squeeze(-2), stride


def _whole(t):
    return None if t is None else t.contiguous()


def _like(t):
    """A contiguous tensor of t's shape and type (half the host's time of torch.empty)."""
    return None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)


def _scratch(n, t):
    """n bytes beside t, an fp32 tensor."""
    return t.new_empty(n + 3 >> 2)


def _in_place(state, name, dtype, tail, device):
    """A cache of states [rows,*tail] that a step moves on."""
    if not isinstance(state, torch.Tensor) or state.dim() != 1 + len(tail):
        raise ValueError(f"{name}: want a GPU tensor [rows,{','.join(map(str, tail))}]")
    _tensor(state, name, dtype, (_count(state.shape[0], "rows of states"), *tail), device)
    if not state.is_contiguous():
        raise ValueError(f"{name}: want a contiguous tensor, since it is updated in place")


def _state_rows(rows, T, state, device):
    if rows is None:
        if state.shape[0] < T:
            raise ValueError(f"state: {state.shape[0]} rows for {T} tokens: name their rows")
    else:
        _tensor(rows, "rows", torch.int32, (T,), device)


def _changed(state):
    if not state.is_inference():
        torch.autograd.graph.increment_version(state)


# -------------------------------------------------------------- convolution --

class _Conv:
    """The checked arguments of one convolution."""

    def __init__(self, x, weight, bias, silu):
        self.device, self.dtype = x.device, x.dtype
        self.lead, self.C, self.T = _shape(x)
        if not isinstance(weight, torch.Tensor) or weight.dim() != 2 or not 2 <= weight.shape[1] <= 4:
            raise ValueError("weight: want fp32 [C,W] with 2 to 4 taps")
        self.W = weight.shape[1]
        _tensor(weight, "weight", torch.float32, (self.C, self.W), self.device)
        if bias is not None:
            _tensor(bias, "bias", torch.float32, (self.C,), self.device)
        self.silu, self.dti = int(bool(silu)), _dtype_id(x.dtype)

    def describe(self, N, x, weight, bias, cu_seqlens):
        """These tensors, copied where the library cannot read them as they are,
        and their descriptor."""
        x, stride = _channel_rows(x, len(self.lead))
        weight, bias, cu_seqlens = _whole(weight), _whole(bias), _whole(cu_seqlens)
        return (x, weight, bias, cu_seqlens), dl_conv_desc(
            self.dti, self.T, N, self.C, self.W, self.silu, stride, _p(cu_seqlens), x.data_ptr(), weight.data_ptr(),
            _p(bias))

    def forward(self, desc, x, N, initial):
        y, end = _like(x), x.new_empty((N, self.W - 1, self.C))
        _check(_lib.dl_short_conv(desc, _p(initial), end.data_ptr(), y.data_ptr(), _current(self.device)),
               "dl_short_conv")
        return y, end


class _ConvFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, s, N, cu_seqlens, x, weight, bias, initial):
        tensors, desc = s.describe(N, x, weight, bias, cu_seqlens)
        out = s.forward(desc, x, N, initial)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(*tensors, initial)
        ctx.conv, ctx.N = s, N
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, d_end):
        s = ctx.conv
        x, weight, bias, cu_seqlens, initial = ctx.saved_tensors
        with _on(s.device, None):
            # (a tensor's layout may be another than when it was saved)
            (x, weight, bias, cu_seqlens), desc = s.describe(ctx.N, x, weight, bias, cu_seqlens)
            initial, dy, d_end = _whole(initial), _whole(dy), _whole(d_end)
            dx = _like(x)
            dw = _like(weight) if ctx.needs_input_grad[4] else None
            db = _like(bias) if ctx.needs_input_grad[5] else None
            d0 = _like(initial) if ctx.needs_input_grad[6] else None
            ws = None if dw is None and db is None else _scratch(dl_short_conv_workspace_bytes(desc), weight)
            _check(_lib.dl_short_conv_backward(desc, _p(initial), _p(dy), _p(d_end), dx.data_ptr(), _p(dw), _p(db),
                                               _p(d0), _p(ws), _current(s.device)), "dl_short_conv_backward")
        return None, None, None, dx, dw, db, d0


def short_conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, silu: bool = True, stream=None):
    """The short causal convolution of every channel, as it stands in front of a
    recurrence: s_t = bias + sum_j weight[:,j] * x_{t-W+1+j}, and s * sigmoid(s)
    of it (``silu`` False: s itself).

    x [T,C] (bf16 or fp32; its rows may be slices of a projection), weight [C,W]
    fp32 with 2 to 4 taps, the last one the token's own, bias [C] fp32 or None: N
    sequences packed one after the other, sequence n being the rows cu_seqlens[n]
    to cu_seqlens[n+1] (GPU, int32; default: one sequence), or x [N,T,C].
    initial_state [N,W-1,C] in x's dtype: the last inputs ahead of each sequence, the
    oldest first (default: zero).

    Returns y, shaped as x, and the end states, as initial_state.  Rows of no
    sequence hold zeros.  Differentiable by x, weight, bias and initial_state."""
    _plain("short_conv", x, weight, bias, initial_state)
    dev = _gpu(x, "x")
    s = _Conv(x, weight, bias, silu)
    N = _sequences(s.lead, cu_seqlens, dev)
    if initial_state is not None:
        _tensor(initial_state, "initial_state", x.dtype, (N, s.W - 1, s.C), dev)
    with _on(dev, stream):
        initial = _whole(initial_state)
        if _wants_grad(x, weight, bias, initial):
            return _ConvFn.apply(s, N, cu_seqlens, x, weight, bias, initial)
        tensors, desc = s.describe(N, x, weight, bias, cu_seqlens)
        return s.forward(desc, x, N, initial)


def short_conv_step(x, state, weight, bias=None, rows=None, silu: bool = True, stream=None):
    """`short_conv` for one token of each of B requests: x [B,C], and ``state``
    [S,W-1,C] (a cache of states, contiguous, in x's dtype), of which the tokens'
    rows are moved on in place: rows[b] (GPU, int32, no row twice; default: row b).
    A row outside the cache (a padded batch's, -1) counts as zero and is not
    written.  Returns y [B,C].  For inference: it has no gradient and refuses
    inputs that want one."""
    _plain("short_conv_step", x, state, weight, bias)
    dev = _gpu(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x: want [B,C], got {tuple(x.shape)}")
    s = _Conv(x, weight, bias, silu)
    _in_place(state, "state", x.dtype, (s.W - 1, s.C), dev)
    _state_rows(rows, s.T, state, dev)
    _no_grad("short_conv_step", x, state, weight, bias)
    with _on(dev, stream):
        tensors, desc = s.describe(1, x, weight, bias, None)
        y, rows = _like(x), _whole(rows)
        _check(_lib.dl_short_conv_step(desc, state.data_ptr(), _p(rows), state.shape[0], y.data_ptr(), _current(dev)),
               "dl_short_conv_step")
        _changed(state)
        return y


# --------------------------------------------------------------------- scan --

class _Ssm:
    """The checked arguments of one selective scan."""

    def __init__(self, x, dt, A, B, C, D, z, dt_bias, softplus):
        dev, dtype, shape = x.device, x.dtype, x.shape
        self.device, self.dtype = dev, dtype
        lead, ch, self.T = _shape(x)
        self.lead, self.C = lead, ch
        self.dti = _dtype_id(dtype)
        _tensor(dt, "dt", dtype, shape, dev)
        if z is not None:
            _tensor(z, "z", dtype, shape, dev)
        if not isinstance(A, torch.Tensor) or A.dim() != 2 or not 1 <= A.shape[1] <= _MOST_STATES:
            raise ValueError(f"A: want fp32 [C,N] with 1 to {_MOST_STATES} states")
        self.S = A.shape[1]
        _tensor(A, "A", torch.float32, (ch, self.S), dev)
        self.grouped = isinstance(B, torch.Tensor) and B.dim() == len(lead) + 2
        self.G = B.shape[-2] if self.grouped else 1
        bc = (*lead, self.G, self.S) if self.grouped else (*lead, self.S)
        _tensor(B, "B", dtype, bc, dev)
        _tensor(C, "C", dtype, bc, dev)
        if self.G < 1 or ch % self.G != 0:
            raise ValueError(f"B: {self.G} groups for {ch} channels")
        if D is not None:
            _tensor(D, "D", torch.float32, (ch,), dev)
        if dt_bias is not None:
            _tensor(dt_bias, "dt_bias", torch.float32, (ch,), dev)
        self.softplus = int(bool(softplus))

    def describe(self, N, x, dt, A, B, C, D, z, dt_bias, cu_seqlens):
        """These tensors, copied where the library cannot read them as they are,
        and their descriptor."""
        n = len(self.lead)
        x, xs = _channel_rows(x, n)
        dt, dts = _channel_rows(dt, n)
        z, zs = _channel_rows(z, n)
        if self.grouped:
            (B, bs), (C, cs) = _rows(B, n, _MOST_STRIDE), _rows(C, n, _MOST_STRIDE)
        else:
            (B, bs), (C, cs) = _channel_rows(B, n), _channel_rows(C, n)
        A, D, dt_bias, cu_seqlens = A.contiguous(), _whole(D), _whole(dt_bias), _whole(cu_seqlens)
        return (x, dt, A, B, C, D, z, dt_bias, cu_seqlens), dl_ssm_desc(
            self.dti, self.T, N, self.C, self.S, self.G, self.softplus, xs, dts, zs, bs, cs, _p(cu_seqlens),
            x.data_ptr(), dt.data_ptr(), _p(z), B.data_ptr(), C.data_ptr(), A.data_ptr(), _p(D), _p(dt_bias))

    def forward(self, desc, x, A, N, initial, saved=None):
        n = dl_ssm_workspace_bytes(desc)
        if n == 0:
            raise ValueError(f"unsupported scan shape tokens={self.T} sequences={N} channels={self.C} states={self.S} "
                             f"groups={self.G}")
        y, end, ws = _like(x), A.new_empty((N, self.C, self.S)), _scratch(n, A)
        _check(_lib.dl_ssm_scan(desc, _p(initial), end.data_ptr(), y.data_ptr(), _p(saved), ws.data_ptr(),
                                _current(self.device)), "dl_ssm_scan")
        return y, end


class _SsmFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, s, N, cu_seqlens, x, dt, A, B, C, D, z, dt_bias, initial):
        tensors, desc = s.describe(N, x, dt, A, B, C, D, z, dt_bias, cu_seqlens)
        saved = _scratch(dl_ssm_saved_bytes(desc), A)
        out = s.forward(desc, x, A, N, initial, saved)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(*tensors, saved)
        ctx.ssm, ctx.N = s, N
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, d_end):
        s, N = ctx.ssm, ctx.N
        *tensors, saved = ctx.saved_tensors
        with _on(s.device, None):
            (x, dt, A, B, C, D, z, dt_bias, cu_seqlens), desc = s.describe(N, *tensors)
            dy = torch.zeros((*s.lead, s.C), dtype=s.dtype, device=s.device) if dy is None else dy.contiguous()
            d_end = _whole(d_end)
            dx, ddt, dB, dC, dA = (_like(t) for t in (x, dt, B, C, A))
            dz = _like(z)
            dD = _like(D) if ctx.needs_input_grad[8] else None
            dbias = _like(dt_bias) if ctx.needs_input_grad[10] else None
            d0 = A.new_empty((N, s.C, s.S)) if ctx.needs_input_grad[11] else None
            ws = _scratch(dl_ssm_backward_workspace_bytes(desc), A)
            _check(_lib.dl_ssm_scan_backward(desc, saved.data_ptr(), dy.data_ptr(), _p(d_end), dx.data_ptr(),
                                             ddt.data_ptr(), _p(dz), dB.data_ptr(), dC.data_ptr(), dA.data_ptr(),
                                             _p(dD), _p(dbias), _p(d0), ws.data_ptr(), _current(s.device)),
                   "dl_ssm_scan_backward")
        return None, None, None, dx, ddt, dA, dB, dC, dD, dz, dbias, d0


def ssm_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, initial_state=None, cu_seqlens=None,
             stream=None):
    """The selective state space recurrence over whole sequences: a diagonal state
    h [N] for each channel, with delta = softplus(dt + dt_bias) (``softplus``
    False: their sum) and channel c in group g = c // (C / G),

        h = exp(delta * A[c]) * h + delta * x * B[g];  y = (C[g] . h + D * x) * z * sigmoid(z)

    x, dt, z [T,C], B, C [T,N] or [T,G,N] (all bf16 or all fp32; rows may be slices
    of a projection), A [C,N], D, dt_bias [C] fp32; D, z (the output gate) and
    dt_bias may be None.  Sequences are packed and cu_seqlens given as for `scan`, or
    all rows have a leading dimension.  initial_state: one fp32 [C,N] per sequence
    (default: zero).  1 <= N <= 64.

    Returns y, shaped as x in its dtype, and the end states, fp32.  Rows of no
    sequence hold zeros, in y and in the gradients.  Differentiable by all of
    them.  A forward pass that will be differentiated keeps the state of every 16th
    token, and with z an fp32 [T,C], until its backward pass."""
    _plain("ssm_scan", x, dt, A, B, C, D, z, dt_bias, initial_state)
    dev = _gpu(x, "x")
    s = _Ssm(x, dt, A, B, C, D, z, dt_bias, softplus)
    N = _sequences(s.lead, cu_seqlens, dev)
    if initial_state is not None:
        _tensor(initial_state, "initial_state", torch.float32, (N, s.C, s.S), dev)
    with _on(dev, stream):
        initial = _whole(initial_state)
        if _wants_grad(x, dt, A, B, C, D, z, dt_bias, initial):
            return _SsmFn.apply(s, N, cu_seqlens, x, dt, A, B, C, D, z, dt_bias, initial)
        tensors, desc = s.describe(N, x, dt, A, B, C, D, z, dt_bias, cu_seqlens)
        return s.forward(desc, x, A, N, initial)


def ssm_step(x, dt, state, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, rows=None, stream=None):
    """`ssm_scan` for one token of each of B requests: x, dt, z [B,C], B, C [B,N] or
    [B,G,N], and ``state`` [S,C,N] fp32 (a cache of states, contiguous), of which the
    tokens' rows are moved on in place: rows[b] (GPU, int32, no row twice; default:
    row b).  A row outside the cache (a padded batch's, -1) counts as zero and is not
    written.  Returns y [B,C].  For inference: it has no gradient and refuses
    inputs that want one."""
    _plain("ssm_step", x, dt, state, A, B, C, D, z, dt_bias)
    dev = _gpu(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x: want [B,C], got {tuple(x.shape)}")
    s = _Ssm(x, dt, A, B, C, D, z, dt_bias, softplus)
    _in_place(state, "state", torch.float32, (s.C, s.S), dev)
    _state_rows(rows, s.T, state, dev)
    _no_grad("ssm_step", x, dt, state, A, B, C, D, z, dt_bias)
    with _on(dev, stream):
        tensors, desc = s.describe(1, x, dt, A, B, C, D, z, dt_bias, None)
        y, rows = _like(x), _whole(rows)
        _check(_lib.dl_ssm_step(desc, state.data_ptr(), _p(rows), state.shape[0], y.data_ptr(), _current(dev)),
               "dl_ssm_step")
        _changed(state)
        return y
