"""The sequence operators beside the decode step, on torch tensors: `scan` (the
recurrence over whole sequences: prefill and training), `gated_norm` and
`residual_norm` (the norms behind and before a recurrent block).

Argument checks, output and workspace allocation and autograd nodes only: the
arithmetic is in libdeltalog (dl_scan, dl_gated_norm, dl_residual_norm and
their backward passes).  All three are differentiable once (in reverse;
forward-mode derivatives and tracing are refused), asynchronous on the current
stream (or ``stream``, on which their outputs are then allocated too; the
inputs have to be ready there, as for torch's own operators) and capturable
into HIP graphs.  Before a backward pass is captured, drop what
still refers to the graph of an eager pass over the same leaves (its loss and
outputs): torch ties a leaf's gradient to the stream of the oldest one.
Tensors may be on any one GPU.
"""
from __future__ import annotations

import contextlib
import sys

import torch
import torch.autograd.forward_ad as _forward_ad

from . import (DTYPES, _check, _dtype_id, _lib, _op_id, dl_gated_norm_workspace_bytes,
               dl_residual_norm_workspace_bytes, dl_scan_backward_workspace_bytes, dl_scan_desc,
               dl_scan_saved_bytes, dl_scan_workspace_bytes)

_HERE = contextlib.nullcontext()


def _on(device, stream):
    """The context of a call: its device current, and `stream` (a torch stream
    or a raw handle) in place of the current one, so that what is allocated
    belongs to it."""
    if stream is None:
        return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)
    if not isinstance(stream, int) and getattr(stream, "device", None) != device:
        raise ValueError(f"stream: want a stream of {device}, got {stream}")
    ctx = contextlib.ExitStack()
    ctx.enter_context(torch.cuda.device(device))
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    ctx.enter_context(torch.cuda.stream(stream))
    return ctx


def _current(device):
    """The raw handle of a device's current stream."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _plain(name, *tensors):
    """Refuse the transforms that would take a call of the library for no
    operation at all: forward-mode derivatives would come out as zero, and a
    traced function would return memory that nothing has written."""
    if _forward_ad._current_level >= 0 and any(
            isinstance(t, torch.Tensor) and _forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError(f"{name} has no forward-mode derivative")
    proxies = sys.modules.get("torch.fx.experimental.proxy_tensor")
    if torch._C._get_tracing_state() is not None or (proxies is not None and proxies.get_proxy_mode() is not None):
        raise NotImplementedError(f"{name} cannot be traced")


def _wants_grad(*tensors):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _bytes(n, device):
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device)


def _tensor(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is required")
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name}: want {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, want {device}")


def _gpu(t, name):
    """The device of a tensor that has to be on a GPU."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: want a GPU tensor")
    return t.device


def _p(t):
    return None if t is None else t.data_ptr()


def _none(t, name, why):
    if t is not None:
        raise ValueError(f"{name}: {why} takes none")


def _count(rows):
    """The library counts rows in an int."""
    if rows >= 1 << 31:
        raise ValueError(f"{rows} rows: want fewer than 2^31")
    return rows


def _state(t):
    """t as the library takes states: contiguous, and on a 16-byte boundary,
    where a view of something larger (an entry of a flat cache, a gradient
    that torch.cat's backward pass cuts out) need not be."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


_MOST_STRIDE = 1 << 22  # elements from one token's row to the next, as dl_scan takes them


def _rows(t, lead, most=None):
    """t [*lead, H, d] as rows of H*d elements a fixed distance apart, of
    ``most`` at the most: the tensor (copied only if it is not laid out so)
    and that distance."""
    H, d = t.shape[-2:]
    if t.is_contiguous():
        return t, H * d
    n = t.numel() // (H * d) if t.numel() else 0
    if n <= 1:
        return t.contiguous(), H * d
    inner = (d == 1 or t.stride(-1) == 1) and (H == 1 or t.stride(-2) == d)
    step = next((t.stride(i) for i in reversed(range(lead)) if t.shape[i] > 1), H * d)
    outer, span = True, step
    for i in reversed(range(lead)):
        if t.shape[i] > 1 and t.stride(i) != span:
            outer = False
        span *= t.shape[i]
    if inner and outer and step >= H * d and (most is None or step <= most):
        return t, step
    return t.contiguous(), H * d


# --------------------------------------------------------------------- scan --

class _Scan:
    """The checked arguments of one scan, and its descriptor for the library."""

    def __init__(self, op, q, k, v, beta, log_decay, u, cu_seqlens):
        opi = _op_id(op)
        if q.dim() not in (3, 4):
            raise ValueError(f"q: want [T,H,d_k] or [N,T,H,d_k], got {tuple(q.shape)}")
        dev, lead = q.device, tuple(q.shape[:-2])
        H, dk = q.shape[-2:]
        dti = _dtype_id(q.dtype)
        if not isinstance(v, torch.Tensor) or v.dim() != q.dim():
            raise ValueError("v: want as many dimensions as q")
        dv = v.shape[-1]
        _tensor(k, "k", q.dtype, (*lead, H, dk), dev)
        _tensor(v, "v", q.dtype, (*lead, H, dv), dev)
        if op == "rwkv6":
            _none(beta, "beta", op)
            _tensor(u, "u", torch.float32, (H, dk), dev)
        else:
            _none(u, "u", op)
            _tensor(beta, "beta", torch.float32, (*lead, H), dev)
        _tensor(log_decay, "log_decay", torch.float32, (*lead, H) if op == "gdn" else (*lead, H, dk), dev)
        if cu_seqlens is not None:
            if q.dim() != 3:
                raise ValueError("cu_seqlens goes with packed tensors [T,H,d]")
            if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
                raise ValueError("cu_seqlens: want a 1-D int32 GPU tensor of at least two offsets")
            _tensor(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, dev)
            cu_seqlens = cu_seqlens.contiguous()
        if H < 1:
            raise ValueError("q: want at least one head")
        self.N = cu_seqlens.numel() - 1 if cu_seqlens is not None else lead[0] if len(lead) == 2 else 1
        if self.N < 1:
            raise ValueError("want at least one sequence")
        T = _count(q.numel() // (H * dk) if q.numel() else 0)
        self.op, self.device, self.dtype, self.H, self.dk, self.dv = op, dev, q.dtype, H, dk, dv
        self.shape = dict(q=q.shape, v=v.shape, h=(*lead, H), ld=log_decay.shape)
        self.sizes = (opi, dti, T, self.N, H, dk, dv)
        # the tensors are kept alive with the descriptor
        self.tensors, self.desc = self.describe(
            *(None if t is None else t.detach() for t in (q, k, v, beta, log_decay, u)), cu_seqlens)
        self.workspace_bytes = dl_scan_workspace_bytes(self.desc)
        if self.workspace_bytes == 0:
            raise ValueError(f"unsupported scan shape {op} tokens={T} sequences={self.N} H={H} d_k={dk} d_v={dv}")

    def describe(self, q, k, v, beta, log_decay, u, cu_seqlens):
        """These tensors, copied where the library cannot read them as they
        are, and their descriptor."""
        (q, qs), (k, ks), (v, vs) = (_rows(t, len(self.shape["h"]) - 1, _MOST_STRIDE) for t in (q, k, v))
        beta, log_decay, u = (None if t is None else t.contiguous() for t in (beta, log_decay, u))
        return (q, k, v, beta, log_decay, u, cu_seqlens), dl_scan_desc(
            *self.sizes, qs, ks, vs, _p(cu_seqlens), q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(beta),
            log_decay.data_ptr(), _p(u))

    def state_shape(self):
        return (self.N, self.H, self.dk, self.dv)

    def empty(self, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def forward(self, initial, final, rows, n_rows, saved=None):
        o = self.empty(self.shape["v"], self.dtype)
        ws = _bytes(self.workspace_bytes, self.device)
        _check(_lib.dl_scan(self.desc, _p(initial), _p(final), _p(rows), n_rows, o.data_ptr(), _p(saved),
                            ws.data_ptr(), _current(self.device)), "dl_scan")
        return o


class _ScanFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, s, q, k, v, beta, log_decay, u, initial):
        final = s.empty(s.state_shape(), torch.float32)
        saved = _bytes(dl_scan_saved_bytes(s.desc), s.device)
        o = s.forward(initial, final, None, 0, saved)
        ctx.set_materialize_grads(False)
        # guarded against changes, and free to move until they are used
        # (checkpoints, offloading): the backward pass describes them anew
        ctx.save_for_backward(*s.tensors, saved)
        ctx.scan, ctx.with_initial = s, initial is not None
        s.tensors = s.desc = None
        return o, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_o, d_final):
        s = ctx.scan
        *tensors, saved = ctx.saved_tensors
        with _on(s.device, None):
            tensors, desc = s.describe(*tensors)
            d_o = None if d_o is None else d_o.contiguous()
            d_final = None if d_final is None else _state(d_final)
            delta = s.op != "rwkv6"
            dq, dk = s.empty(s.shape["q"], s.dtype), s.empty(s.shape["q"], s.dtype)
            dv = s.empty(s.shape["v"], s.dtype)
            dbeta = s.empty(s.shape["h"], torch.float32) if delta else None
            dld = s.empty(s.shape["ld"], torch.float32)
            du = None if delta else s.empty((s.H, s.dk), torch.float32)
            d0 = s.empty(s.state_shape(), torch.float32) if ctx.with_initial else None
            ws = _bytes(dl_scan_backward_workspace_bytes(desc), s.device)
            _check(_lib.dl_scan_backward(desc, saved.data_ptr(), _p(d_o), _p(d_final), dq.data_ptr(), dk.data_ptr(),
                                         dv.data_ptr(), _p(dbeta), dld.data_ptr(), _p(du), _p(d0), ws.data_ptr(),
                                         _current(s.device)), "dl_scan_backward")
        return None, dq, dk, dv, dbeta, dld, du, d0


def _initial(initial_state, shape, device):
    if initial_state is None:
        return None
    _tensor(initial_state, "initial_state", torch.float32, shape, device)
    return _state(initial_state)


def scan(op: str, q, k, v, beta, log_decay, u=None, initial_state=None, cu_seqlens=None, stream=None):
    """The recurrence of `DeltaLogState.step` over whole sequences.

    q (r for RWKV6), k [T,H,d_k], v [T,H,d_v] (bf16 or fp32), beta [T,H] fp32
    (None for RWKV6), log_decay fp32 [T,H] (GDN) or [T,H,d_k], u [H,d_k] fp32
    (RWKV6 only): N sequences packed one after the other, sequence n being the
    rows cu_seqlens[n] to cu_seqlens[n+1] (GPU, int32; default: one sequence).
    Or all with a leading N: N sequences of equal length.  Rows of q, k and v
    may be slices of one wider projection.  initial_state [N,H,d_k,d_v] fp32
    (default: zero).

    Returns o, shaped as v in the input dtype, and the end states
    [N,H,d_k,d_v] fp32.  Rows ahead of the first sequence and behind the last
    hold zeros, in o and in the gradients.  d_k, d_v in {16, 32, 64, 128}.

    Differentiable by q, k, v, beta, log_decay, u and initial_state.  A forward
    pass that will be differentiated keeps, per 64 tokens and head, the state
    and 64 d_v floats until its backward pass."""
    _plain("scan", q, k, v, beta, log_decay, u, initial_state)
    with _on(_gpu(q, "q"), stream):
        probe = _Scan(op, q, k, v, beta, log_decay, u, cu_seqlens)
        initial = _initial(initial_state, probe.state_shape(), probe.device)
        if _wants_grad(q, k, v, beta, log_decay, u, initial):
            return _ScanFn.apply(probe, q, k, v, beta, log_decay, u, initial)
        final = probe.empty(probe.state_shape(), torch.float32)
        return probe.forward(initial, final, None, 0), final


def _prefill(st, q, k, v, beta, log_decay, cu_seqlens, slots, stream):
    _plain("prefill", q, k, v, beta, log_decay)
    with _on(_gpu(q, "q"), stream):
        return _prefill_here(st, q, k, v, beta, log_decay, cu_seqlens, slots)


def _prefill_here(st, q, k, v, beta, log_decay, cu_seqlens, slots):
    s = _Scan(st.op, q, k, v, beta, log_decay, st.u, cu_seqlens)
    if (s.H, s.dk, s.dv, s.dtype) != (st.H, st.d_k, st.d_v, st.dtype):
        raise ValueError(f"prefill: the state has H={st.H} d_k={st.d_k} d_v={st.d_v} {st.dtype}, the inputs "
                         f"H={s.H} d_k={s.dk} d_v={s.dv} {s.dtype}")
    if s.device != st.base.device:
        raise ValueError(f"q is on {s.device}, the state on {st.base.device}")
    if slots is None:
        if s.N != st.B:
            raise ValueError(f"prefill: {s.N} prompts for {st.B} slots: name their slots")
        names = range(st.B)
    else:
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("slots: their list cannot be copied to the GPU while a graph is captured")
        names = [int(i) for i in slots]
        if len(names) != s.N or len(set(names)) != s.N or not all(0 <= i < st.B for i in names):
            raise ValueError(f"slots: want {s.N} distinct slots below {st.B}, got {names}")
    if any(st.slot_log_len(i) != 0 for i in (names if st._per_slot else names[:1])):
        raise ValueError("prefill: a slot's log holds entries; merge it first")
    rows = None if slots is None else torch.tensor(names, dtype=torch.int32, device=s.device)
    return s.forward(st.base, st.base, rows, st.B)


# -------------------------------------------------------------------- norms --

def _gated_norm(o, gate, weight, eps):
    """y, and what its backward pass needs."""
    H, d = o.shape[-2:]
    rows = _count(o.numel() // (H * d))
    o = o.contiguous()
    g, gs = _rows(gate, gate.dim() - 2)
    weight = None if weight is None else weight.contiguous()
    y = torch.empty(gate.shape, dtype=gate.dtype, device=o.device)
    _check(_lib.dl_gated_norm(rows, H, d, DTYPES[o.dtype], DTYPES[gate.dtype], o.data_ptr(), g.data_ptr(), gs,
                              _p(weight), eps, y.data_ptr(), _current(o.device)), "dl_gated_norm")
    return y, (o, g, weight), (rows, H, d, eps)


class _GatedNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, o, gate, weight, eps):
        y, saved, ctx.args = _gated_norm(o, gate, weight, eps)
        ctx.save_for_backward(*saved)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        o, g, weight = ctx.saved_tensors
        rows, H, d, eps = ctx.args
        with _on(o.device, None):
            g, gs = _rows(g, g.dim() - 2)  # its layout may be another than when it was saved
            dy = dy.contiguous()
            d_o = torch.empty_like(o)
            dg = torch.empty(dy.shape, dtype=g.dtype, device=o.device)
            dw = ws = None
            if weight is not None and ctx.needs_input_grad[2]:
                dw = torch.empty_like(weight)
                ws = _bytes(dl_gated_norm_workspace_bytes(rows, H, d), o.device)
            _check(_lib.dl_gated_norm_backward(rows, H, d, DTYPES[o.dtype], DTYPES[g.dtype], o.data_ptr(),
                                               g.data_ptr(), gs, _p(weight), eps, dy.data_ptr(), d_o.data_ptr(),
                                               dg.data_ptr(), _p(dw), _p(ws), _current(o.device)),
                   "dl_gated_norm_backward")
        return d_o, dg, dw, None


def gated_norm(o, gate, weight=None, eps: float = 1e-6, stream=None):
    """rms(o) * weight * silu(gate) per head, rms(a) = a / sqrt(mean(a^2) +
    eps) over the last dimension: the norm behind the recurrence with its
    output gate.  o [...,H,d] fp32 (from `step`) or bf16 (from `scan`), gate
    [...,H,d] bf16 or fp32 (its rows may be slices of a projection), weight
    [d] fp32 or None.  Returns gate's dtype.  d in {16, 32, 64, 128}.
    Differentiable by o, gate and weight."""
    _plain("gated_norm", o, gate, weight)
    dev = _gpu(o, "o")
    _gpu(gate, "gate")
    _dtype_id(o.dtype), _dtype_id(gate.dtype)
    _tensor(gate, "gate", gate.dtype, o.shape, dev)
    if o.dim() < 2 or o.shape[-1] not in (16, 32, 64, 128) or o.shape[-2] < 1:
        raise ValueError(f"o: want heads of 16, 32, 64 or 128, got {tuple(o.shape)}")
    if weight is not None:
        _tensor(weight, "weight", torch.float32, (o.shape[-1],), o.device)
    with _on(o.device, stream):
        if _wants_grad(o, gate, weight):
            return _GatedNormFn.apply(o, gate, weight, float(eps))
        return _gated_norm(o, gate, weight, float(eps))[0]


def _residual_norm(x, y, scale, weight, eps, dtype):
    """x' (None without y) and h, and what their backward pass needs."""
    D = x.shape[-1]
    rows = _count(x.numel() // D)
    x, y, scale, weight = (None if t is None else t.contiguous() for t in (x, y, scale, weight))
    x_out = None if y is None else torch.empty_like(x)
    h = torch.empty(x.shape, dtype=dtype, device=x.device)
    _check(_lib.dl_residual_norm(rows, D, DTYPES[dtype], x.data_ptr(), _p(y), _p(scale), _p(weight), eps, _p(x_out),
                                 h.data_ptr(), _current(x.device)), "dl_residual_norm")
    return (x_out, h), (x if y is None else x_out, y if scale is not None else None, scale, weight), \
        (rows, D, eps, dtype, y is not None)


class _ResidualNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, scale, weight, eps, dtype):
        out, saved, ctx.args = _residual_norm(x, y, scale, weight, eps, dtype)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(*saved)
        return out[1] if y is None else out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, *grads):
        x, y, scale, weight = ctx.saved_tensors
        rows, D, eps, dtype, added = ctx.args
        d_x_out, d_h = grads if added else (None, grads[0])
        with _on(x.device, None):
            d_x_out = None if d_x_out is None else d_x_out.contiguous()
            d_h = None if d_h is None else d_h.contiguous()
            dx = torch.empty_like(x)
            dy = torch.empty(x.shape, dtype=dtype, device=x.device) if added else None
            ds = torch.empty_like(scale) if scale is not None and ctx.needs_input_grad[2] else None
            dw = torch.empty_like(weight) if weight is not None and ctx.needs_input_grad[3] else None
            ws = None
            if ds is not None or dw is not None:
                ws = _bytes(dl_residual_norm_workspace_bytes(rows, D), x.device)
            _check(_lib.dl_residual_norm_backward(rows, D, DTYPES[dtype], x.data_ptr(), _p(y), _p(scale), _p(weight),
                                                  eps, _p(d_x_out), _p(d_h), dx.data_ptr(), _p(dy), _p(ds), _p(dw),
                                                  _p(ws), _current(x.device)), "dl_residual_norm_backward")
        return dx, dy, ds, dw, None, None


def residual_norm(x, y=None, scale=None, weight=None, eps: float = 1e-6, dtype=None, stream=None):
    """x' = x + scale * y and h = rms(x') * weight over the last dimension: the
    residual add behind one block with its per-channel scale, and the norm
    before the next.  x [...,D] fp32 (the residual stream), y [...,D] bf16 or
    fp32, scale and weight [D] fp32 or None; D <= 16384.  Returns (x', h), h in
    y's dtype.  Without y (the first norm): (x, h) with h = rms(x) * weight in
    ``dtype`` (default bf16).  Differentiable by x, y, scale and weight."""
    _plain("residual_norm", x, y, scale, weight)
    _gpu(x, "x")
    if x.dim() < 1 or x.dtype != torch.float32:
        raise ValueError(f"x: want fp32 [...,D], got {x.dtype} {tuple(x.shape)}")
    D = x.shape[-1]
    if not 1 <= D <= 16384:
        raise ValueError(f"x: want 1 to 16384 columns, got {D}")
    if y is None:
        if scale is not None:
            raise ValueError("scale goes with y")
        dtype = torch.bfloat16 if dtype is None else dtype
        _dtype_id(dtype)
    else:
        if not isinstance(y, torch.Tensor):
            raise ValueError("y: want a GPU tensor shaped as x")
        _dtype_id(y.dtype)
        _tensor(y, "y", y.dtype, x.shape, x.device)
        if dtype is not None and dtype != y.dtype:
            raise ValueError(f"dtype: h has y's type, {y.dtype}")
        dtype = y.dtype
    for t, name in ((scale, "scale"), (weight, "weight")):
        if t is not None:
            _tensor(t, name, torch.float32, (D,), x.device)
    with _on(x.device, stream):
        if not _wants_grad(x, y, scale, weight):
            out = _residual_norm(x, y, scale, weight, float(eps), dtype)[0]
            return (x, out[1]) if y is None else out
        out = _ResidualNormFn.apply(x, y, scale, weight, float(eps), dtype)
        return (x, out) if y is None else out
