"""Python binding of the block operators of libs6 (include/s6_block.h): the
multi-head selective scan with its gradients and single-token step, and the
norms before and after it.

As in ``s6``: argument marshalling only, torch device tensors in and out, work
enqueued on the current stream of the tensors' device.  ``HeadsScan``,
``AddNorm`` and ``GatedNorm`` are the same operators for torch autograd (once
differentiable: a gradient of their gradients is an error).
"""
from __future__ import annotations

import ctypes
import math

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import s6
from .s6 import _DT, _check

S6_DELTA_SOFTPLUS, S6_UNIT_INPUT, S6_GATE_AFTER = 1, 4, 8
MAX_DSTATE = 128


class HeadsDims(ctypes.Structure):
    """s6_heads_dims of include/s6_block.h."""

    _fields_ = [(n, ctypes.c_int64) for n in
                ("batch", "seqlen", "heads", "headdim", "groups", "dstate", "x_batch", "x_token", "delta_batch",
                 "delta_token", "b_batch", "b_token", "c_batch", "c_token")]


_lib = None


def _load():
    global _lib
    if _lib is None:
        lib = s6.load_library()
        i64, vp, i32, f32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        dims, szp = ctypes.POINTER(HeadsDims), ctypes.POINTER(ctypes.c_size_t)
        ws = [vp, sz, vp]  # workspace, workspace_bytes, stream
        for name, args in {
            "s6_heads_scan_fwd": [dims, i32, i32] + [vp] * 10 + ws,
            "s6_heads_scan_fwd_workspace_size": [dims, i32, szp],
            "s6_heads_scan_bwd": [dims, i32, i32] + [vp] * 18 + ws,
            "s6_heads_scan_bwd_workspace_size": [dims, i32, szp],
            "s6_heads_state_update": [dims, i32, i32] + [vp] * 10,
            "s6_add_norm_fwd": [i64, i64, i32, i32, vp, i64, vp, vp, vp, f32, f32, vp, vp, vp],
            "s6_add_norm_bwd": [i64, i64, i32, i32, vp, vp, vp, vp, i64, vp, vp, f32, f32, vp, vp, vp, vp] + ws,
            "s6_add_norm_bwd_workspace_size": [i64, i64, szp],
            "s6_gated_norm_fwd": [i64, i64, i64, i32, i32, vp, i64, vp, i64, vp, f32, vp, vp],
            "s6_gated_norm_bwd": [i64, i64, i64, i32, i32, vp, vp, i64, vp, i64, vp, f32, vp, vp, vp] + ws,
            "s6_gated_norm_bwd_workspace_size": [i64, i64, i64, szp],
        }.items():
            fn = getattr(lib, name)
            fn.restype = i32
            fn.argtypes = args
        _lib = lib
    return _lib


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# The handle of the current stream without a Stream object around it, where
# this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _launch(fn, like, *args):
    """fn(*args, stream) on `like`'s device and its current stream."""
    index = like.device.index
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc:
        _check(rc)


def _at(t):
    return None if t is None else t.data_ptr()


def _same_device(first, *others):
    """The kernels run on the device of `first`: every tensor has to be there."""
    d = first.device
    for t in others:
        if t is not None and t.device != d:
            raise ValueError(f"tensors on {d} and {t.device}")


def _written(*tensors):
    """Tells autograd of tensors of the caller that a kernel writes: a backward
    that saved one of them then refuses what is no longer its value."""
    for t in tensors:
        if t is not None:
            increment_version(t)


def _workspace(query, like, *args):
    """(tensor, pointer, bytes) of a fresh workspace on the current stream."""
    out = ctypes.c_size_t(0)
    index = like.device.index
    if torch.cuda.current_device() == index:
        rc = query(*args, ctypes.byref(out))
    else:
        with torch.cuda.device(index):
            rc = query(*args, ctypes.byref(out))
    if rc:
        _check(rc)
    if out.value == 0:
        return None, None, 0
    t = torch.empty(out.value, dtype=torch.uint8, device=like.device)
    return t, t.data_ptr(), out.value


def _dtype(t, name="x"):
    if t.dtype not in _DT:
        raise ValueError(f"unsupported {name} dtype {t.dtype}")
    return t.dtype


def _need(t, name, shape, dtype):
    """A device tensor of this shape and type (the shape as a tuple or Size)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return t


def _whole(t, name, shape, dtype=torch.float32):
    """As _need, and contiguous; None passes."""
    if t is None:
        return
    if t.shape != shape or t.dtype is not dtype or not t.is_cuda:
        _need(t, name, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t, name, shape, dtype, inner):
    """Strides of the leading dimensions of a device tensor whose last
    `inner` dimensions are contiguous: the leading ones may be strided (slices
    of wider rows)."""
    if t is None or t.shape != shape or t.dtype is not dtype or not t.is_cuda:
        _need(t, name, shape, dtype)
    st = t.stride()
    if t.is_contiguous():
        return st[:-inner]
    lead = len(shape) - inner
    want = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if st[i] != want and shape[i] != 1:
            raise ValueError(f"{name}'s rows must be contiguous")
        want *= shape[i]
    # a stride along a single element is never taken
    return tuple(v if n > 1 else want for v, n in zip(st, shape[:lead]))


def _heads_dims(x, delta, A, Bm, Cm, D, delta_bias, delta_softplus, unit_input, tokens):
    dt = _dtype(x)
    if x.dim() != (4 if tokens else 3) or Bm is None or Bm.dim() != x.dim():
        raise ValueError("x is (batch, seqlen, heads, headdim), Bm and Cm (batch, seqlen, groups, dstate); without "
                         "seqlen for a single token")
    shape = x.shape
    lead, (heads, headdim), (groups, dstate) = shape[:-2], shape[-2:], Bm.shape[-2:]
    gshape = (*lead, groups, dstate)
    xs = _rows(x, "x", shape, dt, 2)
    bs = _rows(Bm, "Bm", gshape, dt, 2)
    cs = _rows(Cm, "Cm", gshape, dt, 2)
    if delta is None:
        if delta_bias is not None or delta_softplus:
            raise ValueError("delta_bias and delta_softplus need a delta")
        ds = (0, 0) if tokens else (0,)
    else:
        ds = _rows(delta, "delta", (*lead, heads), dt, 1)
    if A is None:
        raise ValueError("A is required")
    _whole(A, "A", (heads,))
    _whole(D, "D", (heads,))
    _whole(delta_bias, "delta_bias", (heads,))
    _same_device(x, delta, A, Bm, Cm, D, delta_bias)
    if tokens:
        dims = HeadsDims(*lead, heads, headdim, groups, dstate, *xs, *ds, *bs, *cs)
    else:
        dims = HeadsDims(lead[0], 1, heads, headdim, groups, dstate, xs[0], 0, ds[0], 0, bs[0], 0, cs[0], 0)
    flags = (S6_DELTA_SOFTPLUS if delta_softplus else 0) | (S6_UNIT_INPUT if unit_input else 0)
    return dims, _DT[dt], flags


def heads_scan_fwd(x, delta, A, Bm, Cm, D=None, h0=None, return_last_state=False, delta_bias=None,
                   delta_softplus=False, unit_input=False, y=None, h_last=None):
    """Multi-head selective scan (linear attention with a decay per head).
    x: (batch, L, heads, headdim); delta: (batch, L, heads) or None (a step of
    1: one fixed decay exp(A) per head); Bm, Cm: (batch, L, groups, N), N <=
    128, groups a divisor of heads; A, D, delta_bias: (heads,) fp32; h0:
    (batch, heads, headdim, N) fp32.  x, delta, Bm, Cm share one dtype
    (float32 or bfloat16) and may be slices of wider rows.  unit_input: the
    input term is x B instead of step x B.  Returns y like x (contiguous), and
    h_last (batch, heads, headdim, N) fp32 if requested."""
    dims, dt, flags = _heads_dims(x, delta, A, Bm, Cm, D, delta_bias, delta_softplus, unit_input, True)
    sshape = (dims.batch, dims.heads, dims.headdim, dims.dstate)
    _whole(h0, "h0", sshape)
    _whole(y, "y", x.shape, x.dtype)
    _whole(h_last, "h_last", sshape)
    _same_device(x, h0, y, h_last)
    _written(y, h_last)
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    if return_last_state and h_last is None:
        h_last = torch.empty(sshape, dtype=torch.float32, device=x.device)
    lib = _load()
    ref = ctypes.byref(dims)
    keep, wsp, wsn = _workspace(lib.s6_heads_scan_fwd_workspace_size, x, ref, dt)
    _launch(lib.s6_heads_scan_fwd, x, ref, dt, flags, _at(x), _at(delta), _at(delta_bias), _at(A), _at(Bm), _at(Cm),
            _at(D), _at(h0), _at(y), _at(h_last), wsp, wsn)
    del keep
    return (y, h_last) if return_last_state else y


def heads_scan_bwd(x, delta, A, Bm, Cm, dy, D=None, h0=None, dh_last=None, delta_bias=None, delta_softplus=False,
                   unit_input=False, skip=()):
    """Gradients of <dy, y> + <dh_last, h_last> for heads_scan_fwd with the
    same inputs.  dy: like y, contiguous; dh_last: like h_last or None.
    Returns a dict: dx, ddelta (where delta is given), dBm, dCm in the input
    dtype; dA, and where their input is given dD, ddelta_bias, dh0 in fp32.
    skip: names among the last three to leave out."""
    dims, dt, flags = _heads_dims(x, delta, A, Bm, Cm, D, delta_bias, delta_softplus, unit_input, True)
    sshape = (dims.batch, dims.heads, dims.headdim, dims.dstate)
    _whole(h0, "h0", sshape)
    _whole(dh_last, "dh_last", sshape)
    _whole(_need(dy, "dy", x.shape, x.dtype), "dy", x.shape, x.dtype)
    _same_device(x, h0, dh_last, dy)
    new = lambda t: torch.empty_like(t, memory_format=torch.contiguous_format)  # noqa: E731
    g = {"dx": new(x), "dBm": new(Bm), "dCm": new(Cm), "dA": new(A)}
    if delta is not None:
        g["ddelta"] = new(delta)
    for name, t in (("dD", D), ("ddelta_bias", delta_bias), ("dh0", h0)):
        if t is not None and name not in skip:
            g[name] = new(t)
    lib = _load()
    ref = ctypes.byref(dims)
    keep, wsp, wsn = _workspace(lib.s6_heads_scan_bwd_workspace_size, x, ref, dt)
    _launch(lib.s6_heads_scan_bwd, x, ref, dt, flags, _at(x), _at(delta), _at(delta_bias), _at(A), _at(Bm), _at(Cm),
            _at(D), _at(h0), _at(dy), _at(dh_last), _at(g["dx"]), _at(g.get("ddelta")), _at(g["dA"]), _at(g["dBm"]),
            _at(g["dCm"]), _at(g.get("dD")), _at(g.get("dh0")), _at(g.get("ddelta_bias")), wsp, wsn)
    del keep
    return g


def heads_state_update(h, x, delta, A, Bm, Cm, D=None, delta_bias=None, delta_softplus=False, unit_input=False, y=None):
    """One token of every sequence: h (batch, heads, headdim, N) fp32 is
    advanced in place; x: (batch, heads, headdim), delta: (batch, heads) or
    None, Bm, Cm: (batch, groups, N).  Returns y (batch, heads, headdim) in
    x's dtype."""
    dims, dt, flags = _heads_dims(x, delta, A, Bm, Cm, D, delta_bias, delta_softplus, unit_input, False)
    sshape = (*x.shape, Bm.shape[-1])
    _whole(_need(h, "h", sshape, torch.float32), "h", sshape)
    _whole(y, "y", x.shape, x.dtype)
    _same_device(x, h, y)
    _written(h, y)
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    _launch(_load().s6_heads_state_update, x, ctypes.byref(dims), dt, flags, _at(h), _at(x), _at(delta),
            _at(delta_bias), _at(A), _at(Bm), _at(Cm), _at(D), _at(y))
    return y


def _weight(w, dim):
    if w is None:
        raise ValueError("weight is required")
    _whole(w, "weight", (dim,))


def _flat(t, name, shape, dtype):
    """Row stride of a (..., dim) device tensor seen as rows of dim elements."""
    _need(t, name, shape, dtype)
    dim = shape[-1]
    if t.is_contiguous():
        return dim
    st = t.stride()
    if dim > 1 and st[-1] != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    stride = None  # one stride for all rows: that of the last leading dimension, the others a multiple of it
    size = 1
    for i in range(len(shape) - 2, -1, -1):
        if shape[i] == 1:
            continue
        if stride is None:
            stride = st[i]
        elif st[i] != stride * size:
            raise ValueError(f"{name}'s rows must lie at one stride")
        size *= shape[i]
    if stride is not None and stride < dim:
        raise ValueError(f"{name}'s rows must not overlap")
    return dim if stride is None else stride


def add_norm_fwd(x, weight, residual=None, gamma=None, scale=1.0, eps=1e-5, residual_dtype=None, out=None,
                 residual_out=None):
    """Residual add, residual scale and RMS norm before a block: r' = residual
    + scale * gamma * x, out = r' / sqrt(mean(r'^2) + eps) * weight over the
    last dimension.  x may be a slice of wider rows; weight, gamma: (dim,)
    fp32; residual: like x, in x's dtype or float32 (None: no residual yet, r'
    in residual_dtype, float32 unless given).  Returns (out in x's dtype,
    r' in the residual's dtype); residual_out may be the residual itself."""
    dt = _dtype(x)
    stride = _flat(x, "x", x.shape, dt)
    rt = residual.dtype if residual is not None else residual_dtype or torch.float32
    if rt not in (torch.float32, dt):
        raise ValueError(f"residual dtype {rt}: expected float32 or {dt}")
    dim = x.shape[-1]
    _whole(residual, "residual", x.shape, rt)
    _weight(weight, dim)
    _whole(gamma, "gamma", (dim,))
    _whole(out, "out", x.shape, dt)
    _whole(residual_out, "residual_out", x.shape, rt)
    _same_device(x, weight, residual, gamma, out, residual_out)
    _written(out, residual_out)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    if residual_out is None:
        residual_out = torch.empty_like(x, dtype=rt, memory_format=torch.contiguous_format)
    _launch(_load().s6_add_norm_fwd, x, math.prod(x.shape[:-1]), dim, _DT[dt], _DT[rt], _at(x), stride, _at(residual),
            _at(weight), _at(gamma), scale, eps, _at(out), _at(residual_out))
    return out, residual_out


def add_norm_bwd(dout, residual_out, weight, dresidual_out=None, x=None, gamma=None, scale=1.0, eps=1e-5, skip=()):
    """Gradients of <dout, out> + <dresidual_out, r'> for add_norm_fwd, from
    the r' it returned.  Returns a dict: dx (dout's dtype), dresidual (r''s
    dtype), dweight, and dgamma where gamma is given (then x is needed).
    skip: names among dx, dresidual and dweight, not all three, to leave out."""
    dt = _dtype(dout, "dout")
    rt = residual_out.dtype
    dim = dout.shape[-1]
    if rt not in (torch.float32, dt):
        raise ValueError(f"residual_out dtype {rt}: expected float32 or {dt}")
    _whole(_need(dout, "dout", dout.shape, dt), "dout", dout.shape, dt)
    _whole(residual_out, "residual_out", dout.shape, rt)
    _whole(dresidual_out, "dresidual_out", dout.shape, rt)
    _weight(weight, dim)
    _whole(gamma, "gamma", (dim,))
    stride = dim
    if gamma is not None:
        stride = _flat(x, "x", dout.shape, dt)
    _same_device(dout, residual_out, dresidual_out, weight, gamma, x)
    like = {"dx": dout, "dresidual": residual_out, "dweight": weight}
    g = {name: torch.empty_like(t) for name, t in like.items() if name not in skip}
    if gamma is not None:
        g["dgamma"] = torch.empty_like(gamma)
    lib = _load()
    rows = math.prod(dout.shape[:-1])
    keep, wsp, wsn = _workspace(lib.s6_add_norm_bwd_workspace_size, dout, rows, dim)
    _launch(lib.s6_add_norm_bwd, dout, rows, dim, _DT[dt], _DT[rt], _at(dout), _at(dresidual_out), _at(residual_out),
            _at(x) if gamma is not None else None, stride, _at(weight), _at(gamma), scale, eps, _at(g.get("dx")),
            _at(g.get("dresidual")), _at(g.get("dweight")), _at(g.get("dgamma")), wsp, wsn)
    del keep
    return g


def _gated_args(y, z, weight, groups):
    dt = _dtype(y, "y")
    dim = y.shape[-1]
    if groups < 1 or dim % groups:
        raise ValueError(f"{groups} groups do not divide {dim} columns")
    ys = _flat(y, "y", y.shape, dt)
    zs = dim if z is None else _flat(z, "z", y.shape, dt)
    _weight(weight, dim)
    _same_device(y, z, weight)
    return dt, dim, ys, zs


def gated_norm_fwd(y, z, weight, groups=1, gate_after=False, eps=1e-5, out=None):
    """SiLU gate and RMS norm after the scan, over groups of the last
    dimension: rms(y * SiLU(z)) * weight, or rms(y) * weight * SiLU(z) with
    gate_after.  y and z (None: no gate) may be slices of wider rows.  Returns
    a contiguous tensor in y's dtype."""
    dt, dim, ys, zs = _gated_args(y, z, weight, groups)
    _whole(out, "out", y.shape, dt)
    _same_device(y, out)
    _written(out)
    if out is None:
        out = torch.empty_like(y, memory_format=torch.contiguous_format)
    _launch(_load().s6_gated_norm_fwd, y, math.prod(y.shape[:-1]), dim, groups, _DT[dt],
            S6_GATE_AFTER if gate_after else 0, _at(y), ys, _at(z), zs, _at(weight), eps, _at(out))
    return out


def gated_norm_bwd(dout, y, z, weight, groups=1, gate_after=False, eps=1e-5, skip=()):
    """Gradients of <dout, out> for gated_norm_fwd: a dict of dy, dz (where z
    is given) in y's dtype and dweight in fp32 (left out where skip names it)."""
    dt, dim, ys, zs = _gated_args(y, z, weight, groups)
    _whole(_need(dout, "dout", y.shape, dt), "dout", y.shape, dt)
    _same_device(y, dout)
    g = {"dy": torch.empty_like(dout)}
    if "dweight" not in skip:
        g["dweight"] = torch.empty_like(weight)
    if z is not None:
        g["dz"] = torch.empty_like(dout)
    lib = _load()
    rows = math.prod(y.shape[:-1])
    keep, wsp, wsn = _workspace(lib.s6_gated_norm_bwd_workspace_size, y, rows, dim, groups)
    _launch(lib.s6_gated_norm_bwd, y, rows, dim, groups, _DT[dt], S6_GATE_AFTER if gate_after else 0, _at(dout),
            _at(y), ys, _at(z), zs, _at(weight), eps, _at(g["dy"]), _at(g.get("dz")), _at(g.get("dweight")), wsp, wsn)
    del keep
    return g


def _unasked(ctx, names):
    """The gradients that autograd does not ask for; names: theirs, in the order
    of apply's arguments (of which the last may not have been given)."""
    asked = ctx.needs_input_grad
    return [name for i, name in enumerate(names) if i >= len(asked) or not asked[i]]


class HeadsScan(torch.autograd.Function):
    """heads_scan_fwd with its gradients: y, h_last = HeadsScan.apply(x, delta,
    A, Bm, Cm, D, h0, delta_bias, delta_softplus, unit_input).  delta, D, h0 and
    delta_bias may be None.  The backward recomputes the states."""

    @staticmethod
    def forward(ctx, x, delta, A, Bm, Cm, D=None, h0=None, delta_bias=None, delta_softplus=False, unit_input=False):
        ctx.save_for_backward(x, delta, A, Bm, Cm, D, h0, delta_bias)
        ctx.opts = dict(delta_softplus=delta_softplus, unit_input=unit_input)
        ctx.set_materialize_grads(False)
        return heads_scan_fwd(x, delta, A, Bm, Cm, D=D, h0=h0, return_last_state=True, delta_bias=delta_bias, **ctx.opts)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh_last):
        x, delta, A, Bm, Cm, D, h0, delta_bias = ctx.saved_tensors
        dy = torch.zeros_like(x, memory_format=torch.contiguous_format) if dy is None else dy.contiguous()
        names = ("dx", "ddelta", "dA", "dBm", "dCm", "dD", "dh0", "ddelta_bias")
        g = heads_scan_bwd(x, delta, A, Bm, Cm, dy, D=D, h0=h0, delta_bias=delta_bias,
                           dh_last=None if dh_last is None else dh_last.contiguous(), skip=_unasked(ctx, names),
                           **ctx.opts)
        return (*(g.get(name) for name in names), None, None)


class AddNorm(torch.autograd.Function):
    """add_norm_fwd with its gradients: out, r' = AddNorm.apply(x, weight,
    residual, gamma, scale, eps); residual and gamma may be None."""

    @staticmethod
    def forward(ctx, x, weight, residual=None, gamma=None, scale=1.0, eps=1e-5):
        out, res = add_norm_fwd(x, weight, residual=residual, gamma=gamma, scale=scale, eps=eps)
        ctx.save_for_backward(res, weight, gamma, x if gamma is not None else None)
        ctx.scale, ctx.eps, ctx.dt = scale, eps, x.dtype
        ctx.set_materialize_grads(False)
        return out, res

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dres):
        res, weight, gamma, x = ctx.saved_tensors
        dout = torch.zeros(res.shape, dtype=ctx.dt, device=res.device) if dout is None else dout.contiguous()
        names = ("dx", "dweight", "dresidual", "dgamma")
        skip = _unasked(ctx, names)
        if len(set(skip) - {"dgamma"}) == 3:  # gamma's alone is asked for: one of the others comes with it
            skip.remove("dweight")
        g = add_norm_bwd(dout, res, weight, dresidual_out=None if dres is None else dres.contiguous(), x=x, gamma=gamma,
                         scale=ctx.scale, eps=ctx.eps, skip=skip)
        return (*(g.get(name) for name in names), None, None)


class GatedNorm(torch.autograd.Function):
    """gated_norm_fwd with its gradients: out = GatedNorm.apply(y, z, weight,
    groups, gate_after, eps); z may be None."""

    @staticmethod
    def forward(ctx, y, z, weight, groups=1, gate_after=False, eps=1e-5):
        ctx.save_for_backward(y, z, weight)
        ctx.opts = dict(groups=groups, gate_after=gate_after, eps=eps)
        return gated_norm_fwd(y, z, weight, **ctx.opts)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, z, weight = ctx.saved_tensors
        names = ("dy", "dz", "dweight")
        g = gated_norm_bwd(dout.contiguous(), y, z, weight, skip=_unasked(ctx, names), **ctx.opts)
        return (*(g.get(name) for name in names), None, None, None)
