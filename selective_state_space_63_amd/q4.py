"""Python binding of the projections in few bits (include/s6_q4.h): products
with 4-bit weights and group scales, their packing, and the norm before a
block with an 8-bit output.

As in ``block``: argument marshalling only, torch device tensors in and out,
work enqueued on the current stream of the tensors' device.  These operators are
for answering, not for training: they have no gradients, and q4_linear and
add_norm_q8_fwd refuse inputs that ask for one (unless under torch.no_grad).
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import s6
from .block import _at, _dtype, _flat, _launch, _plain, _same_device, _weight, _whole, _workspace, _written
from .s6 import _DT

S6_E4M3 = 2
GROUPS = (32, 64, 128)
FEW = {torch.float32: 6, torch.bfloat16: 16, torch.float8_e4m3fn: 16}  # rows that need no workspace
_XT = {**_DT, torch.float8_e4m3fn: S6_E4M3}

_lib = None


def _load():
    global _lib
    if _lib is None:
        lib = s6.load_library()
        i64, vp, i32, f32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        for name, args in {
            "s6_q4_pack": [i64, i64, i64, i32, vp, i64, vp, vp, vp],
            "s6_q4_linear": [i64, i64, i64, i64, i32, i32, vp, i64, vp, vp, vp, vp, vp, sz, vp],
            "s6_q4_linear_workspace_size": [i64, i64, i64, i64, i32, ctypes.POINTER(sz)],
            "s6_add_norm_q8_fwd": [i64, i64, i32, i32, vp, i64, vp, vp, vp, f32, f32, vp, vp, vp, vp],
        }.items():
            fn = getattr(lib, name)
            fn.restype = i32
            fn.argtypes = args
        _lib = lib
    return _lib


def _no_gradient(name, *tensors):
    """Refuses inputs whose gradient would be lost."""
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} has no gradient and an input requires one: detach it, or call under "
                             "torch.no_grad()")


def q4_pack(w, group=128):
    """4-bit codes and group scales of w (outer, inner) in float32 or bfloat16
    (rows may be slices of wider ones): (weight, scales), uint8 (outer, inner /
    2) and bfloat16 (outer, inner / group).  group: 32, 64 or 128, a divisor of
    inner."""
    dt = _dtype(w, "w")
    if w.dim() != 2:
        raise ValueError("w is (outer, inner)")
    outer, inner = w.shape
    if group not in GROUPS or inner % group or inner == 0:
        raise ValueError(f"groups of {group} columns: expected 32, 64 or 128, a divisor of {inner}")
    stride = _flat(w, "w", w.shape, dt)
    weight = torch.empty((outer, inner // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((outer, inner // group), dtype=torch.bfloat16, device=w.device)
    _launch(_load().s6_q4_pack, w, outer, inner, group, _DT[dt], _at(w), stride, _at(weight), _at(scales))
    return weight, scales


def q4_linear(x, weight, scales, x_scale=None, out_dtype=None, y=None):
    """x W^T for 4-bit weights as q4_pack leaves them.  x: (..., inner) in
    float32, bfloat16, or float8_e4m3fn with one fp32 factor per row in
    x_scale (...), as add_norm_q8_fwd leaves them; x may be a slice of wider
    rows.  Returns (..., outer) in out_dtype, float32 or bfloat16 (unless
    given: x's, bfloat16 for 8-bit rows)."""
    _no_gradient("q4_linear", x, scales, x_scale)
    dt = x.dtype
    if dt not in _XT:
        raise ValueError(f"unsupported x dtype {dt}")
    yt = out_dtype or (torch.bfloat16 if dt == torch.float8_e4m3fn else dt)
    if yt not in _DT:
        raise ValueError(f"unsupported out_dtype {yt}")
    if weight.dim() != 2 or scales.dim() != 2 or x.dim() < 1:
        raise ValueError("x is (..., inner), weight (outer, inner / 2), scales (outer, inner / group)")
    inner, outer, ngroups = x.shape[-1], weight.shape[0], scales.shape[1]
    if ngroups == 0 or inner % ngroups or inner // ngroups not in GROUPS:
        raise ValueError(f"{ngroups} scales for {inner} columns: groups have 32, 64 or 128")
    lead = x.shape[:-1]
    index = x.get_device()
    stride = inner if index >= 0 and x.is_contiguous() else _flat(x, "x", x.shape, dt)
    if not (_plain(weight, (outer, inner // 2), torch.uint8, index) and
            _plain(scales, (outer, ngroups), torch.bfloat16, index)):
        _whole(weight, "weight", (outer, inner // 2), torch.uint8)
        _whole(scales, "scales", (outer, ngroups), torch.bfloat16)
        _same_device(x, weight, scales)
    if x_scale is not None:
        if dt != torch.float8_e4m3fn:
            raise ValueError("x_scale goes with 8-bit rows")
        if not _plain(x_scale, lead, torch.float32, index):
            _whole(x_scale, "x_scale", lead)
            _same_device(x, x_scale)
    if y is not None:
        _whole(y, "y", (*lead, outer), yt)
        _same_device(x, y)
        _written(y)
    else:
        y = x.new_empty((*lead, outer), dtype=yt)
    lib = _load()
    rows = math.prod(lead)
    group = inner // ngroups
    keep = wsp = None
    wsn = 0
    if rows > FEW[dt]:
        keep, wsp, wsn = _workspace(lib.s6_q4_linear_workspace_size, x, rows, inner, outer, group, _XT[dt])
    _launch(lib.s6_q4_linear, x, rows, inner, outer, group, _XT[dt], _DT[yt], x.data_ptr(), stride, _at(x_scale),
            weight.data_ptr(), scales.data_ptr(), y.data_ptr(), wsp, wsn)
    del keep
    return y


def add_norm_q8_fwd(x, weight, residual=None, gamma=None, scale=1.0, eps=1e-5, residual_dtype=None, out=None,
                    out_scale=None, residual_out=None):
    """block.add_norm_fwd with its output in 8 bits: per row of the last
    dimension, r' = residual + scale * gamma * x, o = r' / sqrt(mean(r'^2) +
    eps) * weight, out_scale = max|o| / 448, out = o / out_scale.  Returns
    (out in float8_e4m3fn, out_scale (...) fp32, r' in the residual's dtype);
    residual_out may be the residual itself."""
    _no_gradient("add_norm_q8_fwd", x, weight, residual, gamma)
    dt = _dtype(x)
    stride = x.shape[-1] if x.is_contiguous() and x.is_cuda else _flat(x, "x", x.shape, dt)
    rt = residual.dtype if residual is not None else residual_dtype or torch.float32
    if rt not in (torch.float32, dt):
        raise ValueError(f"residual dtype {rt}: expected float32 or {dt}")
    dim, lead = x.shape[-1], x.shape[:-1]
    index = x.get_device()
    if residual is not None and not _plain(residual, x.shape, rt, index):
        _whole(residual, "residual", x.shape, rt)
        _same_device(x, residual)
    if weight is None or not _plain(weight, (dim,), torch.float32, index):
        _weight(weight, dim)
        _same_device(x, weight)
    if gamma is not None and not _plain(gamma, (dim,), torch.float32, index):
        _whole(gamma, "gamma", (dim,))
        _same_device(x, gamma)
    if out is not None or out_scale is not None or residual_out is not None:
        _whole(out, "out", x.shape, torch.float8_e4m3fn)
        _whole(out_scale, "out_scale", lead)
        _whole(residual_out, "residual_out", x.shape, rt)
        _same_device(x, out, out_scale, residual_out)
        _written(out, out_scale, residual_out)
    if out is None:
        out = x.new_empty(x.shape, dtype=torch.float8_e4m3fn)
    if out_scale is None:
        out_scale = x.new_empty(lead, dtype=torch.float32)
    if residual_out is None:
        residual_out = x.new_empty(x.shape, dtype=rt)
    _launch(_load().s6_add_norm_q8_fwd, x, math.prod(lead), dim, _DT[dt], _DT[rt], x.data_ptr(), stride, _at(residual),
            weight.data_ptr(), _at(gamma), scale, eps, out.data_ptr(), out_scale.data_ptr(), residual_out.data_ptr())
    return out, out_scale, residual_out
