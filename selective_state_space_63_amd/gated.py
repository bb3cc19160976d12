"""Python binding of the gated recurrence of libs6 (include/s6_gated.h): whole
sequences, gradients and the single-token step.

As in ``block``: argument marshalling only, torch device tensors in and out,
work enqueued on the current stream of the tensors' device.  ``GatedScan`` is
the recurrence for torch autograd (once differentiable).
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.function import once_differentiable

from . import s6
from .block import _at, _dtype, _launch, _need, _plain, _rows, _same_device, _unasked, _whole, _written
from .s6 import _DT, _check

S6_UNIT_INPUT = 4
TOKENS = 128  # tokens from one stored state to the next (S6_GATED_TOKENS)


class GatedDims(ctypes.Structure):
    """s6_gated_dims of include/s6_gated.h."""

    _fields_ = [(n, ctypes.c_int64) for n in
                ("batch", "seqlen", "dim", "x_batch", "x_token", "a_batch", "a_token", "g_batch", "g_token")]


@functools.lru_cache(maxsize=256)
def _struct(*sizes):
    """(the dims of these sizes and strides, a reference to them)."""
    d = GatedDims(*sizes)
    return d, ctypes.byref(d)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(index, batch, seqlen, dim, back, has_states):
    """Bytes of workspace for these sizes on device `index`."""
    d, ref = _struct(batch, seqlen, dim, 0, 0, 0, 0, 0, 0)
    out = ctypes.c_size_t(0)
    lib = _load()
    with torch.cuda.device(index):
        if back:
            _check(lib.s6_gated_scan_bwd_workspace_size(ref, has_states, ctypes.byref(out)))
        else:
            _check(lib.s6_gated_scan_fwd_workspace_size(ref, ctypes.byref(out)))
    return out.value


def _workspace(x, dims, back=False, has_states=False):
    """(tensor, pointer, bytes) of a fresh workspace on the current stream."""
    n = _workspace_bytes(x.get_device(), dims.batch, dims.seqlen, dims.dim, back, has_states)
    if n == 0:
        return None, None, 0
    t = x.new_empty(n, dtype=torch.uint8)
    return t, t.data_ptr(), n


_lib = None


def _load():
    global _lib
    if _lib is None:
        lib = s6.load_library()
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        dims, szp = ctypes.POINTER(GatedDims), ctypes.POINTER(ctypes.c_size_t)
        for name, args in {
            "s6_gated_scan_fwd": [dims, i32, i32] + [vp] * 12 + [sz, vp],
            "s6_gated_scan_fwd_workspace_size": [dims, szp],
            "s6_gated_scan_bwd": [dims, i32, i32] + [vp] * 19 + [sz, vp],
            "s6_gated_scan_bwd_workspace_size": [dims, i32, szp],
            "s6_gated_state_update": [dims, i32, i32] + [vp] * 9,
        }.items():
            fn = getattr(lib, name)
            fn.restype = i32
            fn.argtypes = args
        _lib = lib
    return _lib


def _gated_dims(x, gate_a, gate_x, A, bias_a, bias_x, unit_input, tokens):
    dt = _dtype(x)
    if x.dim() != (3 if tokens else 2):
        raise ValueError("x and the gates are (batch, seqlen, dim); (batch, dim) for a single token")
    shape, index = x.shape, x.get_device()
    xs = _strides(x, "x", shape, dt, index)
    gs = _strides(gate_a, "gate_a", shape, dt, index)
    if gate_x is None:
        if bias_x is not None:
            raise ValueError("bias_x needs a gate_x")
        ys = (0,) * len(xs)
    else:
        ys = _strides(gate_x, "gate_x", shape, dt, index)
    channels = shape[-1:]
    if A is None:
        raise ValueError("A is required")
    for t, name in ((A, "A"), (bias_a, "bias_a"), (bias_x, "bias_x")):
        if t is not None and not _plain(t, channels, torch.float32, index):
            _whole(t, name, channels)
            _same_device(x, t)
    if tokens:
        dims, ref = _struct(*shape, *xs, *gs, *ys)
    else:
        dims, ref = _struct(shape[0], 1, shape[1], xs[0], 0, gs[0], 0, ys[0], 0)
    return dims, ref, _DT[dt], S6_UNIT_INPUT if unit_input else 0


def _strides(t, name, shape, dt, index):
    """Strides of the leading dimensions."""
    if t is not None and index >= 0 and t.shape == shape and t.dtype is dt and t.get_device() == index:
        st = t.stride()
        if st[-1] == 1 and 1 not in shape:
            return st[:-1]
    st = _rows(t, name, shape, dt, 1)
    if t.get_device() != index:
        raise ValueError(f"tensors on cuda:{index} and {t.device}")
    return st


def _starts(starts, x):
    """starts as bytes."""
    if starts is None:
        return None
    if starts.dtype not in (torch.bool, torch.uint8):
        raise ValueError(f"starts has dtype {starts.dtype}, expected bool or uint8")
    _whole(starts, "starts", x.shape[:2], starts.dtype)
    _same_device(x, starts)
    return starts


def _states_shape(x):
    return (x.shape[0], -(-x.shape[1] // TOKENS), x.shape[2])


def gated_scan_fwd(x, gate_a, gate_x, A, bias_a=None, bias_x=None, h0=None, starts=None, unit_input=False,
                   return_last_state=False, return_states=False, y=None, h_last=None, states=None):
    """Gated linear recurrence: with r = sigmoid(gate_a + bias_a), i =
    sigmoid(gate_x + bias_x) and a = exp(A r), the state of a channel goes to
    a h + sqrt(1 - a^2) i x (a h + i x with unit_input), and y is the state.
    x, gate_a and gate_x (None: i = 1): (batch, L, dim), one dtype (float32 or
    bfloat16), slices of wider rows allowed; A (at most 0), bias_a, bias_x:
    (dim,) fp32; h0: (batch, dim) fp32; starts: (batch, L) bool or uint8,
    tokens that begin a sequence of their own.  Returns y like x (contiguous);
    h_last (batch, dim) fp32 if requested; with return_states the state
    entering every 128 tokens, for gated_scan_bwd."""
    dims, ref, dt, flags = _gated_dims(x, gate_a, gate_x, A, bias_a, bias_x, unit_input, True)
    sshape = (dims.batch, dims.dim)
    starts = _starts(starts, x)
    if h0 is not None:
        _whole(h0, "h0", sshape)
        _same_device(x, h0)
    if y is not None or h_last is not None or states is not None:
        _whole(y, "y", x.shape, x.dtype)
        _whole(h_last, "h_last", sshape)
        _whole(states, "states", _states_shape(x))
        _same_device(x, y, h_last, states)
        _written(y, h_last, states)
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    if return_last_state and h_last is None:
        h_last = x.new_empty(sshape, dtype=torch.float32)
    if return_states and states is None:
        states = x.new_empty(_states_shape(x), dtype=torch.float32)
    lib = _load()
    keep, wsp, wsn = _workspace(x, dims)
    _launch(lib.s6_gated_scan_fwd, x, ref, dt, flags, _at(x), _at(gate_a), _at(bias_a), _at(gate_x), _at(bias_x), _at(A),
            _at(starts), _at(h0), _at(y), _at(h_last), _at(states), wsp, wsn)
    del keep
    out = (y,) + ((h_last,) if return_last_state else ()) + ((states,) if return_states else ())
    return out if len(out) > 1 else y


def gated_scan_bwd(x, gate_a, gate_x, A, dy, bias_a=None, bias_x=None, h0=None, starts=None, unit_input=False,
                   dh_last=None, states=None, skip=()):
    """Gradients of <dy, y> + <dh_last, h_last> for gated_scan_fwd with the
    same inputs.  dy: like y, contiguous; dh_last: like h_last or None; states:
    those that the forward returned (None: formed again).  Returns a dict: dx,
    dgate_a, and where gate_x is given dgate_x, in the input dtype; dA, and
    where their input is given dbias_a, dbias_x, dh0 in fp32.  skip: names
    among the last four to leave out."""
    dims, ref, dt, flags = _gated_dims(x, gate_a, gate_x, A, bias_a, bias_x, unit_input, True)
    sshape = (dims.batch, dims.dim)
    starts = _starts(starts, x)
    _whole(h0, "h0", sshape)
    _whole(dh_last, "dh_last", sshape)
    _whole(states, "states", _states_shape(x))
    _whole(_need(dy, "dy", x.shape, x.dtype), "dy", x.shape, x.dtype)
    _same_device(x, h0, dh_last, states, dy)
    g = {"dx": torch.empty_like(dy), "dgate_a": torch.empty_like(dy)}
    if gate_x is not None:
        g["dgate_x"] = torch.empty_like(dy)
    for name, t in (("dA", A), ("dbias_a", bias_a), ("dbias_x", bias_x), ("dh0", h0)):
        if t is not None and name not in skip:
            g[name] = torch.empty_like(t)
    lib = _load()
    keep, wsp, wsn = _workspace(x, dims, True, states is not None)
    _launch(lib.s6_gated_scan_bwd, x, ref, dt, flags, _at(x), _at(gate_a), _at(bias_a), _at(gate_x), _at(bias_x), _at(A),
            _at(starts), _at(h0), _at(states), _at(dy), _at(dh_last), _at(g["dx"]), _at(g["dgate_a"]),
            _at(g.get("dgate_x")), _at(g.get("dA")), _at(g.get("dbias_a")), _at(g.get("dbias_x")), _at(g.get("dh0")), wsp,
            wsn)
    del keep
    return g


def gated_state_update(h, x, gate_a, gate_x, A, bias_a=None, bias_x=None, unit_input=False, y=None):
    """One token of every sequence: h (batch, dim) fp32 is advanced in place;
    x, gate_a, gate_x: (batch, dim).  Returns y (batch, dim) in x's dtype."""
    dims, ref, dt, flags = _gated_dims(x, gate_a, gate_x, A, bias_a, bias_x, unit_input, False)
    if h is None or not _plain(h, x.shape, torch.float32, x.get_device()):
        _whole(_need(h, "h", x.shape, torch.float32), "h", x.shape)
        _same_device(x, h)
    if y is not None:
        _whole(y, "y", x.shape, x.dtype)
        _same_device(x, y)
    _written(h, y)
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    _launch(_load().s6_gated_state_update, x, ref, dt, flags, h.data_ptr(), x.data_ptr(), gate_a.data_ptr(), _at(bias_a),
            _at(gate_x), _at(bias_x), A.data_ptr(), y.data_ptr())
    return y


class GatedScan(torch.autograd.Function):
    """gated_scan_fwd with its gradients: y, h_last = GatedScan.apply(x,
    gate_a, gate_x, A, bias_a, bias_x, h0, starts, unit_input).  gate_x,
    bias_a, bias_x, h0 and starts may be None.  The forward keeps the state
    entering every 128 tokens."""

    @staticmethod
    def forward(ctx, x, gate_a, gate_x, A, bias_a=None, bias_x=None, h0=None, starts=None, unit_input=False):
        y, h_last, states = gated_scan_fwd(x, gate_a, gate_x, A, bias_a=bias_a, bias_x=bias_x, h0=h0, starts=starts,
                                           unit_input=unit_input, return_last_state=True, return_states=True)
        ctx.save_for_backward(x, gate_a, gate_x, A, bias_a, bias_x, h0, starts, states)
        ctx.unit_input = unit_input
        ctx.set_materialize_grads(False)
        return y, h_last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh_last):
        x, gate_a, gate_x, A, bias_a, bias_x, h0, starts, states = ctx.saved_tensors
        dy = torch.zeros_like(x, memory_format=torch.contiguous_format) if dy is None else dy.contiguous()
        names = ("dx", "dgate_a", "dgate_x", "dA", "dbias_a", "dbias_x", "dh0")
        g = gated_scan_bwd(x, gate_a, gate_x, A, dy, bias_a=bias_a, bias_x=bias_x, h0=h0, starts=starts,
                           unit_input=ctx.unit_input, dh_last=None if dh_last is None else dh_last.contiguous(),
                           states=states, skip=_unasked(ctx, names))
        return (*(g.get(name) for name in names), None, None)
