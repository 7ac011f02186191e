"""Thin Python binding of the gated recurrent layer's operators (include/prism_gated.h).

Argument checks and marshalling only, as in ``linattn``: the work runs in libprism.so's kernels,
and a missing library raises.  Token inputs (x, the gates and the gradients that come in) are
[B,T,D] tensors whose channels are contiguous; sequences and tokens may be strided, so slices
of one fused projection serve as they are; tensors expanded over tokens or sequences are refused.
Everything else is contiguous.  All tensors of a call lie on x's device, which need not be the
current one.

Streams are handled as in ``linattn``: a call runs on ``stream`` (default: the current one), what it
allocates there comes from that stream's memory, and its tensors are recorded on the streams that
use them.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import prism as _prism
from .linattn import (_call, _check, _dtype_code, _like, _new, _room, _scratch, _stream, _stride, _strided, _used,
                      _whole)
from .prism import PrismError

PRISM_GATED_CHUNK = 64
EXPORTS = ("prism_layer_norm", "prism_layer_norm_workspace_bytes", "prism_layer_norm_backward",
           "prism_gated_scan_workspace_bytes", "prism_gated_scan_forward", "prism_gated_scan_backward_workspace_bytes",
           "prism_gated_scan_backward", "prism_gated_scan_decode_step", "prism_gated_status")

_vp, _int, _size = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t


class LayerNormDims(ctypes.Structure):
    _fields_ = [("B", _int), ("T", _int), ("D", _int), ("dtype", _int), ("flags", ctypes.c_uint),
                ("eps", ctypes.c_float), ("x_stride", _stride), ("do_stride", _stride)]


class GatedDims(ctypes.Structure):
    _fields_ = [("B", _int), ("T", _int), ("D", _int), ("dtype", _int), ("flags", ctypes.c_uint),
                ("x_stride", _stride), ("f_stride", _stride), ("i_stride", _stride), ("do_stride", _stride)]


@functools.cache
def load():
    """libprism.so with this module's entry points declared (raises if it is missing)."""
    lib = _prism.load()
    for name, args, res in (
            ("prism_layer_norm", [_vp] * 7, _int),
            ("prism_layer_norm_workspace_bytes", [_vp], _size),
            ("prism_layer_norm_backward", [_vp] * 9 + [_size, _vp], _int),
            ("prism_gated_scan_workspace_bytes", [_vp], _size),
            ("prism_gated_scan_forward", [_vp] * 10 + [_size, _vp], _int),
            ("prism_gated_scan_backward_workspace_bytes", [_vp], _size),
            ("prism_gated_scan_backward", [_vp] * 13 + [_size, _vp], _int),
            ("prism_gated_scan_decode_step", [_vp] * 5 + [_int, _vp, _vp, _vp], _int),
            ("prism_gated_status", [ctypes.POINTER(_int), _int], _int)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res
    return lib


def _steps(name, shape, stride):
    """Sequence and token strides of a [B,T,D] tensor."""
    B, T, D = shape
    if 0 in shape:
        raise PrismError(1, f"{name} is empty")
    if stride[2] != 1 and D > 1:
        raise PrismError(1, f"{name}: the channels of a token must be contiguous")
    if (T > 1 and stride[1] < D) or (B > 1 and stride[0] <= 0):     # a step of 0 would be taken for "contiguous"
        raise PrismError(1, f"{name}: every token must have memory of its own; an expanded tensor is not read as it lies "
                            "(call contiguous() on it)")
    return _stride(stride[0] if B > 1 else T * max(stride[1], D), stride[1] if T > 1 else D)


def _width(D, most=None):
    if D % 8 or (most and D > most):
        raise PrismError(2, f"the channels of a token must be a multiple of 8{f' up to {most}' if most else ''}, got {D}")


def _out(t, side):
    """A contiguous tensor of t's shape and type."""
    if side is None and t.is_contiguous():
        return torch.empty_like(t)
    return _new(t.shape, t.dtype, t.device, side)


# Outputs and workspaces that are passed in are checked; what the call makes itself is as it has to be.

def _result(name, t, like, dev, side):
    """A contiguous output of ``like``'s shape and type, and its address."""
    if t is not None:
        return t, _whole(name, t, like.shape, like.dtype, dev)
    t = _out(like, side)
    return t, t.data_ptr()


def _workspace(t, nbytes, device, dev, side):
    """A workspace, its address and its bytes."""
    if t is not None:
        return (t, *_room(t, dev))
    if not nbytes:
        return None, None, 0
    t = _scratch(nbytes, device, side)
    return t, t.data_ptr(), nbytes


# The checked dims of a call by shapes, strides and settings, as in ``linattn``, with their workspace and the shapes of what
# goes with them.

@functools.lru_cache(maxsize=256)
def _norm_dims(xs, xst, dtype, eps, dost):
    if len(xs) != 3:
        raise PrismError(1, f"x must be [B,T,D], got {tuple(xs)}")
    _width(xs[2], 16384)
    d = LayerNormDims(B=xs[0], T=xs[1], D=xs[2], dtype=_dtype_code(dtype), flags=0, eps=eps,
                      x_stride=_steps("x", xs, xst))
    if dost is not None:
        d.do_stride = _steps("d_out", xs, dost)
    return d, ctypes.addressof(d), int(load().prism_layer_norm_workspace_bytes(ctypes.addressof(d))), xs[2:], xs[:1]


@functools.lru_cache(maxsize=256)
def _gated_dims(xs, dtype, xst, fst, ist, dost, flags):
    if len(xs) != 3:
        raise PrismError(1, f"x and the gates must be [B,T,D], got {tuple(xs)}")
    _width(xs[2])
    d = GatedDims(B=xs[0], T=xs[1], D=xs[2], dtype=_dtype_code(dtype), flags=flags, x_stride=_steps("x", xs, xst),
                  f_stride=_steps("forget", xs, fst))
    if ist is not None:
        d.i_stride = _steps("input_gate", xs, ist)
    if dost is not None:
        d.do_stride = _steps("d_out", xs, dost)
    rows = torch.Size((xs[0], -(-xs[1] // PRISM_GATED_CHUNK), xs[2]))
    size = load().prism_gated_scan_workspace_bytes if dost is None else load().prism_gated_scan_backward_workspace_bytes
    return d, ctypes.addressof(d), int(size(ctypes.addressof(d))), rows, rows[::2], xs[:1]


@functools.lru_cache(maxsize=256)
def _decode_dims(xs, dtype, xst, fst, ist):
    if len(xs) != 2:
        raise PrismError(1, f"x and the gates must be [B,D], got {tuple(xs)}")
    B, D = xs
    _width(D)

    def steps(name, st):
        return _steps(name, (B, 1, D), (st[0], D, st[1]))

    d = GatedDims(B=B, T=1, D=D, dtype=_dtype_code(dtype), flags=0, x_stride=steps("x", xst),
                  f_stride=steps("forget", fst))
    if ist is not None:
        d.i_stride = steps("input_gate", ist)
    return d, ctypes.addressof(d), xs[:1]


def prism_layer_norm(x, *, weight=None, bias=None, eps=1e-5, seq_lens=None, out=None, stream=None):
    """Layer norm of every token of x [B,T,D]: (x - mean) / sqrt(var + eps) * weight + bias, ``weight``
    and ``bias`` [D] fp32 (None: ones, zeros).  Returns out [B,T,D], contiguous, in x's type,
    0 at padding tokens."""
    keep, dims, _, D, B = _norm_dims(x.shape, x.stride(), x.dtype, float(eps), None)
    dev, raw, side = _stream(x, stream, "x")
    if side is not None:
        _used(side, x, weight, bias, seq_lens, out)
    w, b = _whole("weight", weight, D, torch.float32, dev), _whole("bias", bias, D, torch.float32, dev)
    lens = _whole("seq_lens", seq_lens, B, torch.int32, dev)
    out, to = _result("out", out, x, dev, side)
    _call(dev, load().prism_layer_norm, dims, x.data_ptr(), w, b, lens, to, raw)
    return out


def prism_layer_norm_backward(x, d_out, *, weight=None, bias=None, eps=1e-5, seq_lens=None, grads=None,
                              workspace=None, stream=None):
    """Gradients through prism_layer_norm given ``d_out`` [B,T,D] in x's type.  Returns a dict: x in its
    type, weight and bias fp32 (None where the norm had none).  ``grads`` may pass preallocated
    outputs with the same keys."""
    xs = x.shape
    _like("d_out", d_out, xs, x.dtype)
    keep, dims, nbytes, D, B = _norm_dims(xs, x.stride(), x.dtype, float(eps), d_out.stride())
    dev, raw, side = _stream(x, stream, "x")
    g = dict(grads) if grads else {}
    if side is not None:
        _used(side, x, d_out, weight, bias, seq_lens, workspace, *g.values())
    w = _whole("weight", weight, D, torch.float32, dev)
    _whole("bias", bias, D, torch.float32, dev)
    lens, dy = _whole("seq_lens", seq_lens, B, torch.int32, dev), _strided("d_out", d_out, dev)
    g["x"], dx = _result("grads['x']", g.get("x"), x, dev, side)
    to = {}
    for n, t in (("weight", weight), ("bias", bias)):
        mine = g.get(n)
        if mine is None and t is not None:
            g[n], to[n] = _result(n, None, t, dev, side)
        else:
            g[n], to[n] = mine, _whole(f"grads['{n}']", mine, D, torch.float32, dev)
    wanted = to["weight"] is not None or to["bias"] is not None
    keep2, room, size = _workspace(workspace, nbytes if wanted else 0, x.device, dev, side)
    _call(dev, load().prism_layer_norm_backward, dims, x.data_ptr(), w, lens, dy, dx, to["weight"], to["bias"], room, size, raw)
    return g


def _gates(x, forget, input_gate):
    xs, dt = x.shape, x.dtype
    _like("forget", forget, xs, dt)
    if input_gate is None:
        return xs, dt, None
    _like("input_gate", input_gate, xs, dt)
    return xs, dt, input_gate.stride()


def gated_scan_states(x):
    """Room for the states that prism_gated_scan_forward leaves to the backward pass of x [B,T,D]."""
    B, T, D = x.shape
    return torch.empty((B, -(-T // PRISM_GATED_CHUNK), D), dtype=torch.float32, device=x.device)


def prism_gated_scan_forward(x, forget, *, input_gate=None, initial_state=None, out=None, final_state=None,
                             states=None, seq_lens=None, workspace=None, stream=None, want_state=True, flags=0):
    """The gated linear recurrence over x [B,T,D]: h_t = a_t h_(t-1) + w_t x_t with a = sigmoid(``forget``) and
    w = sigmoid(``input_gate``), or 1 - a without one; h before the first token is
    ``initial_state`` [B,D] fp32 (None: zero).  Returns ``(out, final_state)``: h of every token
    [B,T,D] in x's type, and the last one in fp32 (None when ``want_state`` is False and none was passed;
    it may be initial_state itself).  ``states`` (see gated_scan_states) is filled for the backward pass."""
    xs, dt, ist = _gates(x, forget, input_gate)
    keep, dims, nbytes, rows, ss, B = _gated_dims(xs, dt, x.stride(), forget.stride(), ist, None, int(flags))
    dev, raw, side = _stream(x, stream, "x")
    if side is not None:
        _used(side, x, forget, input_gate, initial_state, out, final_state, states, seq_lens, workspace)
    f, i = _strided("forget", forget, dev), None if input_gate is None else _strided("input_gate", input_gate, dev)
    s0, st = _whole("initial_state", initial_state, ss, torch.float32, dev), _whole("states", states, rows, torch.float32, dev)
    lens = _whole("seq_lens", seq_lens, B, torch.int32, dev)
    out, to = _result("out", out, x, dev, side)
    if final_state is None and want_state:
        final_state = _new(ss, torch.float32, x.device, side)
        s1 = final_state.data_ptr()
    else:
        s1 = _whole("final_state", final_state, ss, torch.float32, dev)
    keep2, room, size = _workspace(workspace, nbytes, x.device, dev, side)
    _call(dev, load().prism_gated_scan_forward, dims, x.data_ptr(), f, i, s0, to, s1, st, lens, room, size, raw)
    return out, final_state


def prism_gated_scan_backward(x, forget, states, d_out, *, input_gate=None, d_final_state=None, seq_lens=None,
                              grads=None, workspace=None, stream=None, want_initial_state=False, flags=0):
    """Gradients through prism_gated_scan_forward given ``d_out`` [B,T,D] in x's type (and
    ``d_final_state`` [B,D] fp32), with the ``states`` that it filled for the same inputs.  Returns a dict: x,
    forget and input_gate in their type (None without an input gate), initial_state fp32 (None unless
    ``want_initial_state``).  ``grads`` may pass preallocated outputs with the same keys."""
    xs, dt, ist = _gates(x, forget, input_gate)
    _like("d_out", d_out, xs, dt)
    keep, dims, nbytes, rows, ss, B = _gated_dims(xs, dt, x.stride(), forget.stride(), ist, d_out.stride(), int(flags))
    dev, raw, side = _stream(x, stream, "x")
    g = dict(grads) if grads else {}
    if side is not None:
        _used(side, x, forget, input_gate, states, d_out, d_final_state, seq_lens, workspace, *g.values())
    f, i = _strided("forget", forget, dev), None if input_gate is None else _strided("input_gate", input_gate, dev)
    st, dy = _whole("states", states, rows, torch.float32, dev), _strided("d_out", d_out, dev)
    s1, lens = _whole("d_final_state", d_final_state, ss, torch.float32, dev), _whole("seq_lens", seq_lens, B, torch.int32, dev)
    g["x"], dx = _result("grads['x']", g.get("x"), x, dev, side)
    g["forget"], df = _result("grads['forget']", g.get("forget"), forget, dev, side)
    if input_gate is not None:
        g["input_gate"], di = _result("grads['input_gate']", g.get("input_gate"), input_gate, dev, side)
    else:
        di = _whole("grads['input_gate']", g.setdefault("input_gate", None), xs, dt, dev)
    if g.get("initial_state") is None and want_initial_state:
        g["initial_state"] = _new(ss, torch.float32, x.device, side)
        d0 = g["initial_state"].data_ptr()
    else:
        d0 = _whole("grads['initial_state']", g.setdefault("initial_state", None), ss, torch.float32, dev)
    keep2, room, size = _workspace(workspace, nbytes, x.device, dev, side)
    _call(dev, load().prism_gated_scan_backward, dims, x.data_ptr(), f, i, st, dy, s1, dx, df, di, d0, lens, room, size, raw)
    return g


def prism_gated_scan_decode_step(x, forget, state, *, input_gate=None, slots=None, out=None, stream=None):
    """One token of every sequence: x and the gates [B,D]; ``state`` [N,D] fp32 is updated in place.
    ``slots`` [B] int32 says which state each sequence has (None: its own index; outside 0..N-1: the
    sequence is not there, its output is 0).  Returns out [B,D] in x's type."""
    xs, dt, ist = _gates(x, forget, input_gate)
    keep, dims, B = _decode_dims(xs, dt, x.stride(), forget.stride(), ist)
    dev, raw, side = _stream(x, stream, "x")
    N = state.shape[0]
    if side is not None:
        _used(side, x, forget, input_gate, state, slots, out)
    f, i = _strided("forget", forget, dev), None if input_gate is None else _strided("input_gate", input_gate, dev)
    st, at = _whole("state", state, (N, xs[1]), torch.float32, dev), _whole("slots", slots, B, torch.int32, dev)
    out, to = _result("out", out, x, dev, side)
    _call(dev, load().prism_gated_scan_decode_step, dims, x.data_ptr(), f, i, st, N, at, to, raw)
    return out


def gated_status(clear: bool = True) -> int:
    """The word of bounded waits that gave up on the current device (0: none; synchronises)."""
    word = _int(-1)
    _check(load().prism_gated_status(ctypes.byref(word), 1 if clear else 0))
    return word.value
