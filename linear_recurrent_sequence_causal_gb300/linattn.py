"""Thin Python binding of the linear attention layer's operators (include/prism_linattn.h).

Argument checks and marshalling only, as in ``prism``: the work runs in libprism.so's
kernels, and a missing library raises.  Token inputs (q, k, v and the gradients that come in)
are [B,T,H,D] tensors whose heads are contiguous; sequences and tokens may be strided, so
slices of one fused projection serve as they are; tensors expanded over tokens or sequences are
refused.  Everything else is contiguous.  All tensors of a call lie on q's device, which need not be
the current one.

A call runs on ``stream`` (default: the current one), ordered after what is there already.  Where
that is not the current stream, what the call allocates comes from that stream's memory, and
the tensors of the call are recorded on the streams that use them, so that none is handed out
again before its kernels are done.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import prism as _prism
from .prism import PRISM_BF16, PRISM_F32, PrismError

PRISM_ROPE_INTERLEAVED = 1
EXPORTS = ("prism_qk_norm_rope", "prism_qk_norm_rope_workspace_bytes", "prism_qk_norm_rope_backward",
           "prism_linattn_workspace_bytes", "prism_linattn_forward", "prism_linattn_backward_workspace_bytes",
           "prism_linattn_backward", "prism_linattn_decode_step", "prism_linattn_status")

_vp, _int, _size = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_stride = ctypes.c_longlong * 2


class RopeDims(ctypes.Structure):
    _fields_ = [("B", _int), ("T", _int), ("Hq", _int), ("Hk", _int), ("d", _int), ("rotary_dim", _int),
                ("table_rows", _int), ("dtype", _int), ("flags", ctypes.c_uint), ("eps", ctypes.c_float),
                ("q_scale", ctypes.c_float), ("k_scale", ctypes.c_float), ("q_stride", _stride),
                ("k_stride", _stride), ("dq_stride", _stride), ("dk_stride", _stride)]


class LinattnDims(ctypes.Structure):
    _fields_ = [("B", _int), ("T", _int), ("H", _int), ("d", _int), ("dtype", _int), ("flags", ctypes.c_uint),
                ("scale", ctypes.c_float), ("q_stride", _stride), ("k_stride", _stride), ("v_stride", _stride),
                ("do_stride", _stride)]


@functools.cache
def load():
    """libprism.so with this module's entry points declared (raises if it is missing)."""
    lib = _prism.load()
    for name, args, res in (
            ("prism_qk_norm_rope", [_vp] * 11, _int),
            ("prism_qk_norm_rope_workspace_bytes", [_vp], _size),
            ("prism_qk_norm_rope_backward", [_vp] * 15 + [_size, _vp], _int),
            ("prism_linattn_workspace_bytes", [_vp], _size),
            ("prism_linattn_forward", [_vp] * 10 + [_size, _vp], _int),
            ("prism_linattn_backward_workspace_bytes", [_vp], _size),
            ("prism_linattn_backward", [_vp] * 14 + [_size, _vp], _int),
            ("prism_linattn_decode_step", [_vp] * 6 + [_int, _vp, _vp, _vp], _int),
            ("prism_linattn_status", [ctypes.POINTER(_int), _int], _int)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res
    return lib


def _check(code: int):
    if code != 0:
        raise PrismError(code, _prism.strerror(code))


def _dtype_code(t) -> int:
    if t == torch.bfloat16:
        return PRISM_BF16
    if t == torch.float32:
        return PRISM_F32
    raise PrismError(1, f"unsupported dtype {t}")


def _steps(name, shape, stride):
    """Sequence and token strides of a [B,T,H,D] tensor; (0, 0) stands for contiguous."""
    B, T, H, D = shape
    if 0 in shape:
        raise PrismError(1, f"{name} is empty")
    if stride[3] != 1 or (H > 1 and stride[2] != D):
        raise PrismError(1, f"{name}: the heads of a token must be contiguous")
    if (T > 1 and stride[1] < H * D) or (B > 1 and stride[0] <= 0):     # a step of 0 would be taken for "contiguous"
        raise PrismError(1, f"{name}: every token must have memory of its own; an expanded tensor is not read as it lies "
                            "(call contiguous() on it)")
    return _stride(stride[0] if B > 1 else T * max(stride[1], H * D), stride[1] if T > 1 else H * D)


def _like(name, t, shape, dtype):
    if t.dtype != dtype or t.shape != shape:
        raise PrismError(1, f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} of {tuple(t.shape)}")


def _whole(name, t, shape, dtype, dev):
    """The address of an optional contiguous tensor of this shape and type on device ``dev``."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape:
        raise PrismError(1, f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} of {tuple(t.shape)}")
    if t.get_device() != dev or not t.is_contiguous():
        raise PrismError(1, f"{name} must be a contiguous CUDA tensor on the call's device")
    return t.data_ptr()


def _strided(name, t, dev):
    if t.get_device() != dev:
        raise PrismError(1, f"{name} must be a CUDA tensor on the call's device")
    return t.data_ptr()


def _room(t, dev):
    """Address and bytes of an optional workspace."""
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise PrismError(1, "workspace must be a contiguous CUDA tensor on the call's device")
    return t.data_ptr(), t.numel() * t.element_size()


def _stream(t, stream, name="q"):
    """The call's device, the handle of its stream, and the stream itself where it is not the
    device's current one."""
    dev = t.get_device()
    if dev < 0:
        raise PrismError(1, f"{name} must be a CUDA tensor")
    here = torch._C._cuda_getCurrentRawStream(dev)
    if stream is None:
        return dev, here, None
    if stream.device.index != dev:
        raise PrismError(1, f"stream is on device {stream.device.index}, {name} on device {dev}")
    return dev, stream.cuda_stream, None if stream.cuda_stream == here else stream


def _call(dev, f, *args):
    """f on device ``dev``: the library launches on the current one."""
    if torch._C._cuda_getDevice() == dev:
        _check(f(*args))
    else:
        with torch.cuda.device(dev):
            _check(f(*args))


def _scratch(nbytes, device, side):
    """Memory for this call alone.  It goes back to the stream that it came from: the call's own."""
    if side is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(side):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _new(shape, dtype, device, side):
    """An output: written on the call's stream, read by the caller on the current one."""
    if side is None:
        return torch.empty(shape, dtype=dtype, device=device)
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(side):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(caller)
    return t


def _out(t, side):
    """A contiguous tensor of t's shape and type."""
    if side is None and t.is_contiguous():
        return torch.empty_like(t)
    return _new(t.shape, t.dtype, t.device, side)


def _used(side, *tensors):
    """The call's tensors, which may be dropped once it returns, are used on its stream."""
    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(side)


# The checked dims of a call by shapes, strides and settings: a layer calls with the same ones
# over and over.  The structures are only read afterwards.  Settings are plain numbers here (a
# tensor would be known by its identity, whatever value it holds later).

@functools.lru_cache(maxsize=256)
def _rope_dims(qs, qst, ks, kst, dtype, table_shape, interleaved, eps, q_scale, k_scale, dqst, dkst):
    if len(qs) != 4 or len(ks) != 4 or qs[:2] != ks[:2] or qs[3] != ks[3]:
        raise PrismError(1, f"q and k must be [B,T,heads,D] of the same B, T and D, got {tuple(qs)} and {tuple(ks)}")
    if table_shape is not None and len(table_shape) != 2:
        raise PrismError(1, "table must be [positions, rotary_dim]")
    rows, rot = table_shape if table_shape is not None else (0, 0)
    d = RopeDims(B=qs[0], T=qs[1], Hq=qs[2], Hk=ks[2], d=qs[3], rotary_dim=rot, table_rows=rows,
                 dtype=_dtype_code(dtype), flags=PRISM_ROPE_INTERLEAVED if interleaved else 0, eps=eps,
                 q_scale=q_scale, k_scale=k_scale, q_stride=_steps("q", qs, qst), k_stride=_steps("k", ks, kst))
    if dqst is not None:
        d.dq_stride, d.dk_stride = _steps("dq_out", qs, dqst), _steps("dk_out", ks, dkst)
    return d, ctypes.addressof(d), int(load().prism_qk_norm_rope_workspace_bytes(ctypes.addressof(d)))


@functools.lru_cache(maxsize=256)
def _linattn_dims(qs, dtype, scale, qst, kst, vst, dost, flags=0):
    if len(qs) != 4:
        raise PrismError(1, f"q, k and v must be [B,T,H,D], got {tuple(qs)}")
    d = LinattnDims(B=qs[0], T=qs[1], H=qs[2], d=qs[3], dtype=_dtype_code(dtype), flags=flags, scale=scale,
                    q_stride=_steps("q", qs, qst), k_stride=_steps("k", qs, kst), v_stride=_steps("v", qs, vst))
    if dost is not None:
        d.do_stride = _steps("d_out", qs, dost)
    size = load().prism_linattn_workspace_bytes if dost is None else load().prism_linattn_backward_workspace_bytes
    return d, ctypes.addressof(d), int(size(ctypes.addressof(d)))


@functools.lru_cache(maxsize=256)
def _decode_dims(qs, dtype, scale, qst, kst, vst):
    if len(qs) != 3:
        raise PrismError(1, f"q, k and v must be [B,H,D], got {tuple(qs)}")
    B, H, D = qs

    def steps(name, st):
        return _steps(name, (B, 1, H, D), (st[0], H * D, st[1], st[2]))

    d = LinattnDims(B=B, T=1, H=H, d=D, dtype=_dtype_code(dtype), flags=0, scale=scale, q_stride=steps("q", qst),
                    k_stride=steps("k", kst), v_stride=steps("v", vst))
    return d, ctypes.addressof(d)


def prism_qk_norm_rope(q, k, table, *, q_weight=None, k_weight=None, q_scale=1.0, k_scale=1.0, eps=1e-6,
                       positions=None, seq_lens=None, interleaved=False, q_out=None, k_out=None, stream=None):
    """Norm of every head of q [B,T,Hq,D] and k [B,T,Hk,D], weighted, scaled and turned by its
    token's angles.  ``table`` [P, r] fp32: the cosines, then the sines, of the r/2 pairs at
    each position (None: no rotation); ``positions`` [B,T] int32 (None: 0..T-1; outside
    0..P-1: padding).  The pairs are (i, i + r/2), or (2i, 2i+1) with ``interleaved``.
    Returns ``(q_out, k_out)``, contiguous, in q's type, 0 at padding tokens."""
    qs, ks, dt = q.shape, k.shape, q.dtype
    if k.dtype != dt:
        raise PrismError(1, f"q and k must have one type, got {dt} and {k.dtype}")
    keep, dims, _ = _rope_dims(qs, q.stride(), ks, k.stride(), dt, None if table is None else table.shape,
                               bool(interleaved), float(eps), float(q_scale), float(k_scale), None, None)
    dev, raw, side = _stream(q, stream)
    if side is not None:
        _used(side, q, k, table, q_weight, k_weight, positions, seq_lens, q_out, k_out)
    if q_out is None:
        q_out = _out(q, side)
    if k_out is None:
        k_out = _out(k, side)
    D = qs[3:]
    _call(
        dev, load().prism_qk_norm_rope, dims, _strided("q", q, dev), _strided("k", k, dev),
        _whole("q_weight", q_weight, D, torch.float32, dev), _whole("k_weight", k_weight, D, torch.float32, dev),
        None if table is None else _whole("table", table, table.shape, torch.float32, dev),
        _whole("positions", positions, qs[:2], torch.int32, dev), _whole("seq_lens", seq_lens, qs[:1], torch.int32, dev),
        _whole("q_out", q_out, qs, dt, dev), _whole("k_out", k_out, ks, dt, dev), raw)
    return q_out, k_out


def prism_qk_norm_rope_backward(q, k, table, dq_out, dk_out, *, q_weight=None, k_weight=None, q_scale=1.0,
                                k_scale=1.0, eps=1e-6, positions=None, seq_lens=None, interleaved=False, grads=None,
                                workspace=None, stream=None):
    """Gradients through prism_qk_norm_rope given those of its outputs.  Returns a dict: q, k in
    their type, q_weight, k_weight fp32 (None where there is no weight).  ``grads`` may
    pass preallocated outputs with the same keys."""
    qs, ks, dt = q.shape, k.shape, q.dtype
    if k.dtype != dt:
        raise PrismError(1, f"q and k must have one type, got {dt} and {k.dtype}")
    _like("dq_out", dq_out, qs, dt)
    _like("dk_out", dk_out, ks, dt)
    keep, dims, nbytes = _rope_dims(qs, q.stride(), ks, k.stride(), dt, None if table is None else table.shape,
                                    bool(interleaved), float(eps), float(q_scale), float(k_scale), dq_out.stride(),
                                    dk_out.stride())
    dev, raw, side = _stream(q, stream)
    D = qs[3:]
    g = dict(grads) if grads else {}
    if side is not None:
        _used(side, q, k, table, dq_out, dk_out, q_weight, k_weight, positions, seq_lens, workspace, *g.values())
    for n, t in (("q", q), ("k", k), ("q_weight", q_weight), ("k_weight", k_weight)):
        if g.get(n) is None:
            g[n] = None if t is None else _out(t, side)
    if workspace is None:
        workspace = _scratch(nbytes, q.device, side)
    _call(
        dev, load().prism_qk_norm_rope_backward, dims, _strided("q", q, dev), _strided("k", k, dev),
        _whole("q_weight", q_weight, D, torch.float32, dev), _whole("k_weight", k_weight, D, torch.float32, dev),
        None if table is None else _whole("table", table, table.shape, torch.float32, dev),
        _whole("positions", positions, qs[:2], torch.int32, dev), _whole("seq_lens", seq_lens, qs[:1], torch.int32, dev),
        _strided("dq_out", dq_out, dev), _strided("dk_out", dk_out, dev), _whole("grads['q']", g["q"], qs, dt, dev),
        _whole("grads['k']", g["k"], ks, dt, dev), _whole("grads['q_weight']", g["q_weight"], D, torch.float32, dev),
        _whole("grads['k_weight']", g["k_weight"], D, torch.float32, dev), *_room(workspace, dev), raw)
    return g


def _state_shape(qs):
    return torch.Size((qs[0], qs[2], qs[3], qs[3]))


def prism_linattn_forward(q, k, v, log_decay, *, scale=1.0, initial_state=None, out=None, final_state=None,
                          seq_lens=None, workspace=None, stream=None, want_state=True, flags=0):
    """Causal linear attention over q, k, v [B,T,H,D] with the decay exp(log_decay[h]) a token:
    S_t = exp(log_decay) S_(t-1) + v_t k_t^T, o_t = scale S_t q_t, S_0 = ``initial_state``
    [B,H,D,D] fp32 (None: zero).  Returns ``(out, final_state)``: out [B,T,H,D] in q's type,
    final_state fp32 (None when ``want_state`` is False and none was passed)."""
    qs, dt = q.shape, q.dtype
    _like("k", k, qs, dt)
    _like("v", v, qs, dt)
    keep, dims, nbytes = _linattn_dims(qs, dt, float(scale), q.stride(), k.stride(), v.stride(), None, int(flags))
    dev, raw, side = _stream(q, stream)
    ss = _state_shape(qs)
    if side is not None:
        _used(side, q, k, v, log_decay, initial_state, out, final_state, seq_lens, workspace)
    if out is None:
        out = _out(q, side)
    if final_state is None and want_state:
        final_state = _new(ss, torch.float32, q.device, side)
    if workspace is None and nbytes:
        workspace = _scratch(nbytes, q.device, side)
    _call(
        dev, load().prism_linattn_forward, dims, _strided("q", q, dev), _strided("k", k, dev),
        _strided("v", v, dev), _whole("log_decay", log_decay, qs[2:3], torch.float32, dev),
        _whole("initial_state", initial_state, ss, torch.float32, dev), _whole("out", out, qs, dt, dev),
        _whole("final_state", final_state, ss, torch.float32, dev), _whole("seq_lens", seq_lens, qs[:1], torch.int32, dev),
        *_room(workspace, dev), raw)
    return out, final_state


def prism_linattn_backward(q, k, v, log_decay, d_out, *, scale=1.0, initial_state=None, d_final_state=None,
                           seq_lens=None, grads=None, workspace=None, stream=None, flags=0):
    """Gradients through prism_linattn_forward given ``d_out`` [B,T,H,D] in q's type (and
    ``d_final_state`` [B,H,D,D] fp32).  Returns a dict: q, k, v in their type and initial_state
    fp32 (None where there was none).  ``grads`` may pass preallocated outputs."""
    qs, dt = q.shape, q.dtype
    _like("k", k, qs, dt)
    _like("v", v, qs, dt)
    _like("d_out", d_out, qs, dt)
    keep, dims, nbytes = _linattn_dims(qs, dt, float(scale), q.stride(), k.stride(), v.stride(), d_out.stride(), int(flags))
    dev, raw, side = _stream(q, stream)
    ss = _state_shape(qs)
    g = dict(grads) if grads else {}
    if side is not None:
        _used(side, q, k, v, log_decay, d_out, initial_state, d_final_state, seq_lens, workspace, *g.values())
    for n, t in (("q", q), ("k", k), ("v", v)):
        if g.get(n) is None:
            g[n] = _out(t, side)
    if g.get("initial_state") is None:
        g["initial_state"] = None if initial_state is None else _new(ss, torch.float32, q.device, side)
    if workspace is None and nbytes:
        workspace = _scratch(nbytes, q.device, side)
    _call(
        dev, load().prism_linattn_backward, dims, _strided("q", q, dev), _strided("k", k, dev),
        _strided("v", v, dev), _whole("log_decay", log_decay, qs[2:3], torch.float32, dev),
        _whole("initial_state", initial_state, ss, torch.float32, dev), _strided("d_out", d_out, dev),
        _whole("d_final_state", d_final_state, ss, torch.float32, dev), _whole("grads['q']", g["q"], qs, dt, dev),
        _whole("grads['k']", g["k"], qs, dt, dev), _whole("grads['v']", g["v"], qs, dt, dev),
        _whole("grads['initial_state']", g["initial_state"], ss, torch.float32, dev),
        _whole("seq_lens", seq_lens, qs[:1], torch.int32, dev),
        *_room(workspace, dev), raw)
    return g


def prism_linattn_decode_step(q, k, v, log_decay, state, *, scale=1.0, slots=None, out=None, stream=None):
    """One token of every sequence: q, k, v [B,H,D]; ``state`` [N,H,D,D] fp32 is updated in
    place.  ``slots`` [B] int32 says which state each sequence has (None: its own index; outside
    0..N-1: the sequence is not there, its output is 0).  Returns out [B,H,D] in q's type."""
    qs, dt = q.shape, q.dtype
    _like("k", k, qs, dt)
    _like("v", v, qs, dt)
    keep, dims = _decode_dims(qs, dt, float(scale), q.stride(), k.stride(), v.stride())
    dev, raw, side = _stream(q, stream)
    N = state.shape[0]
    if side is not None:
        _used(side, q, k, v, log_decay, state, slots, out)
    if out is None:
        out = _out(q, side)
    _call(
        dev, load().prism_linattn_decode_step, dims, _strided("q", q, dev), _strided("k", k, dev),
        _strided("v", v, dev), _whole("log_decay", log_decay, qs[1:2], torch.float32, dev),
        _whole("state", state, (N, qs[1], qs[2], qs[2]), torch.float32, dev), N,
        _whole("slots", slots, qs[:1], torch.int32, dev), _whole("out", out, qs, dt, dev), raw)
    return out


def linattn_status(clear: bool = True) -> int:
    """The word of bounded waits that gave up on the current device (0: none; synchronises)."""
    word = _int(-1)
    _check(load().prism_linattn_status(ctypes.byref(word), 1 if clear else 0))
    return word.value
