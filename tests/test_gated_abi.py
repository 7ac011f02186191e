"""The gated recurrent layer's entry points: every declared symbol is exported, and bad arguments are refused on
the host before anything is launched (CPU only)."""
import ctypes
import os
import re

import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import build, gated, prism

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4
OK, ODD, WS = 0x1000, 0x1008, 0x100000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gated.load()


def pair(v):
    return (ctypes.c_longlong * 2)(*v)


def norm_dims(**kw):
    d = gated.LayerNormDims(B=2, T=8, D=64, dtype=prism.PRISM_BF16, flags=0, eps=1e-5)
    for n, v in kw.items():
        setattr(d, n, pair(v) if isinstance(v, tuple) else v)
    return d


def scan_dims(**kw):
    d = gated.GatedDims(B=2, T=3000, D=64, dtype=prism.PRISM_BF16, flags=0)
    for n, v in kw.items():
        setattr(d, n, pair(v) if isinstance(v, tuple) else v)
    return d


def a(d):
    return ctypes.byref(d)          # holds d for the call


def test_exports(lib):
    src = open(os.path.join(ROOT, "include", "prism_gated.h")).read()
    names = set(re.findall(r"PRISM_API\s+[\w\s\*]+?\b(prism_\w+)\s*\(", src))
    assert names == set(gated.EXPORTS) and all(hasattr(lib, n) for n in names)
    assert int(re.search(r"PRISM_GATED_CHUNK (\d+)", src)[1]) == gated.PRISM_GATED_CHUNK


@pytest.mark.parametrize("field,value,code", [
    ("B", 0, ARG), ("T", -1, ARG), ("D", 0, ARG), ("D", 12, UNSUPPORTED), ("D", 16392, UNSUPPORTED), ("dtype", 2, ARG),
    ("flags", 1, ARG), ("flags", 8, ARG), ("eps", -1e-5, ARG), ("eps", float("nan"), ARG), ("x_stride", (512, 56), ARG),
    ("x_stride", (516, 64), ARG), ("x_stride", (512, 68), ARG), ("x_stride", (0, 64), ARG), ("x_stride", (-512, 64), ARG),
    ("T", 1 << 30, UNSUPPORTED)])
def test_norm_bad_dims(lib, field, value, code):
    d = norm_dims(**{field: value})
    assert lib.prism_layer_norm(a(d), OK, OK, OK, None, OK, None) == code
    assert lib.prism_layer_norm_backward(a(d), OK, OK, None, OK, OK, OK, OK, WS, 1 << 40, None) == code
    if not isinstance(value, tuple):
        assert lib.prism_layer_norm_workspace_bytes(a(d)) == 0


def test_norm_bad_pointers(lib):
    d = norm_dims()
    good = [OK, OK, OK, None, OK]
    for i, p in ((0, None), (4, None)):
        assert lib.prism_layer_norm(a(d), *good[:i], p, *good[i + 1:], None) == ARG
    for i in (0, 1, 2, 4):
        assert lib.prism_layer_norm(a(d), *good[:i], ODD, *good[i + 1:], None) == MISALIGNED
    assert lib.prism_layer_norm(a(d), OK, OK, OK, 0x1002, OK, None) == MISALIGNED
    assert lib.prism_layer_norm(None, *good, None) == ARG
    n = lib.prism_layer_norm_workspace_bytes(a(d))
    assert n > 0 and n % 256 == 0
    good = [OK, None, None, OK, OK, OK, OK]

    def back(p, ws=WS, size=n, dims=d):
        return lib.prism_layer_norm_backward(a(dims), *p, ws, size, None)

    for i in (0, 3, 4):
        assert back([*good[:i], None, *good[i + 1:]]) == ARG
    for i in (0, 1, 3, 4, 5, 6):
        assert back([*good[:i], ODD, *good[i + 1:]]) == MISALIGNED
    assert back([OK, None, 0x1002, *good[3:]]) == MISALIGNED
    assert back(good, ws=None) == WORKSPACE and back(good, size=n - 1) == WORKSPACE and back(good, ws=0x100080) == MISALIGNED
    assert back([*good[:6], None], size=n - 1) == back([*good[:5], None, OK], size=n - 1) == WORKSPACE
    assert back(good, dims=norm_dims(do_stride=(512, 32))) == ARG


@pytest.mark.parametrize("field,value,code", [
    ("B", 0, ARG), ("T", 0, ARG), ("D", -8, ARG), ("D", 20, UNSUPPORTED), ("dtype", 9, ARG), ("flags", 1, ARG),
    ("flags", 16, ARG), ("x_stride", (3000 * 64, 32), ARG), ("f_stride", (3000 * 64, 68), ARG), ("f_stride", (0, 64), ARG),
    ("i_stride", (-192000, 64), ARG), ("i_stride", (192004, 64), ARG), ("T", 1 << 30, UNSUPPORTED)])
def test_scan_bad_dims(lib, field, value, code):
    d = scan_dims(**{field: value})
    assert lib.prism_gated_scan_forward(a(d), *[OK] * 7, None, WS, 1 << 62, None) == code
    assert lib.prism_gated_scan_backward(a(d), *[OK] * 10, None, WS, 1 << 62, None) == code
    if not isinstance(value, tuple):
        assert lib.prism_gated_scan_workspace_bytes(a(d)) == lib.prism_gated_scan_backward_workspace_bytes(a(d)) == 0
        if field != "T":
            d.T = 1
            assert lib.prism_gated_scan_decode_step(a(d), *[OK] * 4, 2, None, OK, None) == code


def test_scan_bad_pointers(lib):
    d = scan_dims()
    n, nb = lib.prism_gated_scan_workspace_bytes(a(d)), lib.prism_gated_scan_backward_workspace_bytes(a(d))
    assert n > 0 and nb > 0
    # x, forget, input_gate, initial_state, out, final_state, states, seq_lens
    good = [OK, OK, OK, None, OK, None, None, None]

    def fwd(p, ws=WS, size=n, dims=d):
        return lib.prism_gated_scan_forward(a(dims), *p, ws, size, None)

    for i in (0, 1, 4):
        assert fwd([*good[:i], None, *good[i + 1:]]) == ARG
    for i in range(7):
        assert fwd([*good[:i], ODD, *good[i + 1:]]) == MISALIGNED
    assert fwd([*good[:7], 0x1001]) == MISALIGNED
    assert fwd(good, ws=None) == WORKSPACE and fwd(good, size=n - 1) == WORKSPACE and fwd(good, ws=0x100010) == MISALIGNED
    assert lib.prism_gated_scan_forward(None, *good, WS, n, None) == ARG
    # x, forget, input_gate, states, d_out, d_final, dx, d_forget, d_input_gate, d_initial, seq_lens
    good = [OK, OK, OK, OK, OK, None, OK, OK, OK, None, None]

    def back(p, ws=WS, size=nb, dims=d):
        return lib.prism_gated_scan_backward(a(dims), *p, ws, size, None)

    for i in (0, 1, 2, 3, 4, 6, 7, 8):            # a gate without its gradient, and the other way round
        assert back([*good[:i], None, *good[i + 1:]]) == ARG
    for i in range(10):
        assert back([*good[:i], ODD, *good[i + 1:]]) == MISALIGNED
    assert back([*good[:10], 0x1003]) == MISALIGNED
    assert back(good, ws=None) == WORKSPACE and back(good, size=nb - 1) == WORKSPACE
    assert back(good, dims=scan_dims(do_stride=(3000 * 64, 8))) == ARG


def test_more_tiles_than_a_grid_has(lib):
    d = scan_dims(B=64, D=1 << 30)
    assert lib.prism_gated_scan_forward(a(d), *[OK] * 7, None, WS, 1 << 62, None) == UNSUPPORTED
    assert lib.prism_gated_scan_workspace_bytes(a(d)) == 0


def test_token_numbers_stay_within_32_bits(lib):
    for dims, f, args in ((norm_dims, lib.prism_layer_norm, [OK] * 3 + [None, OK, None]),
                          (scan_dims, lib.prism_gated_scan_forward, [OK] * 7 + [None, WS, 1 << 62, None])):
        assert f(a(dims(B=1, T=(1 << 30) + 1)), *args) == UNSUPPORTED


def test_short_sequences_need_no_workspace(lib):
    for dtype, T, back in ((prism.PRISM_BF16, 128, 64), (prism.PRISM_F32, 64, 64)):
        many = dict(dtype=dtype, B=64, D=2048)
        assert lib.prism_gated_scan_workspace_bytes(a(scan_dims(T=T, **many))) == 0
        assert lib.prism_gated_scan_workspace_bytes(a(scan_dims(T=T + 1, **many))) > 0
        assert lib.prism_gated_scan_backward_workspace_bytes(a(scan_dims(T=back, **many))) == 0
        assert lib.prism_gated_scan_backward_workspace_bytes(a(scan_dims(T=back + 1, **many))) > 0
        assert lib.prism_gated_scan_workspace_bytes(a(scan_dims(T=500, dtype=dtype))) == 0        # a cluster a chain
        assert lib.prism_gated_scan_workspace_bytes(a(scan_dims(T=2049, dtype=dtype))) > 0
        assert lib.prism_gated_scan_workspace_bytes(a(scan_dims(T=32, **many))) == 0


@pytest.mark.parametrize("flags,fine", [(0, True), (8, True), (1, False), (2, False), (4, False), (9, False), (1 << 31, False)])
def test_flags(lib, flags, fine):
    """The wait check alone, and not for single tokens."""
    d = scan_dims(flags=flags)
    want = WORKSPACE if fine else ARG
    assert lib.prism_gated_scan_forward(a(d), *[OK] * 7, None, None, 0, None) == want
    assert lib.prism_gated_scan_backward(a(d), *[OK] * 10, None, None, 0, None) == want
    if flags:
        assert lib.prism_gated_scan_decode_step(a(scan_dims(T=1, flags=flags)), *[OK] * 4, 2, None, OK, None) == ARG


def test_decode_bad_arguments(lib):
    def call(dims=None, p=(OK, OK, None, OK), n=2, slots=None, out=OK):
        return lib.prism_gated_scan_decode_step(a(dims or scan_dims(T=1)), *p, n, slots, out, None)

    assert call(scan_dims(T=2)) == ARG and call(scan_dims(T=1, D=4)) == UNSUPPORTED
    assert call(n=0) == ARG and call(n=1) == ARG and call(out=None) == ARG and call(out=ODD) == MISALIGNED
    for i in (0, 1, 3):
        p = [OK, OK, None, OK]
        p[i] = None
        assert call(p=p) == ARG
    for i in range(4):
        p = [OK] * 4
        p[i] = ODD
        assert call(p=p) == MISALIGNED
    assert call(slots=0x1002) == MISALIGNED
    assert call(scan_dims(T=1, x_stride=(60, 64))) == ARG
    assert lib.prism_gated_status(None, 0) == ARG


def test_binding_refusals():
    """Shapes, types, layouts and devices are refused with the framework's error."""
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    x, f32 = t(2, 8, 16), torch.float32

    def refused(f, *args, **k):
        with pytest.raises(prism.PrismError):
            f(*args, **k)

    fwd, back, step = (gated.prism_gated_scan_forward, gated.prism_gated_scan_backward, gated.prism_gated_scan_decode_step)
    refused(fwd, x, x)                                                     # on the CPU
    refused(fwd, x, x.float())
    refused(fwd, x, t(2, 7, 16))
    refused(fwd, x, x, input_gate=t(2, 8, 8))
    refused(fwd, x.half(), x.half())
    refused(fwd, x[0], x[0])
    refused(fwd, x.transpose(1, 2), x.transpose(1, 2))
    refused(fwd, t(2, 0, 16), t(2, 0, 16))
    refused(back, x, x, t(2, 1, 16, dtype=f32), x.float())
    refused(back, x, x, t(2, 1, 16, dtype=f32), t(2, 8, 8))
    refused(step, t(2, 16), t(2, 16), t(2, 16, dtype=f32))
    refused(step, t(2, 16), t(2, 8), t(2, 16, dtype=f32))
    refused(step, x, x, t(2, 16, dtype=f32))
    for f, args in ((fwd, (t(2, 8, 12),) * 2), (step, (t(2, 12), t(2, 12), t(2, 12, dtype=f32))), (gated.prism_layer_norm, (t(1, 1, 16392),)),
                    (gated.prism_layer_norm, (t(2, 8, 12),))):
        with pytest.raises(prism.PrismError, match="multiple of 8"):
            f(*args)
    refused(gated.prism_layer_norm, x)                                     # on the CPU
    refused(gated.prism_layer_norm, x[0])
    refused(gated.prism_layer_norm, x.half())
    refused(gated.prism_layer_norm, x.transpose(1, 2))
    refused(gated.prism_layer_norm_backward, x, x.float())
    refused(gated.prism_layer_norm_backward, x, t(2, 8, 8))
    assert gated.gated_scan_states(t(2, 129, 16)).shape == (2, 3, 16)
