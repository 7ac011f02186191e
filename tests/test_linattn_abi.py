"""The linear attention layer's entry points: every declared symbol is exported, and bad
arguments are refused on the host before anything is launched (CPU only)."""
import ctypes
import os
import re

import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import build, linattn, prism

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return linattn.load()


def rope_dims(**kw):
    base = dict(B=2, T=8, Hq=4, Hk=2, d=64, rotary_dim=64, table_rows=8, dtype=prism.PRISM_BF16, flags=0, eps=1e-6,
                q_scale=1.0, k_scale=1.0)
    base.update(kw)
    return linattn.RopeDims(**base)


def attn_dims(**kw):
    base = dict(B=2, T=64, H=2, d=64, dtype=prism.PRISM_BF16, flags=0, scale=1.0)
    base.update(kw)
    return linattn.LinattnDims(**base)


def rope(lib, d, ptrs):
    return lib.prism_qk_norm_rope(ctypes.addressof(d), *ptrs, None)


def test_exports(lib):
    src = open(os.path.join(ROOT, "include", "prism_linattn.h")).read()
    names = set(re.findall(r"PRISM_API\s+[\w\s\*]+?\b(prism_\w+)\s*\(", src))
    assert names == set(linattn.EXPORTS) and all(hasattr(lib, n) for n in names)


@pytest.mark.parametrize("field,value,code", [
    ("B", 0, ARG), ("T", -1, ARG), ("Hq", 0, ARG), ("Hk", 0, ARG), ("d", 0, ARG), ("d", 48, UNSUPPORTED),
    ("d", 256, UNSUPPORTED), ("rotary_dim", 12, UNSUPPORTED), ("rotary_dim", 72, UNSUPPORTED), ("rotary_dim", -8, UNSUPPORTED),
    ("dtype", 7, ARG), ("flags", 2, ARG), ("eps", -1.0, ARG), ("eps", float("nan"), ARG), ("table_rows", -1, ARG),
    ("table_rows", 7, ARG), ("table_rows", 0, ARG), ("q_stride", (1024, 100), ARG), ("k_stride", (1024, 132), ARG),
    ("q_stride", (-2048, 256), ARG), ("q_stride", (2044, 256), ARG)])
def test_rope_bad_dims(lib, field, value, code):
    d = rope_dims()
    setattr(d, field, (ctypes.c_longlong * 2)(*value) if isinstance(value, tuple) else value)
    assert rope(lib, d, [0x1000] * 5 + [None, None] + [0x1000] * 2) == code


def test_rope_bad_pointers(lib):
    d = rope_dims()
    good = [0x1000] * 5 + [None, None] + [0x1000] * 2
    for i in (0, 1, 4, 7, 8):                       # q, k, table, q_out, k_out
        p = list(good)
        p[i] = None
        assert rope(lib, d, p) == ARG
    for i in (0, 2, 4, 8):
        p = list(good)
        p[i] = 0x1008
        assert rope(lib, d, p) == MISALIGNED
    assert lib.prism_qk_norm_rope(None, *good, None) == ARG
    n = lib.prism_qk_norm_rope_workspace_bytes(ctypes.addressof(d))
    assert n > 0 and lib.prism_qk_norm_rope_workspace_bytes(ctypes.addressof(rope_dims(d=48))) == 0
    ok = [0x1000] * 5 + [None, None] + [0x1000] * 6

    def back(p, ws=0x100000, size=1 << 30, dims=d):
        return lib.prism_qk_norm_rope_backward(ctypes.addressof(dims), *p, ws, size, None)

    for i in (0, 1, 7, 8, 9, 10):                   # q, k, dq_out, dk_out, dq, dk
        p = list(ok)
        p[i] = None
        assert back(p) == ARG
    assert back(ok, ws=None) == WORKSPACE and back(ok, size=n - 1) == WORKSPACE and back(ok, ws=0x100010) == MISALIGNED
    bad = rope_dims()
    bad.dq_stride[0], bad.dq_stride[1] = 4096, 8     # tokens that overlap
    assert back(ok, dims=bad) == ARG


@pytest.mark.parametrize("field,value,code", [
    ("B", 0, ARG), ("T", 0, ARG), ("H", -1, ARG), ("d", 0, ARG), ("d", 96, UNSUPPORTED), ("dtype", 2, ARG), ("flags", 1, ARG),
    ("q_stride", (8192, 64), ARG), ("k_stride", (8192, 132), ARG), ("v_stride", (0, 128), ARG), ("T", 1 << 30, UNSUPPORTED)])
def test_linattn_bad_dims(lib, field, value, code):
    d = attn_dims()
    setattr(d, field, (ctypes.c_longlong * 2)(*value) if isinstance(value, tuple) else value)
    a = ctypes.addressof(d)
    assert lib.prism_linattn_forward(a, *[0x1000] * 8, 0x100000, 1 << 40, None) == code
    assert lib.prism_linattn_backward(a, *[0x1000] * 12, 0x100000, 1 << 40, None) == code
    if not isinstance(value, tuple):
        assert lib.prism_linattn_workspace_bytes(a) == 0 and lib.prism_linattn_backward_workspace_bytes(a) == 0


def test_linattn_bad_pointers(lib):
    d = attn_dims(T=4096)
    a = ctypes.addressof(d)
    n, nb = lib.prism_linattn_workspace_bytes(a), lib.prism_linattn_backward_workspace_bytes(a)
    assert n > 0 and nb > 0 and n % 256 == 0 and nb % 256 == 0
    ok = [0x1000] * 4 + [None, 0x1000, None, None]
    for i in (0, 1, 2, 3, 5):
        p = list(ok)
        p[i] = None
        assert lib.prism_linattn_forward(a, *p, 0x100000, 1 << 40, None) == ARG
    for i in (0, 2, 4, 5, 6):
        p = list(ok)
        p[i] = 0x1004
        assert lib.prism_linattn_forward(a, *p, 0x100000, 1 << 40, None) == MISALIGNED
    assert lib.prism_linattn_forward(a, *ok, None, 0, None) == WORKSPACE
    assert lib.prism_linattn_forward(a, *ok, 0x100000, n - 1, None) == WORKSPACE
    assert lib.prism_linattn_forward(a, *ok, 0x100010, n, None) == MISALIGNED
    ok = [0x1000] * 4 + [None, 0x1000, None] + [0x1000] * 3 + [None, None]
    for i in (0, 3, 5, 7, 8, 9):
        p = list(ok)
        p[i] = None
        assert lib.prism_linattn_backward(a, *p, 0x100000, 1 << 40, None) == ARG
    assert lib.prism_linattn_backward(a, *ok, 0x100000, nb - 1, None) == WORKSPACE
    assert lib.prism_linattn_backward(None, *ok, 0x100000, nb, None) == ARG


def test_decode_bad_arguments(lib):
    d = attn_dims(T=1)

    def call(dims=d, p=(0x1000,) * 5, n=2, slots=None, out=0x1000):
        return lib.prism_linattn_decode_step(ctypes.addressof(dims), *p, n, slots, out, None)

    assert call(attn_dims(T=2)) == ARG and call(attn_dims(T=1, d=8)) == UNSUPPORTED
    assert call(n=0) == ARG and call(n=1) == ARG and call(out=None) == ARG and call(out=0x1001) == MISALIGNED
    for i in range(5):
        p = [0x1000] * 5
        p[i] = None
        assert call(p=p) == ARG
    assert lib.prism_linattn_status(None, 0) == ARG


def test_binding_refusals():
    """Shapes, types, layouts and devices are refused with the framework's error."""
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    q = t(2, 8, 2, 16)
    ld = t(2, dtype=torch.float32)

    def refused(f, *a, **k):
        with pytest.raises(prism.PrismError):
            f(*a, **k)

    fwd, back, step = linattn.prism_linattn_forward, linattn.prism_linattn_backward, linattn.prism_linattn_decode_step
    refused(fwd, q, q, q, ld)                                              # on the CPU
    refused(fwd, q, q, t(2, 8, 2, 16, dtype=torch.float32), ld)            # mixed types
    refused(fwd, q, t(2, 7, 2, 16), q, ld)                                 # mixed lengths
    refused(fwd, q.half(), q.half(), q.half(), ld)
    refused(fwd, q[0], q[0], q[0], ld)
    refused(fwd, q.transpose(1, 2), q.transpose(1, 2), q.transpose(1, 2), ld)
    refused(fwd, t(2, 0, 2, 16), t(2, 0, 2, 16), t(2, 0, 2, 16), ld)       # no tokens
    refused(back, q, q, q, ld, t(2, 8, 2, 16, dtype=torch.float32))
    refused(step, t(2, 2, 16), t(2, 2, 16), t(2, 2, 16), ld, t(2, 2, 16, 16, dtype=torch.float32))
    rope, rback = linattn.prism_qk_norm_rope, linattn.prism_qk_norm_rope_backward
    table = t(8, 16, dtype=torch.float32)
    refused(rope, q, q, table)                                             # on the CPU
    refused(rope, q, t(2, 8, 2, 32), table)
    refused(rope, q, q.float(), table)
    refused(rope, q, q, table[0])
    refused(rback, q, q, table, q, t(2, 8, 1, 16))
