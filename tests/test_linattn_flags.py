"""The flags of the linear attention entry points (CPU): the wait check alone, and not for single tokens."""
import ctypes

import pytest

from linear_recurrent_sequence_causal_gb300 import build, linattn, prism


@pytest.fixture(scope="module")
def lib():
    build.build()
    return linattn.load()


@pytest.mark.parametrize("flags,fine", [(0, True), (8, True), (1, False), (2, False), (4, False), (9, False), (1 << 31, False)])
def test_flags(lib, flags, fine):
    d = linattn.LinattnDims(B=1, T=4096, H=1, d=64, dtype=prism.PRISM_BF16, flags=flags, scale=1.0)
    a = ctypes.addressof(d)
    # past the dims the missing workspace is what is refused
    want = 4 if fine else 1
    assert lib.prism_linattn_forward(a, *[0x1000] * 4, None, 0x1000, None, None, None, 0, None) == want
    assert lib.prism_linattn_backward(a, *[0x1000] * 4, None, 0x1000, None, *[0x1000] * 3, None, None, None, 0, None) == want
    d0 = linattn.LinattnDims(B=1, T=4096, H=1, d=64, dtype=prism.PRISM_BF16, flags=0, scale=1.0)
    size = lib.prism_linattn_workspace_bytes(ctypes.addressof(d0))
    assert size > 0 and lib.prism_linattn_workspace_bytes(a) == (size if fine else 0)


@pytest.mark.parametrize("flags", [1, 8])
def test_single_tokens_take_no_flags(lib, flags):
    d = linattn.LinattnDims(B=1, T=1, H=1, d=64, dtype=prism.PRISM_BF16, flags=flags, scale=1.0)
    assert lib.prism_linattn_decode_step(ctypes.addressof(d), *[0x1000] * 5, 1, None, 0x1000, None) == 1
