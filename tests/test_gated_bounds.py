"""Sizes at the ends of what the gated scan's 32-bit numbers hold (CPU)."""
import ctypes

import pytest

from linear_recurrent_sequence_causal_gb300 import build, gated, prism

UNSUPPORTED, WORKSPACE = 2, 4
OK, WS = 0x1000, 0x100000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gated.load()


@pytest.mark.parametrize("dtype", [prism.PRISM_BF16, prism.PRISM_F32])
@pytest.mark.parametrize("D", [(1 << 30) + 8, (1 << 31) - 64, (1 << 31) - 8])
def test_more_channels_than_strips_are_counted(lib, D, dtype):
    """(D + 63) / 64 strips and the channels that they end at must stay below 2^31."""
    for T in (1, 9, 3000):
        d = gated.GatedDims(B=1, T=T, D=D, dtype=dtype, flags=0)
        a = ctypes.addressof(d)
        assert lib.prism_gated_scan_workspace_bytes(a) == lib.prism_gated_scan_backward_workspace_bytes(a) == 0
        assert lib.prism_gated_scan_forward(a, *[OK] * 7, None, None, 0, None) == UNSUPPORTED
        assert lib.prism_gated_scan_backward(a, *[OK] * 10, None, None, 0, None) == UNSUPPORTED
        if T == 1:
            assert lib.prism_gated_scan_decode_step(a, *[OK] * 4, 1, None, OK, None) == UNSUPPORTED


def test_the_widest_layer(lib):
    d = gated.GatedDims(B=1, T=3000, D=1 << 30, dtype=prism.PRISM_BF16, flags=0)
    a = ctypes.addressof(d)
    assert lib.prism_gated_scan_workspace_bytes(a) > 0 and lib.prism_gated_scan_backward_workspace_bytes(a) > 0
    assert lib.prism_gated_scan_forward(a, *[OK] * 7, None, None, 0, None) == WORKSPACE
