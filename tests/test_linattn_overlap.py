"""States written over states that other CTAs of the same call still read are refused on the host (CPU)."""
import ctypes

import pytest

from linear_recurrent_sequence_causal_gb300 import build, linattn, prism

ARG, WORKSPACE = 1, 4
OK, STATE, OTHER = 0x1000, 0x10000, 0x20000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return linattn.load()


def dims(T):
    return linattn.LinattnDims(B=1, T=T, H=1, d=64, dtype=prism.PRISM_BF16, flags=0, scale=1.0)


def test_a_state_in_place_where_a_sequence_is_cut(lib):
    """Past this check the missing workspace is what is refused."""
    d = dims(4096)
    a = ctypes.addressof(d)
    assert lib.prism_linattn_workspace_bytes(a) > 0
    call = lambda s0, s1: lib.prism_linattn_forward(a, OK, OK, OK, OK, s0, OK, s1, None, None, 0, None)  # noqa: E731
    assert call(STATE, STATE) == ARG
    assert call(STATE, OTHER) == call(None, STATE) == call(STATE, None) == call(None, None) == WORKSPACE


@pytest.mark.parametrize("T", [64, 4096])
def test_state_gradients_in_place(lib, T):
    d = dims(T)
    a = ctypes.addressof(d)

    def call(s0, ds, out, ws=None):
        return lib.prism_linattn_backward(a, OK, OK, OK, OK, s0, OK, ds, OK, OK, OK, out, None, ws, 0, None)

    assert call(STATE, OTHER, OTHER) == call(STATE, OTHER, STATE) == call(None, STATE, STATE) == ARG
    if T == 4096:
        assert call(STATE, OTHER, 0x30000) == call(STATE, OTHER, None) == WORKSPACE
