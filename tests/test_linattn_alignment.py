"""Pointers to words that are not aligned to them are refused on the host (CPU): a kernel that reads
them would fault."""
import ctypes

import pytest

from linear_recurrent_sequence_causal_gb300 import build, linattn, prism

MISALIGNED = 3
OK, ODD = 0x1000, 0x1002


@pytest.fixture(scope="module")
def lib():
    build.build()
    return linattn.load()


def rope_dims():
    return linattn.RopeDims(B=2, T=8, Hq=4, Hk=2, d=64, rotary_dim=64, table_rows=8, dtype=prism.PRISM_BF16, flags=0,
                            eps=1e-6, q_scale=1.0, k_scale=1.0)


def attn_dims(T):
    return linattn.LinattnDims(B=2, T=T, H=2, d=64, dtype=prism.PRISM_BF16, flags=0, scale=1.0)


@pytest.mark.parametrize("positions,lens", [(ODD, None), (None, ODD), (OK, ODD), (ODD, OK), (0x1001, None)])
def test_positions_and_lengths_of_the_norm(lib, positions, lens):
    d = rope_dims()
    a = ctypes.addressof(d)
    assert lib.prism_qk_norm_rope(a, *[OK] * 5, positions, lens, OK, OK, None) == MISALIGNED
    assert lib.prism_qk_norm_rope_backward(a, *[OK] * 5, positions, lens, *[OK] * 6, 0x100000, 1 << 30, None) == MISALIGNED


@pytest.mark.parametrize("decay,lens", [(ODD, None), (OK, ODD), (0x1003, OK)])
def test_decays_and_lengths_of_linear_attention(lib, decay, lens):
    d = attn_dims(64)
    a = ctypes.addressof(d)
    assert lib.prism_linattn_forward(a, OK, OK, OK, decay, None, OK, None, lens, 0x100000, 1 << 40, None) == MISALIGNED
    assert lib.prism_linattn_backward(a, OK, OK, OK, decay, None, OK, None, OK, OK, OK, None, lens, 0x100000, 1 << 40,
                                      None) == MISALIGNED


@pytest.mark.parametrize("decay,slots", [(ODD, None), (OK, ODD)])
def test_decays_and_slots_of_single_tokens(lib, decay, slots):
    d = attn_dims(1)
    assert lib.prism_linattn_decode_step(ctypes.addressof(d), OK, OK, OK, decay, OK, 2, slots, OK, None) == MISALIGNED
