"""Token inputs of the linear attention layer expanded over tokens or sequences (CPU): the C entry points take a token step
of 0 for "contiguous", so a view of one token's memory as [B,T,H,D] would be read past its end.  Such a call is
refused before anything is launched."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import linattn, prism
from tests.test_linattn_streams import gpu, operands, world  # noqa: F401

CALLS = {
    "rope": lambda q, k, v, d, x: linattn.prism_qk_norm_rope(q, k, x.table),
    "rope_backward": lambda q, k, v, d, x: linattn.prism_qk_norm_rope_backward(q, k, x.table, v, d),
    "forward": lambda q, k, v, d, x: linattn.prism_linattn_forward(q, k, v, x.ld),
    "backward": lambda q, k, v, d, x: linattn.prism_linattn_backward(q, k, v, x.ld, d),
}
READS = {"rope": 2, "rope_backward": 4, "forward": 3, "backward": 4}
SHAPE = (2, 8, 2, 16)


def token(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


VIEWS = {"tokens": lambda: token(2, 1, 2, 16).expand(SHAPE), "sequences": lambda: token(1, 8, 2, 16).expand(SHAPE),
         "both": lambda: token(2, 16).expand(SHAPE), "windows": lambda: token(600).as_strided(SHAPE, (128, 16, 16, 1))}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("view", VIEWS)
def test_expanded_inputs_are_refused(world, call, view):  # noqa: F811
    for n in range(READS[call]):
        t = [gpu(token(*SHAPE)) for _ in range(4)]
        t[n] = gpu(VIEWS[view]())
        with pytest.raises(prism.PrismError, match="memory of its own"):
            CALLS[call](*t, operands())
    assert not world.calls


@pytest.mark.parametrize("n", range(3))
def test_single_tokens_expanded_over_the_batch(world, n):  # noqa: F811
    x, t = operands(), [gpu(token(2, 2, 16)) for _ in range(3)]
    t[n] = gpu(token(2, 16).expand(2, 2, 16))
    with pytest.raises(prism.PrismError, match="memory of its own"):
        linattn.prism_linattn_decode_step(*t, x.ld, x.s)
    assert not world.calls


def test_a_step_that_is_never_taken_may_be_anything(world):  # noqa: F811
    for B, T in ((1, 8), (2, 1)):
        q, k = (gpu(token(B, T, 2, 16).as_strided((B, T, 2, 16), (T * 32 if B > 1 else 0, 32 if T > 1 else 0, 16, 1))) for _ in "qk")
        linattn.prism_qk_norm_rope(q, k, operands().table)
        d = linattn.RopeDims.from_address(world.calls[-1][1][0])
        assert list(d.q_stride) == list(d.k_stride) == [T * 32, 32]
