"""A refusal of the gated layer's binding names the argument that is at fault (CPU)."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import gated, linattn, prism
from tests.test_gated_streams import CALLS, OPERANDS, operands, world  # noqa: F401
from tests.test_linattn_streams import Stream, gpu

NAMES = {"x": "x", "x1": "x", "f": "forget", "f1": "forget", "i": "input_gate", "i1": "input_gate", "w": "weight", "b": "bias",
         "lens": "seq_lens", "do": "d_out", "st": "states", "ds": "d_final_state", "slots": "slots"}


@pytest.mark.parametrize("call", CALLS)
def test_a_tensor_on_the_cpu(world, call):  # noqa: F811
    for n in ("x1" if call == "decode" else "x", *OPERANDS[call]):
        x = operands()
        setattr(x, n, getattr(x, n).as_subclass(torch.Tensor))
        name = NAMES.get(n, "state" if call == "decode" else "initial_state")
        with pytest.raises(prism.PrismError, match=rf": {name} must be a (contiguous )?CUDA tensor"):
            CALLS[call](x)
    assert not world.calls


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_device(world, call):  # noqa: F811
    with pytest.raises(prism.PrismError, match="stream is on device 1, x on device 0"):
        CALLS[call](operands(), stream=Stream(0x51de, 1))


def test_linear_attention_names_its_own(world):  # noqa: F811
    q, k = torch.zeros(2, 8, 2, 16), gpu(torch.zeros(2, 8, 2, 16))
    with pytest.raises(prism.PrismError, match=": q must be a CUDA tensor"):
        linattn.prism_qk_norm_rope(q, k, None)
    with pytest.raises(prism.PrismError, match=": k must be a CUDA tensor"):
        linattn.prism_qk_norm_rope(k, q, None)
    with pytest.raises(prism.PrismError, match="x must be a CUDA tensor"):
        gated.prism_layer_norm(q[:, :, 0])
