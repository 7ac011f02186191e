"""Token inputs expanded over tokens or sequences (CPU, with the library of test_linattn_streams that only takes notes):
the C entry points take a token step of 0 for "contiguous", so a view of one token's memory as [B,T,D] would be read past
its end.  Such a call is refused before anything is launched."""
import types

import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import gated, prism
from tests.test_gated_streams import CALLS, operands, world  # noqa: F401
from tests.test_linattn_streams import gpu

TOKENS = {"norm": ("x",), "norm_backward": ("x", "do"), "forward": ("x", "f", "i"), "backward": ("x", "f", "i", "do")}


def expanded(t, over):
    """t's shape over the memory of its first token, sequence or value."""
    B, T, D = t.shape
    part = {"tokens": torch.zeros(B, 1, D, dtype=t.dtype), "sequences": torch.zeros(1, T, D, dtype=t.dtype),
            "both": torch.zeros(D, dtype=t.dtype)}[over]
    return gpu(part.expand(B, T, D))


@pytest.mark.parametrize("call", TOKENS)
@pytest.mark.parametrize("over", ["tokens", "sequences", "both"])
def test_expanded_inputs_are_refused(world, call, over):  # noqa: F811
    for n in TOKENS[call]:
        x = operands()
        setattr(x, n, expanded(getattr(x, n), over))
        with pytest.raises(prism.PrismError, match="memory of its own"):
            CALLS[call](x)
    assert not world.calls and not world.made


@pytest.mark.parametrize("call", TOKENS)
def test_tokens_closer_than_they_are_wide(world, call):  # noqa: F811
    """Windows of channels that share memory from one token to the next."""
    for n in TOKENS[call]:
        x = operands()
        B, T, D = x.x.shape
        line = torch.zeros(B * T * 8 + D, dtype=torch.bfloat16)
        setattr(x, n, gpu(line.as_strided((B, T, D), (T * 8, 8, 1))))
        with pytest.raises(prism.PrismError, match="memory of its own"):
            CALLS[call](x)
    assert not world.calls


@pytest.mark.parametrize("n", ["x1", "f1", "i1"])
def test_single_tokens_expanded_over_the_batch(world, n):  # noqa: F811
    x = operands()
    setattr(x, n, gpu(torch.zeros(16, dtype=torch.bfloat16).expand(2, 16)))
    with pytest.raises(prism.PrismError, match="memory of its own"):
        CALLS["decode"](x)
    assert not world.calls


def test_the_gradient_of_a_weighted_sum(world):  # noqa: F811
    """What automatic differentiation hands on for it lies in one vector's memory."""
    h, seen = torch.zeros(2, 200, 16, dtype=torch.bfloat16, requires_grad=True), []
    h.register_hook(seen.append)
    (h.sum(1) * torch.ones(16)).sum().backward()
    d, x = seen[0], operands()
    assert d.stride()[1] == 0
    with pytest.raises(prism.PrismError, match="d_out: every token"):
        gated.prism_gated_scan_backward(x.x, x.f, x.st, gpu(d), input_gate=x.i)
    gated.prism_gated_scan_backward(x.x, x.f, x.st, gpu(d.contiguous()), input_gate=x.i)
    assert len(world.calls) == 1


def test_a_step_that_is_never_taken_may_be_anything(world):  # noqa: F811
    """One sequence, one token: no memory is shared."""
    x = types.SimpleNamespace(**vars(operands()))
    one = lambda t, B, T: gpu(torch.zeros(B, T, 16, dtype=t.dtype).as_strided((B, T, 16), (T * 16 if B > 1 else 0, 16 if T > 1 else 0, 1)))  # noqa: E731
    for B, T in ((1, 200), (2, 1)):
        gated.prism_layer_norm(one(x.x, B, T))
        d = gated.LayerNormDims.from_address(world.calls[-1][1][0])
        assert list(d.x_stride) == [T * 16, 16]
