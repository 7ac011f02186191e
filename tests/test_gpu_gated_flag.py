"""Where the check of the look back's failure path acts: in tiles that look back, and nowhere else."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import gated, prism

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,D,looks", [(2, 8, 72, False), (2, 30, 72, False), (2, 64, 72, False), (2, 500, 72, False), (2, 3000, 72, True)])
def test_the_flag_acts_where_a_tile_looks_back(B, T, D, looks, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    x, f, i, d = (torch.randn(B, T, D, generator=g, device="cuda").to(dtype) for _ in range(4))
    states = gated.gated_scan_states(x)
    how = dict(input_gate=i, flags=prism.PRISM_FLAG_CHECK_WAIT_TIMEOUT)
    want = gated.prism_gated_scan_forward(x, f, input_gate=i, states=states)
    wg = gated.prism_gated_scan_backward(x, f, states, d, input_gate=i)
    assert gated.gated_status() == 0
    for call in (lambda: gated.prism_gated_scan_forward(x, f, **how), lambda: gated.prism_gated_scan_backward(x, f, states, d, **how)):
        got = call()
        assert (gated.gated_status() != 0) == looks
        for a, b in zip(got.values(), wg.values()) if isinstance(got, dict) else zip(got, want):
            assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sequences_of_one_tile_do_not_look_back(dtype):
    x, f = (torch.randn(2, 3000, 72, device="cuda").to(dtype) for _ in range(2))
    lens = torch.tensor([64, 1], device="cuda", dtype=torch.int32)
    gated.prism_gated_scan_forward(x, f, seq_lens=lens, flags=prism.PRISM_FLAG_CHECK_WAIT_TIMEOUT)
    assert gated.gated_status() == 0
