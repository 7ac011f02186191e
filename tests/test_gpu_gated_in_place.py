"""States written over those that came in, where two lanes of a warp hold the same channel: tiles of 32 channels that look back,
with sequences that end in their first tile."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import gated

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,B,T,D", [(torch.float32, 100, 300, 504), (torch.bfloat16, 1500, 300, 24)])
def test_states_in_place(dtype, B, T, D):
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, f, i, do = (n(B, T, D).to(dtype) for _ in range(4))
    s0, ds = n(B, D), n(B, D)
    lens = torch.randint(0, 130, (B,), generator=g, device="cuda", dtype=torch.int32)
    states = gated.gated_scan_states(x)
    out, final = gated.prism_gated_scan_forward(x, f, input_gate=i, initial_state=s0, seq_lens=lens, states=states)
    d0 = gated.prism_gated_scan_backward(x, f, states, do, input_gate=i, d_final_state=ds, seq_lens=lens,
                                         want_initial_state=True)["initial_state"]
    for _ in range(5):
        s, d = s0.clone(), ds.clone()
        gated.prism_gated_scan_forward(x, f, input_gate=i, initial_state=s, final_state=s, seq_lens=lens, out=out)
        gated.prism_gated_scan_backward(x, f, states, do, input_gate=i, d_final_state=d, seq_lens=lens,
                                        grads={"initial_state": d})
        assert torch.equal(s, final) and torch.equal(d, d0)
    assert gated.gated_status() == 0
