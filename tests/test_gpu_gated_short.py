"""Short sequences of many channels, where a thread takes four channels instead of two: the bits of the same sequences in
small batches, and a part of them against the 64-bit oracle."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import gated
from tests import gated_oracle as go
from tests.test_gpu_gated_scan import dev, make

pytestmark = pytest.mark.gpu


def run(c, part, resumed, lens):
    s = slice(*part)
    states = gated.gated_scan_states(c["x"][s]).fill_(7.0)
    out, final = gated.prism_gated_scan_forward(c["x"][s], c["f"][s], input_gate=None if c["i"] is None else c["i"][s],
                                                initial_state=c["s0"][s] if resumed else None, seq_lens=lens[s], states=states)
    return out, final, states


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("resumed", [True, False])
@pytest.mark.parametrize("B,T,D", [(1000, 1, 264), (1000, 8, 264), (2000, 3, 264), (1100, 31, 488), (8200, 9, 64), (66000, 2, 8)])
def test_four_channels_a_thread(B, T, D, resumed, gate, dtype):
    z = make(B, T, D, dtype, gate, fused=True)
    c = dev(z, True)
    lens = torch.randint(0, T + 1, (B,), generator=torch.Generator().manual_seed(B), dtype=torch.int32).cuda()
    whole = run(c, (0, B), resumed, lens)
    # fewer than 2^17 channels: two a thread; the last batch as large as the others, since longer sequences of fewer than
    # 2^15 channels go in tiles, whose sums are in another order
    step = min(B, 100000 // D)
    for b in range(0, B, step):
        b = min(b, B - step)
        for a, want in zip(whole, run(c, (b, b + step), resumed, lens)):
            assert torch.equal(a[b:b + step], want)
    n = 40
    cut = {k: None if t is None else t[:n] for k, t in z.items()}
    want = go.scan(cut["x"], cut["f"], cut["i"], cut["s0"] if resumed else None, lens[:n].cpu())
    go.assert_within(whole[0][:n], want["out"], want["err"][:, 1:], "out", z["x"].dtype)
    go.assert_within(whole[1][:n], want["final"], want["err"][:, -1] + 2 * go.U * want["mag"][:, -1], "final state")
