"""Single tokens over a long time: the decay of a head that hardly forgets is not off by the same rounding
in every step.

With v = 0 a state is exp(N log_decay) of what it was after N tokens.  Each step rounds every
element once or twice, by u = 2^-24 at most and independently, so the mean relative error of D^2
elements is within 6 u sqrt(2 N / 3) / D; the decay itself is known to 2 ulp of its difference from
1, which adds 4 u N |log_decay|.  (exp(log_decay) in fp32 is off by about u in every step, always in one
direction: N u after N of them.)"""
import math

import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import linattn
from tests import linattn_oracle as lo

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_steps(dtype):
    D, N = 64, 4096
    ld = -2.0 ** -12 * (1 + torch.arange(8) / 8)
    H = len(ld)
    off = ((torch.exp(ld).double() - torch.exp(ld.double())).abs() / lo.U).max().item()
    assert off > 0.2                                           # the rounding that would add up
    g = torch.Generator(device="cuda").manual_seed(0)
    first = torch.rand(1, H, D, D, generator=g, device="cuda") + 0.5
    state, q = first.clone(), torch.randn(1, H, D, generator=g, device="cuda").to(dtype)
    zero, cl = torch.zeros_like(q), ld.cuda()
    for _ in range(N):
        linattn.prism_linattn_decode_step(q, q, zero, cl, state)
    want = first.double() * torch.exp(N * ld.double()).cuda()[None, :, None, None]
    mean = ((state.double() - want) / want).mean((0, 2, 3)).abs().cpu()
    bound = lo.U * (6 * math.sqrt(2 * N / 3) / D + 4 * N * ld.double().abs())
    assert (mean <= bound).all(), (mean / lo.U, bound / lo.U)


@pytest.mark.parametrize("ld", [-0.4999, -0.5, -0.5001, -3.0, -40.0, -200.0, float("-inf"), 0.0])
def test_one_step_of_any_decay(ld):
    """The share of an old state that is far larger than what is added stays exact to a few ulp."""
    D = 32
    g = torch.Generator().manual_seed(1)
    x = [torch.randn(1, 1, 1, D, generator=g) for _ in range(3)]
    s0 = torch.randn(1, 1, D, D, generator=g) * 2.0 ** 30
    state, dec = s0.cuda(), torch.tensor([ld])
    linattn.prism_linattn_decode_step(*(t[0].cuda() for t in x), dec.cuda(), state)
    _, s = lo.linattn(*(t.double() for t in x), dec.double(), 1.0, s0.double())
    _, m = lo.linattn(*(t.double().abs() for t in x), dec.double(), 1.0, s0.double().abs())
    lo.assert_within(state, s, 16 * lo.U * m, "state")
