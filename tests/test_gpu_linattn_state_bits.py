"""The 24 bits of the states that the bf16 path of linear attention returns.

``STATE`` is derived for one token's share of a returned state, in units of
u = 2^-24: the weight lambda^f, whose exponent |x| <= 2 is off by 3 u |x| (4) and exp2f by 2 ulp (4);
its product with the key (1); what three bf16 terms leave (1); three sums of the tensor core, cut off
and not rounded (6); 3 for each of at most 11 chunks after it (33); the join of the runs, another weight
and a sum (10); together 59.
Two terms would leave up to 256 u (test_linattn_state_bits, on the CPU)."""
import pytest
import torch

from linear_recurrent_sequence_causal_gb300 import linattn
from tests import linattn_oracle as lo
from tests.test_gpu_linattn import make
from tests.test_gpu_linattn_runs import runs

pytestmark = pytest.mark.gpu
STATE = 59 * lo.U


@pytest.mark.parametrize("T", [7, 100, 1300])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
def test_returned_states_hold_24_bits(D, T):
    """One token's share of final_state and of d_initial_state on the bf16 path, while the state still
    remembers it by a quarter: one token of each sequence has a value, the others have none."""
    at = sorted({0, 5 % T, 127 % T, T // 2, T - 2})
    B, ld = len(at), torch.tensor([0.0, -1e-4, -1e-3])
    x = make(B, T, 3, D, "bf16")
    v, do = torch.zeros_like(x["v"]), torch.zeros_like(x["do"])
    for b, t in enumerate(at):
        v[b, t], do[b, t] = x["v"][b, t], x["do"][b, t]
    if T == 1300:
        assert min(runs(x)) > 1
    cl = ld.cuda()
    _, fs = linattn.prism_linattn_forward(x["q"].cuda(), x["k"].cuda(), v.cuda(), cl)
    g = linattn.prism_linattn_backward(x["q"].cuda(), x["k"].cuda(), v.cuda(), cl, do.cuda(), scale=0.5,
                                       initial_state=torch.zeros(B, 3, D, D, device="cuda"))
    wl = ld.double()
    for b, t in enumerate(at):
        k, q = x["k"][b, t].double(), x["q"][b, t].double()
        left = torch.exp((T - 1 - t) * wl)[:, None, None]
        want = left * x["v"][b, t].double()[:, :, None] * k[:, None, :]
        lo.assert_within(fs[b], want, STATE * want.abs(), f"final_state of token {t}")
        want = torch.exp((t + 1) * wl)[:, None, None] * 0.5 * x["do"][b, t].double()[:, :, None] * q[:, None, :]
        lo.assert_within(g["initial_state"][b], want, STATE * want.abs(), f"d_initial_state of token {t}")
